// Tensor memory of an SM among the CTAs that are resident on it.  Host only.
#pragma once

#include <algorithm>
#include <cstddef>

namespace moe {

// tcgen05.alloc waits, without a limit, until an SM has the columns it asks
// for, and the hardware places CTAs by registers, threads and shared memory
// alone.  CTAs of a cluster wait for one another, so two clusters of different
// calls (two streams) that each hold columns on one SM and wait for them on
// another would wait forever.  No allocation ever waits when the CTAs that fit
// an SM's shared memory fit its tensor memory, and so a kernel asks for at
// least its columns' share of the shared memory, used or not:
//   up to 256 columns: 440 bytes a column (512 columns and 32 more, the
//   smallest allocation, take 440 * 544 > kSmSmemBytes);
//   all 512: so much that no CTA of kMinTmemSmem fits beside it, which every
//   kernel that allocates fewer takes.  (What remains is for the prologue of
//   the next kernel on the stream.)
constexpr size_t kSmSmemBytes = 228 * 1024;      // of an SM
constexpr size_t kCtaSmemReserve = 1024;         // taken for every CTA besides its own
constexpr int kTmemColumns = 512;
constexpr size_t kTmemColumnSmem = 440;
constexpr size_t kMinTmemSmem = 36 * 1024;
constexpr size_t kAllTmemSmem = 192 * 1024;
static_assert(kTmemColumnSmem * (kTmemColumns + 32) > kSmSmemBytes, "CTAs with part of the columns");
static_assert(kAllTmemSmem + kMinTmemSmem + 2 * kCtaSmemReserve > kSmSmemBytes, "CTAs with all and with part");
static_assert(2 * (kAllTmemSmem + kCtaSmemReserve) > kSmSmemBytes, "two CTAs with all");

// Dynamic shared memory to ask for by a kernel that uses `smem` bytes and
// allocates `cols` columns (a power of two, 32 to 512)
inline size_t tmem_smem(size_t smem, int cols) {
  return std::max(smem, cols == kTmemColumns ? kAllTmemSmem
                                             : std::max(kMinTmemSmem, kTmemColumnSmem * (size_t)cols));
}

}  // namespace moe
