// The dense operators' products on the 5th-generation tensor cores (sm_100a).
//
//   acc[m, n] = sum_k A(m, k) B(n, k),  fp32 accumulators in TMEM
//
// One persistent CTA pair per two SMs, tiles of 256 rows x bn columns (bn 256
// or 128).  Per 64-wide k-block each CTA of the pair stages 128 rows of A and
// half of the B tile by TMA (128-byte swizzle) into a six-stage ring, and the
// even CTA issues tcgen05.mma.cta_group::2, which reads both CTAs' shared
// memory: 32 KB a CTA and k-block instead of the 48 KB that a 128 x 256 tile
// of one CTA takes, whose shared-memory traffic would bound it.  Either operand may be
// K-major or MN-major in memory (x W^T; dz W; dz^T x), so no transposed copy
// is ever made.  The accumulators are double-buffered: the epilogue of a tile
// runs beside the products of the next.  Measured: 8192 x 4096 x 8192 bf16 with
// bias and GELU in 360 us alone (1.53 PFLOP/s, tensor pipe 88% busy), 1.27 in
// the power-limited steady state; dx, dW1, dW3, dW2 of an 8192 x 2048 x 5632
// block in one launch, 630 us (1.5 PFLOP/s).  At K = 2048 a tile's MMAs take
// 16400 cycles and its epilogue 5700 (store), 9000 (residual) or 20000 and more
// (gradients), which then bounds it; fp32 4096^3: 650 us with its
// splits (212 TFLOP/s).
//
//   warp 0     TMA producer             warp 2     TMEM allocation
//   warp 1     MMA issuer (even CTA)    warps 4-11 epilogue, a TMEM lane
//                                                  (= row of the tile) a thread
//
// A product may run over several segments of k (dx = dA W1 + dU W3) and a
// launch over up to four products (dx and the weight gradients), so that they
// share one last wave.  Every wait is bounded; on expiry the kernel sets the
// timeout bit of the workspace's error word, lets its copies and MMAs in
// flight finish (bounded) and returns.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "dense_internal.h"
#include "dense_math.cuh"
#include "sm100_ptx.cuh"
#include "tmem_share.h"

namespace moe {
namespace {

constexpr int BM = 128;                 // rows of a CTA's half tile
constexpr int BK = 64;
constexpr int kBks = 2;                      // k-blocks of a stage
constexpr int kStages = 6 / kBks;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 128 + 32 * kEpiWarps;
constexpr int kRegsLaunch = 168, kRegsLow = 88, kRegsHigh = 208;
constexpr int kAccCols = 256;
constexpr int kTmemCols = 512;
constexpr uint32_t kABytes = BM * BK * 2;
constexpr int kGroupM = 16;                  // row tiles of a raster group
constexpr int kMaxProblems = 4;
constexpr int kMaxSegs = 12;

// fp32 products (planes, see dense_pack.cu): the accumulator is read out every
// chunk of kBks k-blocks and the chunks are added in registers.  The tensor
// core adds into its accumulator with truncation, about half an ulp of the
// accumulator lost towards zero an MMA (measured: 2.6e-6 relative after 49 of
// them); eight MMAs of leading products a chunk keep that below 4e-7 for any
// K.  The small products come first in a chunk, while the accumulator is small.
template <typename T>
constexpr bool kChunked = sizeof(T) == 4;

// kDenseGatedGrad with outputs in two planes (bf16 calls of very few rows): an
// instance of its own, the second pass costs the first one registers
constexpr int kGradPlanes = 16;
__host__ __device__ constexpr bool is_grad(int epi) { return epi == kDenseGatedGrad || epi == kGradPlanes; }

// A stretch of k-blocks: tensor map and plane (third coordinate) of each operand
struct Seg {
  uint8_t a, az, b, bz;
};

struct TcProblem {
  CUtensorMap a[2], b[2];
  int64_t M;
  int32_t N, KB;                 // k-blocks of one segment
  int32_t segs, amn, bmn;        // segments; A / B MN-major
  Seg seg[kMaxSegs];
  int32_t tiles_m, tile_end;     // row tiles; tiles of this and the problems before it
  const void *bias, *bias3, *residual, *pre_in, *pre3_in;
  void *out, *pre, *pre3, *out2, *out3;
  int64_t ld_r, ld_o, lo_stride;
};

struct TcParams {
  TcProblem pr[kMaxProblems];
  // the shared tail: tiles from dp_tiles on are cut into steps (below), laid
  // end to end and split evenly over `workers` pairs.  Problem p's tail tiles
  // are [tail_tile[p], tile_end), their steps [tail_step[p], tail_step[p+1])
  int32_t dp_tiles, workers, tail_tile[kMaxProblems];
  int64_t tail_step[kMaxProblems + 1];
  float *part;                   // partial tiles, two slots a worker
  int32_t nprob, act;
  int32_t bn, bnh;               // accumulator columns; output columns of a tile
  uint32_t *err;
};

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// tma_load_3d_pair to a shared-memory address
__device__ __forceinline__ void tma_load_3d_at(uint32_t dst, const CUtensorMap *map, uint32_t bar, int c0, int c1,
                                               int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

struct TilePos {
  int m, n;
};

// Raster order within a problem: groups of kGroupM row tiles, columns outer
// within a group, so that the pairs at work share few row and column panels
// in L2.
__device__ __forceinline__ TilePos tile_pos(const TcParams &P, int p, int t) {
  const int first = p ? P.pr[p - 1].tile_end : 0;
  t -= first;
  const int tm = P.pr[p].tiles_m, tn = (P.pr[p].tile_end - first) / tm;
  const int g = t / (kGroupM * tn), in = t - g * kGroupM * tn;
  const int gm = min(kGroupM, tm - g * kGroupM);
  return {g * kGroupM + in % gm, in / gm};
}

// ----------------------------------- work ---------------------------------------
// A tile's steps are the fills of its ring stages: kBks k-blocks of one
// segment.  bf16: segment by segment; fp32 (chunked): k-block pair by pair, all
// segments of each.  A pair's work: whole tiles of the full waves, dealt
// round-robin, then its share of the tail.  A tile cut between pairs is summed
// by whichever of its pieces is finished last, in the pieces' order: nobody
// ever waits for another pair, and the result does not depend on which it was.
struct Piece {
  int tile, p;                   // p: its problem
  int s0, s1, steps;             // steps [s0, s1) of the tile's
  int index, count;              // this piece among the tile's
  int slot;                      // partial tile of this piece (worker * 2 + 0 / 1)
  int first_worker, tail;        // worker of piece 0; tile's number in the tail
  __device__ __forceinline__ bool whole() const { return count == 1; }
};

template <typename T>
__device__ __forceinline__ int steps_of(const TcProblem &Q) {
  return (Q.KB + kBks - 1) / kBks * Q.segs;
}

template <typename T>
struct Work {
  const TcParams &P;
  const int pair, npairs;
  int t;
  int64_t x, x1;                 // what is left of the tail share
  __device__ Work(const TcParams &p, int pair_, int npairs_) : P(p), pair(pair_), npairs(npairs_), t(pair_) {
    const int64_t R = p.tail_step[p.nprob];
    x = pair < p.workers ? R * pair / p.workers : 0;
    x1 = pair < p.workers ? R * (pair + 1) / p.workers : 0;
  }
  // the worker whose share holds step y
  __device__ __forceinline__ int owner(int64_t y) const {
    return (int)(((y + 1) * P.workers - 1) / P.tail_step[P.nprob]);
  }
  __device__ __forceinline__ bool next(Piece &q) {
    if (t < P.dp_tiles) {
      q.tile = t;
      q.p = 0;
      while (q.p + 1 < P.nprob && t >= P.pr[q.p].tile_end) ++q.p;
      q.steps = steps_of<T>(P.pr[q.p]);
      q.s0 = 0;
      q.s1 = q.steps;
      q.index = 0;
      q.count = 1;
      t += npairs;
      return true;
    }
    if (x >= x1) return false;
    q.p = 0;
    while (x >= P.tail_step[q.p + 1]) ++q.p;
    q.steps = steps_of<T>(P.pr[q.p]);
    const int64_t in = x - P.tail_step[q.p];
    const int k = (int)(in / q.steps);
    const int64_t begin = P.tail_step[q.p] + (int64_t)k * q.steps;      // the tile's first step
    q.tile = P.tail_tile[q.p] + k;
    q.s0 = (int)(x - begin);
    q.s1 = (int)min((int64_t)q.steps, x1 - begin);
    q.first_worker = owner(begin);
    q.index = pair - q.first_worker;
    q.count = owner(begin + q.steps - 1) - q.first_worker + 1;
    q.slot = 2 * pair + (q.index == 0 ? 1 : 0);
    q.tail = q.tile - P.dp_tiles;
    x = begin + q.s1;
    return true;
  }
};

// ------------------------------- epilogue pieces --------------------------------
// A warp moves its 32 rows in chunks of CW columns (64 bytes of a row: four
// 16-byte pieces).  A thread owns a row; memory is touched by whole row
// pieces, eight rows an instruction.  Between the two layouts lies the warp's
// staging buffer, piece c of row r at slot c ^ (r / 2 mod 4): free of bank
// conflicts both ways.
template <typename T>
constexpr int kCols = 64 / sizeof(T);
constexpr int kStgBytes = 32 * 64;

__device__ __forceinline__ int stg_at(int r, int c) { return r * 4 + (c ^ ((r >> 1) & 3)); }

// A [M, N] matrix the epilogue reads or writes; vec: its rows are 16-byte
// aligned, so whole pieces move at once
template <typename T>
struct Rows {
  static constexpr int E = 16 / sizeof(T);
  T *p;
  int64_t ld, M;
  int N;
  bool vec;
  __device__ Rows(const void *q, int64_t ld_, int64_t M_, int N_)
      : p(static_cast<T *>(const_cast<void *>(q))), ld(ld_), M(M_), N(N_),
        vec(((reinterpret_cast<uintptr_t>(q) | (uintptr_t)(ld_ * (int64_t)sizeof(T))) & 15) == 0) {}
  // the chunk moves in whole pieces (of the rows and pieces that exist): one
  // branch a chunk, predicates within it (a branch a piece serialises the
  // accesses: the gradient epilogue alone took 211 us with it, 160 without)
  __device__ __forceinline__ bool pieces(int col) const { return vec && (col + kCols<T> <= N || N % E == 0); }
};

// Element by element, for rows that are not 16-byte aligned and the matrix's
// edges: instruction i of a warp covers 32 consecutive elements of the chunk,
// so that its lanes touch whole row stretches.  Calls of their own, so that
// the common path keeps its registers and its instruction cache lines.
template <typename T>
__device__ __forceinline__ T &staged(uint4 *stg, int r, int c) {
  constexpr int E = 16 / sizeof(T);
  return reinterpret_cast<T *>(stg + stg_at(r, c / E))[c % E];
}
// p: row row0, column col; rows, cols: what lies inside the matrix
template <typename T>
__device__ __noinline__ void store_edge(T *p, int64_t ld, int rows, int cols, uint4 *stg, int lane) {
  constexpr int CW = kCols<T>;
#pragma unroll 8
  for (int i = 0; i < CW; ++i) {
    const int r = i * (32 / CW) + lane / CW, c = lane % CW;
    if (r < rows && c < cols) p[r * ld + c] = staged<T>(stg, r, c);
  }
}
template <typename T>
__device__ __noinline__ void load_edge(const T *p, int64_t ld, int rows, int cols, uint4 *stg, int lane) {
  constexpr int CW = kCols<T>;
  T v[CW];                       // all of them in flight
#pragma unroll
  for (int i = 0; i < CW; ++i) {
    const int r = i * (32 / CW) + lane / CW, c = lane % CW;
    from_f32(v[i], 0.0f);
    if (r < rows && c < cols) v[i] = p[r * ld + c];
  }
#pragma unroll
  for (int i = 0; i < CW; ++i) staged<T>(stg, i * (32 / CW) + lane / CW, lane % CW) = v[i];
}

// each thread's row, four packed pieces, to rows row0 ... of `o`
template <typename T>
__device__ __forceinline__ void store_chunk(const Rows<T> &o, int64_t row0, int col, const uint4 (&w)[4],
                                            uint4 *stg, int lane) {
#pragma unroll
  for (int c = 0; c < 4; ++c) stg[stg_at(lane, c)] = w[c];
  __syncwarp();
  const int r0 = lane / 4, c = lane % 4;
  if (o.pieces(col)) {
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = stg[stg_at(i * 8 + r0, c)];
    T *q = o.p + (row0 + r0) * o.ld + col + c * o.E;
    const int rows = col + c * o.E < o.N ? (int)min((int64_t)32, o.M - row0) : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i * 8 + r0 < rows) *reinterpret_cast<uint4 *>(q + i * 8 * o.ld) = v[i];
  } else {
    store_edge<T>(o.p + row0 * o.ld + col, o.ld, (int)min((int64_t)32, o.M - row0), o.N - col, stg, lane);
  }
  __syncwarp();
}

template <typename T>
__device__ __forceinline__ void store_vals(const Rows<T> &o, int64_t row0, int col, const float (&v)[kCols<T>],
                                           uint4 *stg, int lane) {
  uint4 w[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) w[c] = pack16<T>(v + c * o.E);
  store_chunk(o, row0, col, w, stg, lane);
}

// 16 bytes of what rounding v to T leaves
template <typename T>
__device__ __forceinline__ uint4 low16(const float *v) {
  constexpr int E = 16 / sizeof(T);
  float h[E];
  unpack16<T>(pack16<T>(v), h);
#pragma unroll
  for (int i = 0; i < E; ++i) h[i] = rest_of(v[i], h[i]);
  return pack16<T>(h);
}
// 16 bytes; the 256-byte stretch around them is brought to L2, where the
// chunks to come find it
__device__ __forceinline__ uint4 ld16_ahead(const void *p) {
  uint4 v;
  asm volatile("ld.global.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// a chunk on its way in: whole row pieces in registers, then staged so that
// each thread finds its row (after a __syncwarp); a chunk that does not move
// in whole pieces is read when it is staged (zeros beyond the matrix)
template <typename T>
struct Incoming {
  uint4 w[4];
  __device__ __forceinline__ void fetch(const Rows<T> &o, int64_t row0, int col, int lane) {
    if (!o.pieces(col)) return;
    const T *q = o.p + (row0 + lane / 4) * o.ld + col + lane % 4 * o.E;
    const int rows = col + lane % 4 * o.E < o.N ? (int)min((int64_t)32, o.M - row0) : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = make_uint4(0, 0, 0, 0);
      if (i * 8 + lane / 4 < rows) w[i] = ld16_ahead(q + i * 8 * o.ld);
    }
  }
  __device__ __forceinline__ void stage(const Rows<T> &o, int64_t row0, int col, uint4 *stg, int lane) const {
    if (o.pieces(col)) {
#pragma unroll
      for (int i = 0; i < 4; ++i) stg[stg_at(i * 8 + lane / 4, lane % 4)] = w[i];
    } else {
      load_edge<T>(o.p + row0 * o.ld + col, o.ld, (int)min((int64_t)32, o.M - row0), o.N - col, stg, lane);
    }
  }
};

// columns [taddr, taddr + N) of this thread's TMEM lane
template <int N>
__device__ __forceinline__ void acc_cols(uint32_t taddr, float (&v)[N]) {
  uint32_t r[N];
  if constexpr (N == 32) tmem_ld32(taddr, r);
  else tmem_ld16(taddr, r);
  tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = __uint_as_float(r[i]);
}

template <int N>
__device__ __forceinline__ void add_bias(float (&v)[N], const float *bias) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const float4 b = *reinterpret_cast<const float4 *>(bias + i);
    const float2 p = add2(make_float2(v[i], v[i + 1]), make_float2(b.x, b.y));
    const float2 q = add2(make_float2(v[i + 2], v[i + 3]), make_float2(b.z, b.w));
    v[i] = p.x;
    v[i + 1] = p.y;
    v[i + 2] = q.x;
    v[i + 3] = q.y;
  }
}

// This warp's 32 rows (row0 ...) x columns [c0, c1) of the tile's output
// columns (the tile's first is col0) from the accumulator at taddr.  sb: the
// bias of those columns in shared memory (gated: W1's, then W3's).  What the
// epilogue reads from global memory does not depend on the accumulator: each
// chunk's is fetched a chunk ahead, the first (begin) before the wait for
// the accumulator.
template <int EPI, typename T>
struct Epilogue {
  static constexpr bool FAST = sizeof(T) == 2;
  static constexpr int CW = kCols<T>, E = 16 / sizeof(T);
  static constexpr int kIn = is_grad(EPI) ? 2 : 1;      // matrices read, staging buffers
  const TcParams &P;
  const TcProblem &Q;
  const int64_t row0;
  const int col0, c0, c1, lane;
  uint4 *stg;
  Incoming<T> in[kIn];

  __device__ Epilogue(const TcParams &p, const TcProblem &q, int64_t row, int col, int a, int b, uint8_t *st, int l)
      : P(p), Q(q), row0(row), col0(col), c0(a), c1(min(b, q.N - col)), lane(l),
        stg(reinterpret_cast<uint4 *>(st)) {}

  __device__ __forceinline__ Rows<T> packed(const void *p) const { return Rows<T>(p, Q.N, Q.M, Q.N); }

  __device__ __forceinline__ void fetch(int c) {
    if (row0 >= Q.M || c >= c1) return;
    if (EPI == kDenseLinear && Q.residual)
      in[0].fetch(Rows<T>(Q.residual, Q.ld_r, Q.M, Q.N), row0, col0 + c, lane);
    if (is_grad(EPI)) {
      in[0].fetch(packed(Q.pre_in), row0, col0 + c, lane);
      in[kIn - 1].fetch(packed(Q.pre3_in), row0, col0 + c, lane);
    }
  }
  __device__ __forceinline__ void begin() { fetch(c0); }

  __device__ __forceinline__ void run(uint32_t taddr, const float *sb) {
    if (row0 >= Q.M) return;
    const Rows<T> out(Q.out, Q.ld_o, Q.M, Q.N);
    for (int c = c0; c < c1; c += CW) {
      float v[CW];
      const int col = col0 + c;
      if (EPI == kDenseStore) {
        acc_cols(taddr + c, v);
        store_vals(out, row0, col, v, stg, lane);
      } else if (EPI == kDenseLinear) {
        acc_cols(taddr + c, v);
        if (Q.bias) add_bias(v, sb + c - c0);
        if (Q.pre) store_vals(packed(Q.pre), row0, col, v, stg, lane);
        with_act(P.act, [&](auto A) {
#pragma unroll
          for (int i = 0; i < CW; i += 2) {
            const float2 y = act_fwd2<FAST, decltype(A)::value>(make_float2(v[i], v[i + 1]));
            v[i] = y.x;
            v[i + 1] = y.y;
          }
        });
        if (Q.residual) {
          in[0].stage(Rows<T>(Q.residual, Q.ld_r, Q.M, Q.N), row0, col, stg, lane);
          __syncwarp();
          fetch(c + CW);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float r[E];
            unpack16<T>(stg[stg_at(lane, k)], r);
#pragma unroll
            for (int i = 0; i < E; i += 2) {
              const float2 y = add2(make_float2(v[k * E + i], v[k * E + i + 1]), make_float2(r[i], r[i + 1]));
              v[k * E + i] = y.x;
              v[k * E + i + 1] = y.y;
            }
          }
          __syncwarp();
        }
        store_vals(out, row0, col, v, stg, lane);
      } else if (EPI == kDenseGated) {
        float u[CW];
        acc_cols(taddr + c, v);
        acc_cols(taddr + P.bnh + c, u);
        if (Q.bias) {
          add_bias(v, sb + c - c0);
          add_bias(u, sb + kAccCols / 4 + c - c0);
        }
        if (Q.pre) {
          store_vals(packed(Q.pre), row0, col, v, stg, lane);
          store_vals(packed(Q.pre3), row0, col, u, stg, lane);
        }
        with_act(P.act, [&](auto A) {
#pragma unroll
          for (int i = 0; i < CW; i += 2) {
            const float2 f = act_fwd2<FAST, decltype(A)::value>(make_float2(v[i], v[i + 1]));
            const float2 y = mul2(f, make_float2(u[i], u[i + 1]));
            v[i] = y.x;
            v[i + 1] = y.y;
          }
        });
        store_vals(out, row0, col, v, stg, lane);
      } else {                                           // kDenseGatedGrad
        // a and u staged side by side; dA, dU and h packed piece by piece, so
        // that no more than one matrix is held in fp32
        acc_cols(taddr + c, v);
        // low: a pass of its own for the second planes, the parts that the
        // first one's rounding left (few rows only)
        auto grads = [&](auto low) {
          constexpr bool LOW = decltype(low)::value;
          if (LOW) fetch(c);
          uint4 *stg_u = stg + (kIn - 1) * (kStgBytes / 16);
          in[0].stage(packed(Q.pre_in), row0, col, stg, lane);
          in[kIn - 1].stage(packed(Q.pre3_in), row0, col, stg_u, lane);
          __syncwarp();
          fetch(c + CW);
          uint4 wa[4], wu[4], wh[4];
          with_act(P.act, [&](auto A) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              float a[E], u[E], h[E];
              unpack16<T>(stg[stg_at(lane, k)], a);
              unpack16<T>(stg_u[stg_at(lane, k)], u);
#pragma unroll
              for (int i = 0; i < E; i += 2) {
                float2 f, d;
                act_both2<FAST, decltype(A)::value>(make_float2(a[i], a[i + 1]), f, d);
                const float2 dh = make_float2(v[k * E + i], v[k * E + i + 1]), uu = make_float2(u[i], u[i + 1]);
                const float2 da = mul2(mul2(dh, uu), d), hh = mul2(f, uu), du = mul2(dh, f);
                a[i] = da.x;
                a[i + 1] = da.y;
                h[i] = hh.x;
                h[i + 1] = hh.y;
                u[i] = du.x;
                u[i + 1] = du.y;
              }
              wa[k] = LOW ? low16<T>(a) : pack16<T>(a);
              wu[k] = LOW ? low16<T>(u) : pack16<T>(u);
              wh[k] = LOW ? low16<T>(h) : pack16<T>(h);
            }
          });
          __syncwarp();
          const int64_t at = LOW ? Q.lo_stride : 0;
          store_chunk(Rows<T>(static_cast<T *>(Q.out) + at, Q.ld_o, Q.M, Q.N), row0, col, wa, stg, lane);
          store_chunk(Rows<T>(static_cast<T *>(Q.out2) + at, Q.ld_o, Q.M, Q.N), row0, col, wu, stg, lane);
          store_chunk(Rows<T>(static_cast<T *>(Q.out3) + at, Q.ld_o, Q.M, Q.N), row0, col, wh, stg, lane);
        };
        grads(IntC<0>{});
        if constexpr (EPI == kGradPlanes) grads(IntC<1>{});
      }
    }
  }
};

// 32 accumulator columns back into this thread's TMEM lane
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float (&v)[32]) {
  uint32_t r[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(v[i]);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
      "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
      "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Accumulator column of a warp's group i of 32 (its half of the output
// columns; gated: of the gate's, then of the up-projection's); -1: none
// (cols: the tile's output columns that exist)
template <int EPI>
__device__ __forceinline__ int group_col(int bnh, int cols, int half, int i) {
  const int w = bnh / 2, g = EPI == kDenseGated ? i >> 1 : 0, c = 32 * (EPI == kDenseGated ? i & 1 : i);
  return c < w && half * w + c < cols ? g * bnh + half * w + c : -1;
}

// fp32: the accumulators of a piece's chunks, one after another, into a sum in
// registers, which takes the last one's place in TMEM at the end.  Returns the
// accumulator it is in (bit 0) and its phase (bit 1), -1 after a wait that ran
// out.  A call of its own: the sum takes 128 registers, and what the caller
// keeps is spilled once a tile instead of once a chunk.
struct ChunkWaits {
  uint64_t *full;
  uint32_t empty0, empty1;           // the even CTA's
  volatile int *abort;
  uint32_t *err;
  uint64_t limit;
};
template <int EPI>
__device__ __noinline__ int sum_chunks(const ChunkWaits w, uint32_t tmem, int bnh, int cols, int half, int chunks,
                                       int acc, uint32_t phase) {
  float sum[4][32] = {};
  for (int c = 0;; ++c) {
    if (!__all_sync(0xffffffffu, mbar_wait(w.full + acc, phase, w.abort, w.err, w.limit))) return -1;
    tc_fence_after();
    const uint32_t ta = tmem + (uint32_t)(acc * kAccCols);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int col = group_col<EPI>(bnh, cols, half, i);
      if (col >= 0) {
        uint32_t r[32];
        tmem_ld32(ta + col, r);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 32; ++j) sum[i][j] += __uint_as_float(r[j]);
        if (c + 1 == chunks) tmem_st32(ta + col, sum[i]);
      }
    }
    if (c + 1 == chunks) break;
    tc_fence_before();
    mbar_arrive_cluster(acc ? w.empty1 : w.empty0);
    if (++acc == 2) {
      acc = 0;
      phase ^= 1u;
    }
  }
  tmem_st_wait();
  return acc | (int)(phase << 1);
}

// A piece that is not the whole tile: this warp's part of the accumulator to
// the piece's slot, then a count of the pieces that are there.  The warp that
// finds itself last adds the tile's pieces in order, puts the sum in TMEM and
// returns true.  A field of four bits a warp counts its pieces (at most
// kMaxPieces) and is back at zero afterwards, for the next launch.
constexpr int kMaxPieces = 14;
constexpr size_t kTailCountOffset = 1024;             // into the workspace's control block
constexpr int kMaxTail = 320;                         // tiles of the tail at most
constexpr int64_t kSlotFloats = 2 * BM * kAccCols;    // a pair's accumulators
static_assert(kTailCountOffset + 4 * 2 * kMaxTail <= kCtrlBytes, "counters of the tail");

template <int EPI>
__device__ __noinline__ bool join_pieces(float *parts, uint32_t *count, int bnh, int cols, int slot, int first_worker, int pieces,
                                         uint32_t ta, int rank, int ew, int lane) {
  const int half = ew >> 2;
  auto at = [&](int64_t slot) {
    return reinterpret_cast<float4 *>(parts + slot * kSlotFloats) + (rank * kEpiWarps + ew) * (4 * 8 * 32) + lane;
  };
  float4 *mine = at(slot);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int col = group_col<EPI>(bnh, cols, half, i);
    if (col < 0) continue;
    uint32_t r[32];
    tmem_ld32(ta + col, r);
    tmem_ld_wait();
#pragma unroll
    for (int j = 0; j < 8; ++j)
      __stcg(mine + (i * 8 + j) * 32, make_float4(__uint_as_float(r[4 * j]), __uint_as_float(r[4 * j + 1]),
                                                  __uint_as_float(r[4 * j + 2]), __uint_as_float(r[4 * j + 3])));
  }
  __threadfence();
  __syncwarp();
  int last = 0;
  if (lane == 0) {
    const uint32_t old = atomicAdd(count, 1u << (4 * ew));
    last = (int)((old >> (4 * ew)) & 15u) == pieces - 1;
    if (last) atomicSub(count, (uint32_t)pieces << (4 * ew));
  }
  last = __shfl_sync(0xffffffffu, last, 0);
  if (!last) return false;
  __threadfence();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int col = group_col<EPI>(bnh, cols, half, i);
    if (col < 0) continue;
    // two pieces in flight
    float v[32] = {};
    for (int k = 0; k < pieces; k += 2) {
      float4 f[2][8];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (k + h >= pieces) break;
        // piece 0 is the end of its worker's share, the others begin theirs
        const float4 *src = at(2 * (first_worker + k + h) + (k + h == 0 ? 1 : 0)) + i * 8 * 32;
#pragma unroll
        for (int j = 0; j < 8; ++j) f[h][j] = __ldcg(src + j * 32);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (k + h >= pieces) break;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[4 * j] += f[h][j].x;
          v[4 * j + 1] += f[h][j].y;
          v[4 * j + 2] += f[h][j].z;
          v[4 * j + 3] += f[h][j].w;
        }
      }
    }
    tmem_st32(ta + col, v);
  }
  tmem_st_wait();
  return true;
}

// --------------------------------- the kernel ----------------------------------
template <int EPI, typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    dense_pair_kernel(const __grid_constant__ TcParams P) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full_bar[kStages];
  __shared__ __align__(8) uint64_t empty_bar[kStages];
  __shared__ __align__(8) uint64_t accf_bar[2];
  __shared__ __align__(8) uint64_t acce_bar[2];
  __shared__ __align__(8) uint64_t drain_bar;
  __shared__ __align__(16) float s_bias[kEpiWarps][kAccCols / 2];     // each epilogue warp's columns
  __shared__ uint32_t s_tmem_base;
  __shared__ volatile int s_abort;
  __shared__ uint64_t s_limit_sh;

  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const uint32_t b_bytes = (uint32_t)(P.bn / 2) * BK * 2;
  const uint32_t stage_bytes = kBks * (kABytes + b_bytes);       // A blocks, then B blocks
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;

  if (tid == 32) {
    for (int st = 0; st < kStages; ++st) {
      mbar_init(&full_bar[st], 1);
      mbar_init(&empty_bar[st], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&accf_bar[a], 1);
      mbar_init(&acce_bar[a], 2 * kEpiWarps * 32);
    }
    mbar_init(&drain_bar, 1);
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem_base)),
                 "r"(kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  if (tid == 0) {
    tma_prefetch_map(&P.pr[0].a[0]);
    tma_prefetch_map(&P.pr[0].b[0]);
  }
  pdl_wait();
  pdl_trigger();
  if (tid == 0) s_limit_sh = wait_limit_ns(P.err);
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = s_tmem_base;
  const uint64_t s_limit = s_limit_sh;

  // Registers: 168 a thread at launch (384 threads); the four warps of the
  // first warpgroup give most of theirs to the epilogue:
  // 128 * 88 + 256 * 208 = 384 * 168
  static_assert(128 * kRegsLow + 256 * kRegsHigh <= kThreads * kRegsLaunch, "registers of the block");
  if (warp < 4) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLow));
  if (warp == 0 && lane == 0) {
    // ------------------------------ TMA producer ------------------------------
    int stage = 0;
    uint32_t phase = 0, armed = 0, armed_parity = 0;
    const uint32_t smem0 = smem_u32(smem), fb0 = smem_u32(full_bar) & 0xFEFFFFFFu;      // the even CTA's barriers
    const bool wide = P.bn == 256;
    // k-blocks [kb, kb1) of one segment; the operand orders are constants of the
    // loop (a stage has to be refilled within the time of one stage's MMAs)
    auto fill = [&](auto amn, auto bmn, const CUtensorMap *ma, const CUtensorMap *mb, int am, int bn0, int kb,
                    int kb1, Seg S) -> bool {
      for (; kb < kb1; kb += kBks) {
        if (!mbar_wait(&empty_bar[stage], phase ^ 1u, &s_abort, P.err, s_limit)) return false;
        uint32_t sa = smem0 + (uint32_t)stage * stage_bytes, sb = sa + kBks * kABytes;
        const uint32_t fb = fb0 + 8 * stage;
        const int nq = min(kBks, kb1 - kb);
        if (rank == 0) {
          mbar_expect_tx(&full_bar[stage], 2 * nq * (kABytes + b_bytes));
          armed |= 1u << stage;
          armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
        }
#pragma unroll
        for (int q2 = 0; q2 < kBks; ++q2) {
          if (q2 >= nq) break;
          const int k = (kb + q2) * BK;
          if (decltype(amn)::value) {
            tma_load_3d_at(sa, ma, fb, am, k, S.az);
            tma_load_3d_at(sa + 8192, ma, fb, am + 64, k, S.az);
          } else {
            tma_load_3d_at(sa, ma, fb, k, am, S.az);
          }
          if (decltype(bmn)::value) {
            tma_load_3d_at(sb, mb, fb, bn0, k, S.bz);
            if (wide) tma_load_3d_at(sb + 8192, mb, fb, bn0 + 64, k, S.bz);
          } else {
            tma_load_3d_at(sb, mb, fb, k, bn0, S.bz);
          }
          sa += kABytes;
          sb += b_bytes;
        }
        if (++stage == kStages) { stage = 0; phase ^= 1u; }
      }
      return true;
    };
    bool ok = true;
    Work<T> work(P, pair, npairs);
    Piece w;
    while (ok && work.next(w)) {
      const TilePos q = tile_pos(P, w.p, w.tile);
      const TcProblem &Q = P.pr[w.p];
      const int am = q.m * 2 * BM + (int)rank * BM;
      // gated: the even CTA stages rows of W1, the odd one the same rows of W3
      const int bn0 = q.n * P.bnh + (EPI == kDenseGated ? 0 : (int)rank * (P.bn / 2));
      // runs of steps in one segment
      const int per = kChunked<T> ? 1 : w.steps / Q.segs;
      for (int st = w.s0, run; ok && st < w.s1; st += run) {
        const int sg = kChunked<T> ? st % Q.segs : st / per;
        const int i = kChunked<T> ? st / Q.segs : st - sg * per;
        run = kChunked<T> ? 1 : min(per - i, w.s1 - st);
        const int kb = i * kBks, kb1 = min(Q.KB, (i + run) * kBks);
        const Seg S = Q.seg[sg];
        const CUtensorMap *ma = &Q.a[S.a];
        const CUtensorMap *mb = &Q.b[EPI == kDenseGated ? (int)rank : S.b];
        if (Q.amn) {
          ok = Q.bmn ? fill(IntC<1>{}, IntC<1>{}, ma, mb, am, bn0, kb, kb1, S)
                     : fill(IntC<1>{}, IntC<0>{}, ma, mb, am, bn0, kb, kb1, S);
        } else {
          ok = Q.bmn ? fill(IntC<0>{}, IntC<1>{}, ma, mb, am, bn0, kb, kb1, S)
                     : fill(IntC<0>{}, IntC<0>{}, ma, mb, am, bn0, kb, kb1, S);
        }
      }
    }
    if (!ok && rank == 0) {
      for (int st = 0; st < kStages; ++st)
        if (armed & (1u << st)) mbar_wait_drain(&full_bar[st], (armed_parity >> st) & 1u);
    }
  } else if (warp == 1 && lane == 0 && rank == 0) {
    // ------------------------ MMA issuer (even CTA only) ------------------------
    // (K-major: a K step of 16 is 32 bytes on; MN-major: 16 lines of 128 bytes)
    const uint32_t smem0 = smem_u32(smem);
    int stage = 0, acc = 0;
    uint32_t phase = 0, acc_phase = 0;
    bool ok = true;
    Work<T> work(P, pair, npairs);
    Piece w;
    while (ok && work.next(w)) {
      const TcProblem &Q = P.pr[w.p];
      const int KB = Q.KB, segs = Q.segs, per = kChunked<T> ? segs : w.steps / segs;
      const bool amn = Q.amn, bmn = Q.bmn;
      const uint32_t idesc = idesc_bf16(2 * BM, P.bn) | (amn ? 1u << 15 : 0u) | (bmn ? 1u << 16 : 0u);
      // descriptors of stage 0; the address field counts 16 bytes
      const uint64_t adesc = amn ? mn128_desc(smem0) : sw128_desc(smem0);
      const uint64_t bdesc = bmn ? mn128_desc(smem0 + kBks * kABytes) : sw128_desc(smem0 + kBks * kABytes);
      const uint32_t astep = amn ? 2048 >> 4 : 32 >> 4, bstep = bmn ? 2048 >> 4 : 32 >> 4;
      // one accumulator a piece (fp32: a chunk of it)
      for (int st = w.s0; ok && st < w.s1;) {
        if (!mbar_wait<true>(&acce_bar[acc], acc_phase ^ 1u, &s_abort, P.err, s_limit)) { ok = false; break; }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + (uint32_t)(acc * kAccCols);
        const int end = kChunked<T> ? min(w.s1, st - st % segs + segs) : w.s1;
        int i = kChunked<T> ? st / segs : st % per;          // step within its segment
        uint32_t accum = 0;
        for (; st < end; ++st) {
          if (!mbar_wait<true>(&full_bar[stage], phase, &s_abort, P.err, s_limit)) { ok = false; break; }
          tc_fence_after();
          uint64_t ad = adesc + (uint32_t)stage * (stage_bytes >> 4), bd = bdesc + (uint32_t)stage * (stage_bytes >> 4);
          const int nq = min(kBks, KB - i * kBks);
          for (int q2 = 0; q2 < nq; ++q2) {
#pragma unroll
            for (int k = 0; k < BK / 16; ++k) {
              umma_bf16_pair(d_tmem, ad + k * astep, bd + k * bstep, idesc, accum);
              accum = 1;
            }
            ad += kABytes >> 4;
            bd += b_bytes >> 4;
          }
          umma_commit_pair_both(&empty_bar[stage]);
          if (++stage == kStages) { stage = 0; phase ^= 1u; }
          if (!kChunked<T> && ++i == per) i = 0;
        }
        if (!ok) break;
        umma_commit_pair_both(&accf_bar[acc]);
        if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
      }
    }
    umma_commit_pair_local(&drain_bar);
    mbar_wait_drain(&drain_bar, 0);
  }
  __syncwarp();
  } else {
    // -------------------------------- epilogue --------------------------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsHigh));
    // two warps a TMEM lane quarter (a warp reaches lanes 32 (warp mod 4) ...
    // of its CTA only), each with half of the tile's columns
    const int ew = warp - 4, quarter = ew & 3, half = ew >> 2;
    uint8_t *stg = smem + (size_t)kStages * stage_bytes + (size_t)ew * (Epilogue<EPI, T>::kIn * kStgBytes);
    const uint32_t acce_even[2] = {mapa_shared(smem_u32(&acce_bar[0]), 0), mapa_shared(smem_u32(&acce_bar[1]), 0)};
    float *sb = s_bias[ew];
    int acc = 0;
    uint32_t acc_phase = 0;
    Work<T> work(P, pair, npairs);
    Piece pc;
    while (work.next(pc)) {
      const TilePos q = tile_pos(P, pc.p, pc.tile);
      const TcProblem &Q = P.pr[pc.p];
      const int col0 = q.n * P.bnh, w = P.bnh / 2;
      if ((EPI == kDenseLinear || EPI == kDenseGated) && Q.bias) {
        for (int i = lane; i < w; i += 32) {
          const int n = col0 + half * w + i;
          sb[i] = n < Q.N ? to_f32(static_cast<const T *>(Q.bias)[n]) : 0.0f;
          if (EPI == kDenseGated)
            sb[kAccCols / 4 + i] = n < Q.N ? to_f32(static_cast<const T *>(Q.bias3)[n]) : 0.0f;
        }
        __syncwarp();
      }
      Epilogue<EPI, T> ep(P, Q, (int64_t)q.m * 2 * BM + rank * BM + quarter * 32, col0, half * w, half * w + w, stg,
                          lane);
      const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
      if (!kChunked<T> && pc.whole()) ep.begin();
      bool ok = true;
      if (kChunked<T>) {
        const int chunks = (pc.s1 - 1) / Q.segs - pc.s0 / Q.segs + 1;
        const ChunkWaits cw{accf_bar, acce_even[0], acce_even[1], &s_abort, P.err, s_limit};
        const int at = sum_chunks<EPI>(cw, tmem_base + lanes, P.bnh, Q.N - col0, half, chunks, acc, acc_phase);
        ok = at >= 0;
        if (ok) {
          acc = at & 1;
          acc_phase = (uint32_t)at >> 1;
          if (pc.whole()) ep.begin();
        }
      } else {
        ok = __all_sync(0xffffffffu, mbar_wait(&accf_bar[acc], acc_phase, &s_abort, P.err, s_limit));
        tc_fence_after();
      }
      if (!ok) break;
      const uint32_t ta = tmem_base + (uint32_t)(acc * kAccCols) + lanes;
      bool finish = true;
      if (!pc.whole()) {
        // (a warp without rows has nothing to join, in any piece)
        finish = ep.row0 < Q.M && join_pieces<EPI>(P.part, P.err + kTailCountOffset / 4 + pc.tail * 2 + rank, P.bnh, Q.N - col0, pc.slot,
                                  pc.first_worker, pc.count, ta, (int)rank, ew, lane);
        if (finish) ep.begin();
      }
      if (finish) ep.run(ta, sb);
      __syncwarp();
      tc_fence_before();
      mbar_arrive_cluster(acce_even[acc]);
      if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
    }
  }

  tc_fence_before();
  cluster_sync_all();              // neither CTA leaves while the pair may still touch it
  tc_fence_after();
  if (warp == 2)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(kTmemCols));
}

// ------------------------------- host side --------------------------------------
constexpr int kMaxDevices = 64;
constexpr int kMaxPairs = 80;           // pairs of a launch at most (slots of the workspace)
constexpr int kJoinSteps = 14, kMinSteps = 8;

// As many CTA pairs as fit at once.  The attribute is set and the occupancy
// asked once a device (a second thread that asks meanwhile gets the same).
template <auto kern>
cudaError_t pairs_of(size_t smem, int *pairs) {
  static std::atomic<int> cache[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int n = dev < kMaxDevices ? cache[dev].load(std::memory_order_acquire) : 0;
  if (n == 0) {
    // the epilogue's larger share must be there: it would wait for it forever
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, kern);
    if (e != cudaSuccess) return e;
    if (fa.numRegs < kRegsLaunch) return cudaErrorInvalidConfiguration;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (device_sms() / 2), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
    if (e != cudaSuccess || n <= 0) {
      cudaGetLastError();
      n = device_sms() / 2;
    }
    if (dev < kMaxDevices) cache[dev].store(n, std::memory_order_release);
  }
  *pairs = n;
  return cudaSuccess;
}

template <int EPI, typename T>
cudaError_t launch_pair_as(TcParams &P, cudaStream_t s) {
  constexpr auto kern = dense_pair_kernel<EPI, T>;
  constexpr size_t smem = 1024 + kStages * kBks * (kABytes + 128 * BK * 2) +
                          kEpiWarps * Epilogue<EPI, T>::kIn * kStgBytes;
  static_assert(smem >= kAllTmemSmem, "beside kernels that allocate fewer columns");
  int pairs = 0;
  const cudaError_t e = pairs_of<kern>(smem, &pairs);
  if (e != cudaSuccess) return e;
  pairs = std::min(pairs, kMaxPairs);
  // The tail: the tiles behind the last full wave, when spreading them over
  // more pairs saves more than joining their pieces costs.  A plain last wave
  // takes a tile's steps; spread over W workers, total / W steps and the join:
  // the partial tiles' way through L2 and back, about kJoinSteps plus two a
  // piece (bf16, 256 x 14336 x 4096: 81 us plain, 51 us in pieces; 512 x 4096 x
  // 14336: 54.5 us plain, 61 us in pieces).  W is a multiple of the tail's
  // tiles where that leaves each tile at least two pieces (a share that
  // straddles two tiles adds a piece to both).
  // Tiles that take more than about half of a pair's fair share of the whole
  // launch are in the tail however many they are.
  const int tiles = P.pr[P.nprob - 1].tile_end;
  auto steps = [&](int p) { return (int64_t)((P.pr[p].KB + kBks - 1) / kBks) * P.pr[p].segs; };
  auto begin = [&](int p) { return p ? P.pr[p - 1].tile_end : 0; };
  int64_t all = 0;
  for (int p = 0; p < P.nprob; ++p) all += steps(p) * (P.pr[p].tile_end - begin(p));
  int dp = tiles - tiles % pairs;
  bool outliers = false;
  for (int p = P.nprob - 1; p >= 0; --p)
    if (2 * steps(p) * pairs > all && tiles - begin(p) <= kMaxTail && begin(p) < dp) {
      dp = begin(p);
      outliers = true;
    }
  P.dp_tiles = tiles;
  P.workers = 0;
  if (dp < tiles && P.part) {
    const int last = tiles - dp;
    int64_t total = 0, deepest = 0;
    for (int p = 0; p < P.nprob; ++p) {
      const int from = std::max(dp, begin(p)), n = std::max(0, P.pr[p].tile_end - from);
      P.tail_tile[p] = from;
      P.tail_step[p] = total;
      total += n * steps(p);
      if (n) deepest = std::max(deepest, steps(p));
    }
    P.tail_step[P.nprob] = total;
    // at least kMinSteps a worker, at most kMaxPieces pieces a tile
    const int64_t least = std::max<int64_t>(kMinSteps, (deepest + kMaxPieces - 3) / (kMaxPieces - 2));
    int workers = (int)std::min<int64_t>(pairs, total / least);
    if (workers >= 2 * last) workers -= workers % last;
    const double plain = outliers ? (double)std::max(deepest, total / pairs) : (double)deepest;
    if (workers > 0 && (double)total / workers + kJoinSteps + 2.0 * deepest * workers / total < plain) {
      P.dp_tiles = dp;
      P.workers = workers;
    }
  }
  if (P.workers == 0)
    for (int p = 0; p <= P.nprob; ++p) P.tail_step[p] = 0;
  const int grid = std::min(pairs, std::max(P.dp_tiles, P.workers));
  return launch_kernel(kern, 2 * (unsigned)grid, kThreads, smem, s, P);
}

template <typename T>
cudaError_t launch_as(int epi, TcParams &P, cudaStream_t s) {
  switch (epi) {
    case kDenseLinear: return launch_pair_as<kDenseLinear, T>(P, s);
    case kDenseGated: return launch_pair_as<kDenseGated, T>(P, s);
    case kDenseGatedGrad:
      if constexpr (sizeof(T) == 2)
        if (P.pr[0].lo_stride) return launch_pair_as<kGradPlanes, T>(P, s);
      return launch_pair_as<kDenseGatedGrad, T>(P, s);
    default: return launch_pair_as<kDenseStore, T>(P, s);
  }
}

bool kmajor(const Operand &o) { return o.ks == 1; }

// `rows` x K bf16 operand for TMA: 16-byte aligned base and lines
bool tma_ok(const Operand &o, int64_t rows, int64_t K) {
  if (!kmajor(o) && o.rs != 1) return false;
  const int64_t ld = kmajor(o) ? o.rs : o.ks, lines = kmajor(o) ? rows : K;
  return (reinterpret_cast<uintptr_t>(o.p) & 15) == 0 && (lines == 1 || ld % 8 == 0);
}

// Map {inner, lines, planes} of an operand in boxes of 64 inner elements x
// `box` lines x 1 plane, 128-byte swizzle
bool map_operand(CUtensorMap *m, const Operand &o, int64_t rows, int64_t K, int box) {
  const bool km = kmajor(o);
  const int64_t inner = km ? K : rows, lines = km ? rows : K;
  const int64_t ld = lines == 1 ? pack_ld(inner) : (km ? o.rs : o.ks);
  const int planes = std::max(1, o.planes);
  return make_map3d(m, o.p, inner, lines, planes, ld, planes == 1 ? ld * lines : o.plane_stride, box);
}

// The pairs of planes of an fp32 product, smallest products first
constexpr uint8_t kPlanePairs[6][2] = {{2, 0}, {0, 2}, {1, 1}, {1, 0}, {0, 1}, {0, 0}};

}  // namespace

bool dense_tc_ok(const DenseGemm &g) {
  if (g.K < 1 || g.M < 1 || g.M > 0x7ffffe00 || g.K > 0x7ffffe00 || g.N > 0x7ffffe00) return false;
  const bool f32 = g.dtype == MOE_F32;
  for (const Operand *o : {&g.b, &g.b3, &g.b2})
    if (o->p && (!tma_ok(*o, g.N, g.K) || o->planes > (f32 ? 3 : 2) || f32 != (o->planes == 3))) return false;
  for (const Operand *o : {&g.a, &g.a2})
    if (o->p && (!tma_ok(*o, g.M, g.K) || f32 != (o->planes == 3))) return false;
  return (!g.a2.p || (kmajor(g.a) == kmajor(g.a2) && kmajor(g.b) == kmajor(g.b2))) &&
         (!g.b3.p || kmajor(g.b) == kmajor(g.b3)) && (g.epi != kDenseGated || kmajor(g.b));
}

size_t dense_tail_bytes() { return (size_t)kMaxPairs * 2 * kSlotFloats * 4; }

cudaError_t launch_dense_tc(const DenseGemm *g, int n, uint32_t *err, float *part, cudaStream_t s) {
  if (n < 1 || n > kMaxProblems) return cudaErrorInvalidValue;
  TcParams P{};
  P.err = err;
  P.part = part;
  P.act = g[0].act;
  P.nprob = n;
  // columns of a tile: 256, or 128 (about 0.8 of the time each) where that
  // spreads a small product over more pairs or pads less
  const bool gated = g[0].epi == kDenseGated;
  auto tiles_of = [&](const DenseGemm &q, int bn) {
    const int w = gated ? bn / 2 : bn;
    return ((q.M + 2 * BM - 1) / (2 * BM)) * ((q.N + w - 1) / w);
  };
  auto tiles_at = [&](int bn) {
    int64_t t = 0;
    for (int p = 0; p < n; ++p) t += tiles_of(g[p], bn);
    return t;
  };
  const double pairs = std::max(1, device_sms() / 2);
  // in steps of 256 columns: full waves, then a plain last wave or its cut form
  auto cost = [&](int bn) {
    double steps = 0;
    for (int p = 0; p < n; ++p)
      steps += (double)tiles_of(g[p], bn) * (double)((g[p].K + kBks * BK - 1) / (kBks * BK)) *
               ((g[p].a2.p ? 2 : 1) * (g[p].dtype == MOE_F32 ? 6 : 1));
    const double tiles = (double)tiles_at(bn), S = steps / tiles, full = std::floor(tiles / pairs);
    const double rest = tiles - full * pairs;
    const double last = rest == 0 ? 0 : std::min(S, rest * S / pairs + kJoinSteps + 2 * std::ceil(pairs / rest));
    return (full * S + last) * (bn == 256 ? 1.0 : 0.8);
  };
  P.bn = cost(128) < cost(256) ? 128 : 256;
  P.bnh = gated ? P.bn / 2 : P.bn;
  if (tiles_at(P.bn) > 0x3fffffff) return cudaErrorInvalidValue;
  auto box_b = [&](const Operand &o) { return kmajor(o) ? P.bn / 2 : BK; };
  // longest contractions last: they are then in the tail, which can be cut
  int order[kMaxProblems] = {0, 1, 2, 3};
  auto depth = [&](int p) { return g[p].K * (g[p].a2.p ? 2 : 1); };
  std::stable_sort(order, order + n, [&](int a, int b) { return depth(a) < depth(b); });
  int64_t end = 0;
  for (int p = 0; p < n; ++p) {
    TcProblem &Q = P.pr[p];
    const DenseGemm &G = g[order[p]];
    bool ok = map_operand(&Q.a[0], G.a, G.M, G.K, kmajor(G.a) ? BM : BK) &&
              map_operand(&Q.b[0], G.b, G.N, G.K, box_b(G.b));
    if (G.a2.p)
      ok = ok && map_operand(&Q.a[1], G.a2, G.M, G.K, kmajor(G.a2) ? BM : BK) &&
           map_operand(&Q.b[1], G.b2, G.N, G.K, box_b(G.b2));
    if (G.b3.p) ok = ok && map_operand(&Q.b[1], G.b3, G.N, G.K, box_b(G.b3));
    if (!ok) return cudaErrorInvalidValue;
    // segments, smallest products first
    auto segments = [&](uint8_t az, uint8_t bz) {
      for (uint8_t i = 0; i < (G.a2.p ? 2 : 1); ++i) Q.seg[Q.segs++] = {i, az, i, bz};
    };
    if (G.dtype == MOE_F32)
      for (const auto &q : kPlanePairs) segments(q[0], q[1]);
    else
      for (int az = std::max(1, G.a.planes) - 1; az >= 0; --az)
        for (int bz = std::max(1, G.b.planes) - 1; bz >= 0; --bz) segments((uint8_t)az, (uint8_t)bz);
    Q.amn = !kmajor(G.a);
    Q.bmn = !kmajor(G.b);
    Q.M = G.M;
    Q.N = G.N;
    Q.KB = (int32_t)((G.K + BK - 1) / BK);
    Q.tiles_m = (int32_t)((G.M + 2 * BM - 1) / (2 * BM));
    Q.tile_end = (int32_t)(end += tiles_of(G, P.bn));
    Q.bias = G.bias;
    Q.bias3 = G.bias3;
    Q.residual = G.residual;
    Q.ld_r = G.ld_r;
    Q.out = G.out;
    Q.ld_o = G.ld_o;
    Q.lo_stride = G.lo_stride;
    Q.pre = G.pre;
    Q.pre3 = G.pre3;
    Q.pre_in = G.pre_in;
    Q.pre3_in = G.pre3_in;
    Q.out2 = G.out2;
    Q.out3 = G.out3;
  }
  return g[0].dtype == MOE_F32 ? launch_as<float>(g[0].epi, P, s) : launch_as<__nv_bfloat16>(g[0].epi, P, s);
}

}  // namespace moe
