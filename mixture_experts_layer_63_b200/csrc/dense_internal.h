// Host-side declarations of the dense operators beside the MoE layer: the
// matrix product with bias, activation and residual in its epilogue, the
// gated feed-forward block, their backward passes, and gradient clipping.
#pragma once

#include "moe_internal.h"

namespace moe {

// A matrix operand of a product: element (row, k) at p + row * rs + k * ks
// (strides in elements).  ks == 1: the contraction index is contiguous
// (K-major); rs == 1: the rows are (MN-major).
// planes: bf16 matrices plane_stride elements apart whose sum is the operand
// (0: p has the product's own dtype).  Three for the tensor cores' copy of an
// fp32 matrix; two (the value rounded, and the rest rounded) for what a bf16
// call of few rows hands from one of its products to the next.
struct Operand {
  const void *p;
  int64_t rs, ks;
  int planes;
  int64_t plane_stride;
};

enum DenseEpilogue : int {
  kDenseStore = 0,      // out = acc
  kDenseLinear = 1,     // z = acc + bias;  out = act(z) + residual;  pre = z
  kDenseGated = 2,      // a = acc + bias, u = acc3 + bias3;  out = act(a) * u;  pre = a, pre3 = u
  kDenseGatedGrad = 3,  // dh = acc, a = pre_in, u = pre3_in:  out = dh u act'(a),
                        //   out2 = dh act(a),  out3 = act(a) u
};

// One product  acc[m, n] = sum_k A(m, k) B(n, k)  (+ a second pair of
// operands a2, b2 contracted over as many k into the same sums) with its
// epilogue.  kDenseGated contracts A with b into acc and with b3 into acc3.
// Every matrix of a product has the type `dtype`.
struct DenseGemm {
  int epi, act, dtype;
  int64_t M, K;
  int32_t N;
  Operand a, b, b3, a2, b2;      // b3.p / a2.p null: absent
  const void *bias, *bias3;      // [N] or null
  const void *residual;          // [M] rows, ld_r apart, or null
  int64_t ld_r;
  void *out;                     // [M] rows, ld_o apart
  int64_t ld_o;
  int64_t lo_stride;             // not 0: out, out2, out3 are two planes this far apart
  void *pre, *pre3;              // [M, N] packed, or null
  const void *pre_in, *pre3_in;  // [M, N] packed
  void *out2, *out3;             // rows ld_o apart
};

inline size_t dense_elem(int dtype) { return dtype == MOE_F32 ? 4 : 2; }

// CUDA-core product (dense_simt.cu): any strides, any sizes
cudaError_t launch_dense_simt(const DenseGemm &g, cudaStream_t s);

// Tensor-core products (dense_tc.cu).  dense_tc_ok: every operand is bf16 (or
// bf16 planes) with base and lines 16-byte aligned.  launch_dense_tc runs up
// to four products with one epilogue in one launch.
bool dense_tc_ok(const DenseGemm &g);
// err: the workspace's control block; part: dense_tail_bytes() of scratch for
// tiles that are cut between CTA pairs.
size_t dense_tail_bytes();
cudaError_t launch_dense_tc(const DenseGemm *g, int n, uint32_t *err, float *part, cudaStream_t s);

// Copies of matrices for the tensor cores (dense_pack.cu): `lines` lines of
// `inner` elements, ld apart, into bf16 planes of round_up(inner, 8) elements a
// line: one plane (bf16, to align the lines) or the three planes of an fp32
// matrix.  Up to kMaxPack matrices in one launch.
constexpr int kMaxPack = 8;
struct PackJob {
  const void *src;
  int64_t lines, inner, ld;
  void *dst;
};
__host__ __device__ inline int64_t pack_ld(int64_t inner) { return (inner + 7) / 8 * 8; }
inline size_t pack_bytes(int dtype, int64_t lines, int64_t inner) {
  return (size_t)(lines * pack_ld(inner)) * 2 * (dtype == MOE_F32 ? 3 : 1);
}
cudaError_t launch_pack(int dtype, const PackJob *jobs, int n, cudaStream_t s);

// Forward products of few rows (dense_few.cu): bf16, one tile of tokens.
// Against 256-row tiles (dense_tc.cu), single calls from cold caches, K = 4096, N =
// 14336: 37 us against 43 at 64 rows, 41 against 45 at 128, 57 against 45 at 192; N
// = 4096: 20 against 31 at 128; the gated block 4096 / 14336 90 against 115 at 64
// rows, 100 - 117 against 117 at 128, 147 against 117 at 192.
constexpr int64_t kFewRows = 128;
bool dense_few_ok(const DenseGemm &g);
cudaError_t launch_dense_few(const DenseGemm &g, uint32_t *err, cudaStream_t s);

// The same on CUDA cores, any strides (dense_rows.cu): fp32, up to this many
// rows (small matrices: twice as many), and bf16 operands that are not aligned
constexpr int64_t kRegisterRows = 16;
bool dense_rows_ok(const DenseGemm &g);
cudaError_t launch_dense_rows(const DenseGemm &g, cudaStream_t s);

// Column sums out[n] = sum_m src[m, n] (fp32, in a fixed order), up to three
// matrices of M rows in one launch.  With z (packed [M, N])
// and dz (lines ld_dz apart): dz = src * act'(z) first, and the sums are dz's;
// out may then be null.
// part: scratch of colsum_scratch(M, widest N, count) bytes.
constexpr int kMaxColSums = 3;
struct ColSum {
  const void *src;
  int64_t ld, src_lo;            // src_lo not 0: src is two planes this far apart
  int N;
  const void *z;
  void *dz;
  int64_t ld_dz, lo_stride;      // lo_stride not 0: dz is two planes this far apart
  void *out;
};
size_t colsum_scratch(int64_t M, int N, int count);
cudaError_t launch_colsums(int act, int dtype, int64_t M, const ColSum *q, int count, float *part,
                           cudaStream_t s);

// --- gradient clipping (clip.cu) ----------------------------------------------
size_t clip_scratch(int32_t count);
// max_norm < 0: the norm alone
cudaError_t launch_clip(const moe_grad *g, int32_t count, float max_norm, float *norm, double *part,
                        cudaStream_t s);

}  // namespace moe
