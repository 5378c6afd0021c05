// C ABI of the dense operators (declared in include/moe.h): argument
// validation, workspace layout and the launch sequence of each entry point.
#include <algorithm>
#include <cmath>
#include <vector>

#include <nvtx3/nvToolsExt.h>

#include "dense_internal.h"

namespace moe {
namespace {

struct DenseRange {
  explicit DenseRange(const char *name) { nvtxRangePushA(name); }
  ~DenseRange() { nvtxRangePop(); }
  DenseRange(const DenseRange &) = delete;
  DenseRange &operator=(const DenseRange &) = delete;
};

constexpr int64_t kMaxRows = 0x7fffffff;
size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

// Workspace: pieces of the caller's buffer, one after another.
struct Taker {
  size_t o = align256(kCtrlBytes);
  size_t take(size_t bytes) {
    const size_t at = o;
    o = align256(o + bytes);
    return at;
  }
};

// ---- memory spans -------------------------------------------------------------
// `rows` rows of `width` elements, `ld` apart
struct Span {
  const void *p;
  int64_t rows, width, ld;
  int es;
  uintptr_t begin() const { return reinterpret_cast<uintptr_t>(p); }
  uintptr_t end() const { return begin() + (uintptr_t)((rows - 1) * ld + width) * es; }
  bool none() const { return !p || rows == 0; }
};

bool overlap(const Span &a, const Span &b) {
  if (a.none() || b.none() || a.end() <= b.begin() || b.end() <= a.begin()) return false;
  // column slices of one buffer: the same row stride, no common column
  if (a.ld == b.ld && a.es == b.es && a.rows > 1 && b.rows > 1) {
    const Span &lo = a.begin() <= b.begin() ? a : b, &hi = a.begin() <= b.begin() ? b : a;
    const uintptr_t gap = hi.begin() - lo.begin(), row = (uintptr_t)a.ld * a.es;
    const uintptr_t col = gap % row;
    if (col >= (uintptr_t)lo.width * a.es && col + (uintptr_t)hi.width * a.es <= row) return false;
  }
  return true;
}

bool aligned_to(const void *p, int es) { return !p || reinterpret_cast<uintptr_t>(p) % es == 0; }

// outputs against inputs and one another; every pointer aligned to its element
moe_status check_spans(const std::initializer_list<Span> &in, const std::initializer_list<Span> &out) {
  for (const Span &s : in)
    if (!aligned_to(s.p, s.es)) return MOE_ERR_INVALID_ARG;
  for (const Span *o = out.begin(); o != out.end(); ++o) {
    if (!aligned_to(o->p, o->es)) return MOE_ERR_INVALID_ARG;
    for (const Span &s : in)
      if (overlap(*o, s)) return MOE_ERR_INVALID_ARG;
    for (const Span *q = out.begin(); q != o; ++q)
      if (overlap(*o, *q)) return MOE_ERR_INVALID_ARG;
  }
  return MOE_OK;
}

moe_status check_dense_ws(const void *ws, size_t ws_bytes, size_t need) {
  if (!ws || reinterpret_cast<uintptr_t>(ws) % 256 != 0) return MOE_ERR_INVALID_ARG;
  return ws_bytes < need ? MOE_ERR_WORKSPACE : MOE_OK;
}

moe_status dense_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

bool bad_ld(int64_t ld, int64_t width) { return ld != 0 && (ld < width || ld > kMaxRows); }

// beyond any memory, and the byte counts here: 2^48 elements
bool too_large(int64_t rows, int64_t ld) { return rows > 0 && ld > ((int64_t)1 << 48) / rows; }

moe_status validate_act(int32_t act, int32_t dtype) {
  if (act < MOE_DENSE_IDENTITY || act > MOE_DENSE_GELU_TANH) return MOE_ERR_INVALID_ARG;
  return dtype == MOE_F32 || dtype == MOE_BF16 ? MOE_OK : MOE_ERR_INVALID_ARG;
}

// ---- linear ---------------------------------------------------------------------
moe_status validate_linear(const moe_linear_config *in, moe_linear_config *c) {
  if (!in) return MOE_ERR_INVALID_ARG;
  *c = *in;
  if (c->M < 0 || c->K < 1 || c->N < 1 || c->reserved != 0) return MOE_ERR_INVALID_ARG;
  const moe_status st = validate_act(c->act, c->dtype);
  if (st != MOE_OK) return st;
  if (bad_ld(c->ld_x, c->K) || bad_ld(c->ld_w, c->K) || bad_ld(c->ld_r, c->N) || bad_ld(c->ld_y, c->N))
    return MOE_ERR_INVALID_ARG;
  if (c->ld_x == 0) c->ld_x = c->K;
  if (c->ld_w == 0) c->ld_w = c->K;
  if (c->ld_r == 0) c->ld_r = c->N;
  if (c->ld_y == 0) c->ld_y = c->N;
  if (c->M > kMaxRows || too_large(c->M, std::max({c->ld_x, c->ld_r, c->ld_y})) || too_large(c->N, c->ld_w))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Do the tensor cores need a copy of a matrix with lines ld elements apart?
// fp32: its planes; bf16: where a line is not 16-byte aligned.
bool needs_copy(int dtype, int64_t lines, int64_t ld, const void *p = nullptr) {
  return dtype == MOE_F32 || (lines > 1 && ld % 8 != 0) || reinterpret_cast<uintptr_t>(p) % 16 != 0;
}
size_t copy_room(int dtype, int64_t lines, int64_t inner) { return align256(pack_bytes(dtype, lines, inner)); }
// Room for it, before the matrix's address is known
size_t pack_room(int dtype, int64_t lines, int64_t inner, int64_t ld) {
  return needs_copy(dtype, lines, ld) ? copy_room(dtype, lines, inner) : 0;
}

// bf16 calls of few rows hand dz, h, dA and dU from one product to the next in
// two planes (the value rounded to bf16, and the rest rounded): 16 significant
// bits instead of 8, so that their results carry one rounding.  (Of more rows
// the errors average out in the sums.)  Forward the time is the weights'
// stream, and the second plane is free: up to 16 rows.  Backward it doubles
// products that are short beside their launches (one row of a 2048 / 5632
// block: 111 us against 83): up to 4 rows.
int planes_of(int dtype, int64_t rows, bool backward) {
  return dtype == MOE_BF16 && rows <= (backward ? 4 : 16) ? 2 : 1;
}

// Room for cut tiles (dense_tc.cu): forward calls of few rows never get there
size_t tail_room(int dtype, int64_t rows, bool backward) {
  return !backward && rows <= (dtype == MOE_F32 ? kRegisterRows : kFewRows) ? 0 : dense_tail_bytes();
}

struct LinearLayout {
  size_t dz, part, tail, pack, total;
};

LinearLayout linear_layout(const moe_linear_config &c, bool backward) {
  LinearLayout L{};
  Taker t;
  // x and dy always have room for a copy: a column slice may start anywhere
  size_t room = copy_room(c.dtype, c.M, c.K) + pack_room(c.dtype, c.N, c.K, c.ld_w);
  if (backward) {
    const bool act = c.act != MOE_DENSE_IDENTITY;
    L.dz = t.take(act ? (size_t)c.M * pack_ld(c.N) * dense_elem(c.dtype) * planes_of(c.dtype, c.M, true) : 0);
    L.part = t.take(colsum_scratch(c.M, c.N, 1));
    room += act ? pack_room(c.dtype, c.M, c.N, pack_ld(c.N)) : copy_room(c.dtype, c.M, c.N);
  }
  L.tail = t.take(tail_room(c.dtype, c.M, backward));
  L.pack = t.take(room);
  L.total = t.o;
  return L;
}

// The products of one call: each group of up to four with one epilogue runs
// on the kernel that suits it.  Copies made for the tensor cores stay for the
// later groups of the call.
class Products {
 public:
  Products(int dtype, void *ws, size_t tail, size_t pack, size_t end, cudaStream_t s)
      : dtype_(dtype), base_(static_cast<char *>(ws)), tail_(tail), first_(pack), at_(pack), end_(end), s_(s) {}

  cudaError_t run(DenseGemm *g, int n) {
    uint32_t *err = reinterpret_cast<uint32_t *>(base_);
    if (n == 1 && dense_few_ok(g[0])) return launch_dense_few(g[0], err, s_);
    if (n == 1 && dense_rows_ok(g[0]) && (dtype_ == MOE_F32 || !dense_tc_ok(g[0])))
      return launch_dense_rows(g[0], s_);
    double macs = 0;
    int64_t depth = 0;
    for (int i = 0; i < n; ++i) {
      macs += (double)g[i].M * g[i].N * g[i].K * (g[i].a2.p || g[i].b3.p ? 2 : 1);
      depth = std::max(depth, g[i].K);
    }
    if (macs >= kTcMacs || depth > kSimtDepth || dtype_ == MOE_BF16) {
      DenseGemm q[4];
      const size_t at = at_;
      bool ok = true;
      for (int i = 0; i < n && ok; ++i) {
        q[i] = g[i];
        ok = prepare(&q[i].a, g[i].M, g[i].K) && prepare(&q[i].b, g[i].N, g[i].K) &&
             prepare(&q[i].b3, g[i].N, g[i].K) && prepare(&q[i].a2, g[i].M, g[i].K) &&
             prepare(&q[i].b2, g[i].N, g[i].K) && dense_tc_ok(q[i]);
      }
      if (ok) {
        cudaError_t e = cudaSuccess;
        if (launched_ < jobs_) e = launch_pack(dtype_, job_ + launched_, jobs_ - launched_, s_);
        launched_ = jobs_;
        if (e != cudaSuccess) return e;
        if (n == 1 && dense_few_ok(q[0])) return launch_dense_few(q[0], err, s_);
        return launch_dense_tc(q, n, err, tail_ < first_ ? reinterpret_cast<float *>(base_ + tail_) : nullptr, s_);
      }
      jobs_ = launched_;
      at_ = at;
    }
    cudaError_t e = cudaSuccess;
    for (int i = 0; i < n && e == cudaSuccess; ++i) e = launch_dense_simt(g[i], s_);
    return e;
  }
  cudaError_t run(DenseGemm &g) { return run(&g, 1); }

 private:
  // fewer multiply-adds than this stay on the CUDA cores in fp32: the splits
  // and the tensor-core launch cost more than they save
  static constexpr double kTcMacs = 1 << 22;
  // ... unless a contraction is longer than this, which one CUDA-core block
  // would run through alone
  static constexpr int64_t kSimtDepth = 512;
  static constexpr int kMaxJobs = kMaxPack;

  // `o`, rows x K, replaced by its copy where the tensor cores need one
  bool prepare(Operand *o, int64_t rows, int64_t K) {
    if (!o->p || rows == 0 || K == 0) return true;
    const bool km = o->ks == 1;
    const int64_t lines = km ? rows : K, inner = km ? K : rows, ld = km ? o->rs : o->ks;
    if (!needs_copy(dtype_, lines, ld, o->p)) return true;
    int j = 0;
    while (j < jobs_ && !(job_[j].src == o->p && job_[j].lines == lines && job_[j].inner == inner &&
                          job_[j].ld == ld))
      ++j;
    if (j == jobs_) {
      const size_t need = copy_room(dtype_, lines, inner);
      if (jobs_ == kMaxJobs || at_ + need > end_) return false;
      job_[jobs_++] = {o->p, lines, inner, ld, base_ + at_};
      at_ += need;
    }
    o->p = job_[j].dst;
    (km ? o->rs : o->ks) = pack_ld(inner);
    if (dtype_ == MOE_F32) {
      o->planes = 3;
      o->plane_stride = lines * pack_ld(inner);
    }
    return true;
  }

  int dtype_;
  char *base_;
  size_t tail_, first_, at_, end_;        // cut tiles; copies: their first, next and last byte
  cudaStream_t s_;
  PackJob job_[kMaxJobs];
  int jobs_ = 0, launched_ = 0;
};

Operand transposed(Operand o) {
  std::swap(o.rs, o.ks);
  return o;
}

// out [M, N] = sum over k < K of a(m, k) b(n, k)
DenseGemm product(int dtype, int64_t M, int64_t K, int32_t N, const Operand &a, const Operand &b, void *out,
                  int64_t ld_o) {
  DenseGemm g{};
  g.epi = kDenseStore;
  g.dtype = dtype;
  g.M = M;
  g.K = K;
  g.N = N;
  g.a = a;
  g.b = b;
  g.out = out;
  g.ld_o = ld_o;
  return g;
}

// ---- gated block ------------------------------------------------------------------
moe_status validate_gated(const moe_gated_ffn_config *in, moe_gated_ffn_config *c) {
  if (!in) return MOE_ERR_INVALID_ARG;
  *c = *in;
  if (c->T < 0 || c->d_model < 1 || c->d_ff < 1 || c->reserved != 0) return MOE_ERR_INVALID_ARG;
  const moe_status st = validate_act(c->act, c->dtype);
  if (st != MOE_OK) return st;
  if (bad_ld(c->ld_x, c->d_model) || bad_ld(c->ld_r, c->d_model) || bad_ld(c->ld_y, c->d_model))
    return MOE_ERR_INVALID_ARG;
  if (c->ld_x == 0) c->ld_x = c->d_model;
  if (c->ld_r == 0) c->ld_r = c->d_model;
  if (c->ld_y == 0) c->ld_y = c->d_model;
  if (c->T > kMaxRows || too_large(c->T, std::max<int64_t>({c->ld_x, c->ld_r, c->ld_y, c->d_ff})) ||
      too_large(c->d_ff, c->d_model))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

struct GatedLayout {
  size_t h, da, du, part, tail, pack, total;
};

GatedLayout gated_layout(const moe_gated_ffn_config &c, bool backward) {
  GatedLayout L{};
  Taker t;
  // h, dA and dU have aligned lines of their own
  const int64_t T = c.T, d = c.d_model, f = c.d_ff, ldh = pack_ld(f);
  const size_t tf = (size_t)T * ldh * dense_elem(c.dtype) * planes_of(c.dtype, T, backward);
  auto room = [&](int64_t lines, int64_t inner, int64_t ld) { return pack_room(c.dtype, lines, inner, ld); };
  size_t pack = copy_room(c.dtype, T, d) + 2 * room(f, d, d) + room(d, f, f) + room(T, f, ldh);
  L.h = t.take(tf);
  if (backward) {
    L.da = t.take(tf);
    L.du = t.take(tf);
    // (the sums of a subset may be cut into more parts than those of all)
    L.part = t.take(std::max(colsum_scratch(T, c.d_ff, 3), colsum_scratch(T, c.d_model, 3)));
    pack += 2 * room(T, f, ldh) + copy_room(c.dtype, T, d);
  }
  L.tail = t.take(tail_room(c.dtype, T, backward));
  L.pack = t.take(pack);
  L.total = t.o;
  return L;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_query_linear_size(const moe_linear_config *cfg, int32_t backward, size_t *bytes) {
  moe_linear_config c;
  if (!bytes || (backward != 0 && backward != 1)) return MOE_ERR_INVALID_ARG;
  const moe_status st = validate_linear(cfg, &c);
  if (st == MOE_OK) *bytes = linear_layout(c, backward != 0).total;
  return st;
}

moe_status moe_linear(const moe_linear_config *cfg, const void *x, const void *w, const void *bias,
                      const void *residual, void *y, void *z, void *ws, size_t ws_bytes,
                      moe_stream_t stream) {
  DenseRange range("moe_linear");
  moe_linear_config c;
  moe_status st = validate_linear(cfg, &c);
  if (st != MOE_OK) return st;
  const LinearLayout L = linear_layout(c, false);
  if ((st = check_dense_ws(ws, ws_bytes, L.total)) != MOE_OK) return st;
  if (c.M == 0) return MOE_OK;
  if (!x || !w || !y) return MOE_ERR_INVALID_ARG;
  const int es = (int)dense_elem(c.dtype);
  const Span sx{x, c.M, c.K, c.ld_x, es}, sw{w, c.N, c.K, c.ld_w, es}, sb{bias, 1, c.N, c.N, es},
      sr{residual, c.M, c.N, c.ld_r, es}, sy{y, c.M, c.N, c.ld_y, es}, sz{z, c.M, c.N, c.N, es};
  const bool in_place = residual == y && c.ld_r == c.ld_y;
  if ((st = check_spans({sx, sw, sb, in_place ? Span{} : sr}, {sy, sz})) != MOE_OK) return st;
  DenseGemm g{};
  g.epi = kDenseLinear;
  g.act = c.act;
  g.dtype = c.dtype;
  g.M = c.M;
  g.N = c.N;
  g.K = c.K;
  g.a = {x, c.ld_x, 1};
  g.b = {w, c.ld_w, 1};
  g.bias = bias;
  g.residual = residual;
  g.ld_r = c.ld_r;
  g.out = y;
  g.ld_o = c.ld_y;
  g.pre = z;
  Products run(c.dtype, ws, L.tail, L.pack, L.total, reinterpret_cast<cudaStream_t>(stream));
  return dense_status(run.run(g));
}

moe_status moe_linear_backward(const moe_linear_config *cfg, const void *x, const void *w, const void *z,
                               const void *dy, void *dx, void *dw, void *dbias, void *ws, size_t ws_bytes,
                               moe_stream_t stream) {
  DenseRange range("moe_linear_backward");
  moe_linear_config c;
  moe_status st = validate_linear(cfg, &c);
  if (st != MOE_OK) return st;
  const LinearLayout L = linear_layout(c, true);
  if ((st = check_dense_ws(ws, ws_bytes, L.total)) != MOE_OK) return st;
  const bool act = c.act != MOE_DENSE_IDENTITY;
  if (!dx && !dw && !dbias) return MOE_ERR_INVALID_ARG;
  if (c.M > 0 && (!dy || (dw && !x) || (dx && !w) || (act && !z))) return MOE_ERR_INVALID_ARG;
  const int es = (int)dense_elem(c.dtype);
  const Span sx{x, c.M, c.K, c.ld_x, es}, sw{w, c.N, c.K, c.ld_w, es},
      sz{act ? z : nullptr, c.M, c.N, c.N, es}, sdy{dy, c.M, c.N, c.ld_y, es};
  if ((st = check_spans({sx, sw, sz, sdy}, {Span{dx, c.M, c.K, c.ld_x, es}, Span{dw, c.N, c.K, c.K, es},
                                            Span{dbias, 1, c.N, c.N, es}})) != MOE_OK)
    return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  char *base = static_cast<char *>(ws);
  cudaError_t e = cudaSuccess;
  Operand dz{dy, c.ld_y, 1};
  if (act || dbias) {
    // dz and its column sums in one pass over dy and z
    const int64_t ldz = pack_ld(c.N), lo = planes_of(c.dtype, c.M, true) == 2 ? c.M * ldz : 0;
    const ColSum q{dy, c.ld_y, 0, c.N, act ? z : nullptr, act ? base + L.dz : nullptr, ldz, lo, dbias};
    e = launch_colsums(c.act, c.dtype, c.M, &q, 1, reinterpret_cast<float *>(base + L.part), s);
    if (act) dz = {base + L.dz, ldz, 1, lo ? 2 : 0, lo};
  }
  DenseGemm g[2] = {};
  int n = 0;
  if (dx && c.M > 0) g[n++] = product(c.dtype, c.M, c.N, c.K, dz, {w, 1, c.ld_w}, dx, c.ld_x);
  if (dw) g[n++] = product(c.dtype, c.N, c.M, c.K, transposed(dz), {x, 1, c.ld_x}, dw, c.K);
  Products run(c.dtype, ws, L.tail, L.pack, L.total, s);
  if (e == cudaSuccess && n > 0) e = run.run(g, n);
  return dense_status(e);
}

moe_status moe_query_gated_ffn_size(const moe_gated_ffn_config *cfg, int32_t backward, size_t *bytes) {
  moe_gated_ffn_config c;
  if (!bytes || (backward != 0 && backward != 1)) return MOE_ERR_INVALID_ARG;
  const moe_status st = validate_gated(cfg, &c);
  if (st == MOE_OK) *bytes = gated_layout(c, backward != 0).total;
  return st;
}

moe_status moe_gated_ffn(const moe_gated_ffn_config *cfg, const void *x, const void *w1, const void *b1,
                         const void *w3, const void *b3, const void *w2, const void *b2,
                         const void *residual, void *y, void *a, void *u, void *ws, size_t ws_bytes,
                         moe_stream_t stream) {
  DenseRange range("moe_gated_ffn");
  moe_gated_ffn_config c;
  moe_status st = validate_gated(cfg, &c);
  if (st != MOE_OK) return st;
  const GatedLayout L = gated_layout(c, false);
  if ((st = check_dense_ws(ws, ws_bytes, L.total)) != MOE_OK) return st;
  if (c.T == 0) return MOE_OK;
  if (!x || !w1 || !w3 || !w2 || !y || !b1 != !b3 || !a != !u) return MOE_ERR_INVALID_ARG;
  const int es = (int)dense_elem(c.dtype);
  const int64_t T = c.T, d = c.d_model, f = c.d_ff, ldh = pack_ld(f);
  const bool in_place = residual == y && c.ld_r == c.ld_y;
  const Span sr{residual, T, d, c.ld_r, es};
  if ((st = check_spans({Span{x, T, d, c.ld_x, es}, Span{w1, f, d, d, es}, Span{w3, f, d, d, es},
                         Span{w2, d, f, f, es}, Span{b1, 1, f, f, es}, Span{b3, 1, f, f, es},
                         Span{b2, 1, d, d, es}, in_place ? Span{} : sr},
                        {Span{y, T, d, c.ld_y, es}, Span{a, T, f, f, es}, Span{u, T, f, f, es}})) != MOE_OK)
    return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  char *base = static_cast<char *>(ws);
  DenseGemm g{};
  g.epi = kDenseGated;
  g.act = c.act;
  g.dtype = c.dtype;
  g.M = T;
  g.N = c.d_ff;
  g.K = d;
  g.a = {x, c.ld_x, 1};
  g.b = {w1, d, 1};
  g.b3 = {w3, d, 1};
  g.bias = b1;
  g.bias3 = b3;
  const int64_t lo = planes_of(c.dtype, T, false) == 2 ? T * ldh : 0;
  g.out = base + L.h;
  g.ld_o = ldh;
  g.lo_stride = lo;
  g.pre = a;
  g.pre3 = u;
  Products run(c.dtype, ws, L.tail, L.pack, L.total, s);
  cudaError_t e = run.run(g);
  if (e != cudaSuccess) return MOE_ERR_CUDA;
  DenseGemm q{};
  q.epi = kDenseLinear;
  q.act = MOE_DENSE_IDENTITY;
  q.dtype = c.dtype;
  q.M = T;
  q.N = c.d_model;
  q.K = f;
  q.a = {base + L.h, ldh, 1, lo ? 2 : 0, lo};
  q.b = {w2, f, 1};
  q.bias = b2;
  q.residual = residual;
  q.ld_r = c.ld_r;
  q.out = y;
  q.ld_o = c.ld_y;
  return dense_status(run.run(q));
}

moe_status moe_gated_ffn_backward(const moe_gated_ffn_config *cfg, const void *x, const void *w1,
                                  const void *w3, const void *w2, const void *a, const void *u,
                                  const void *dy, void *dx, void *dw1, void *db1, void *dw3, void *db3,
                                  void *dw2, void *db2, void *ws, size_t ws_bytes, moe_stream_t stream) {
  DenseRange range("moe_gated_ffn_backward");
  moe_gated_ffn_config c;
  moe_status st = validate_gated(cfg, &c);
  if (st != MOE_OK) return st;
  const GatedLayout L = gated_layout(c, true);
  if ((st = check_dense_ws(ws, ws_bytes, L.total)) != MOE_OK) return st;
  if (!dw1 != !dw3 || !db1 != !db3 || (!dx && !dw1 && !db1 && !dw2 && !db2)) return MOE_ERR_INVALID_ARG;
  const bool hidden = dx || dw1 || db1 || dw2;       // dA, dU or h are needed
  if (c.T > 0 && (!dy || (hidden && (!w2 || !a || !u)) || (dw1 && !x) || (dx && (!w1 || !w3))))
    return MOE_ERR_INVALID_ARG;
  const int es = (int)dense_elem(c.dtype);
  const int64_t T = c.T, d = c.d_model, f = c.d_ff, ldh = pack_ld(f);
  if ((st = check_spans({Span{x, T, d, c.ld_x, es}, Span{w1, f, d, d, es}, Span{w3, f, d, d, es},
                         Span{w2, d, f, f, es}, Span{a, T, f, f, es}, Span{u, T, f, f, es},
                         Span{dy, T, d, c.ld_y, es}},
                        {Span{dx, T, d, c.ld_x, es}, Span{dw1, f, d, d, es}, Span{db1, 1, f, f, es},
                         Span{dw3, f, d, d, es}, Span{db3, 1, f, f, es}, Span{dw2, d, f, f, es},
                         Span{db2, 1, d, d, es}})) != MOE_OK)
    return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  char *base = static_cast<char *>(ws);
  char *h = base + L.h, *da = base + L.da, *du = base + L.du;
  float *part = reinterpret_cast<float *>(base + L.part);
  cudaError_t e = cudaSuccess;
  Products run(c.dtype, ws, L.tail, L.pack, L.total, s);
  const int64_t lo = planes_of(c.dtype, T, true) == 2 ? T * ldh : 0;
  auto hidden_rows = [&](const void *p) { return Operand{p, ldh, 1, lo ? 2 : 0, lo}; };
  if (hidden && T > 0) {
    DenseGemm g{};
    g.epi = kDenseGatedGrad;
    g.act = c.act;
    g.dtype = c.dtype;
    g.M = T;
    g.N = c.d_ff;
    g.K = d;
    g.a = {dy, c.ld_y, 1};
    g.b = {w2, 1, f};                       // W2 [d, f] contracted over its rows
    g.pre_in = a;
    g.pre3_in = u;
    g.out = da;
    g.ld_o = ldh;
    g.lo_stride = lo;
    g.out2 = du;
    g.out3 = h;
    e = run.run(g);
  }
  // dx and the weight gradients (each contracts two matrices over the rows) in one launch
  DenseGemm g[4] = {};
  int n = 0;
  if (dx && T > 0) {
    g[n] = product(c.dtype, T, f, c.d_model, hidden_rows(da), {w1, 1, d}, dx, c.ld_x);
    g[n].a2 = hidden_rows(du);
    g[n++].b2 = {w3, 1, d};
  }
  if (dw1) {
    g[n++] = product(c.dtype, f, T, c.d_model, transposed(hidden_rows(da)), {x, 1, c.ld_x}, dw1, d);
    g[n++] = product(c.dtype, f, T, c.d_model, transposed(hidden_rows(du)), {x, 1, c.ld_x}, dw3, d);
  }
  if (dw2) g[n++] = product(c.dtype, d, T, c.d_ff, {dy, 1, c.ld_y}, transposed(hidden_rows(h)), dw2, f);
  if (e == cudaSuccess && n > 0) e = run.run(g, n);
  ColSum bq[3];
  int nb = 0;
  if (db1) bq[nb++] = {da, ldh, lo, c.d_ff, nullptr, nullptr, 0, 0, db1};
  if (db3) bq[nb++] = {du, ldh, lo, c.d_ff, nullptr, nullptr, 0, 0, db3};
  if (db2) bq[nb++] = {dy, c.ld_y, 0, c.d_model, nullptr, nullptr, 0, 0, db2};
  if (e == cudaSuccess && nb > 0) e = launch_colsums(0, c.dtype, T, bq, nb, part, s);
  return dense_status(e);
}

static moe_status validate_grads(const moe_grad *g, int32_t count, bool clip) {
  if (count < 0 || (count > 0 && !g)) return MOE_ERR_INVALID_ARG;
  // beyond any memory, the byte counts here and the chunk counts of a launch
  // (at least 2^16 elements each there): 2^46 elements in all
  constexpr int64_t kMost = (int64_t)1 << 46;
  int64_t total = 0;
  bool large = false;
  for (int32_t i = 0; i < count; ++i) {
    if (g[i].n < 0 || g[i].reserved != 0 || (g[i].dtype != MOE_F32 && g[i].dtype != MOE_BF16))
      return MOE_ERR_INVALID_ARG;
    const int es = (int)dense_elem(g[i].dtype);
    if (g[i].n > 0 && (!g[i].src || !aligned_to(g[i].src, es) ||
                       (clip && (!g[i].dst || !aligned_to(g[i].dst, es)))))
      return MOE_ERR_INVALID_ARG;
    large = large || g[i].n > kMost - total;
    if (!large) total += g[i].n;
  }
  return large ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

// In address order, what is written (dst and the norm) may not reach into the next piece.
static bool grads_overlap(const moe_grad *g, int32_t count, const float *norm) {
  struct Part {
    uintptr_t b, e;
    bool write;
  };
  std::vector<Part> v;
  v.reserve(2 * (size_t)count + 1);
  const uintptr_t nb = reinterpret_cast<uintptr_t>(norm);
  if (norm) v.push_back({nb, nb + 4, true});
  for (int32_t i = 0; i < count; ++i) {
    if (g[i].n == 0) continue;
    const uintptr_t n = (uintptr_t)g[i].n * dense_elem(g[i].dtype);
    const uintptr_t s = reinterpret_cast<uintptr_t>(g[i].src), d = reinterpret_cast<uintptr_t>(g[i].dst);
    v.push_back({d, d + n, true});
    if (s != d) v.push_back({s, s + n, false});
  }
  std::sort(v.begin(), v.end(), [](const Part &a, const Part &b) { return a.b < b.b; });
  uintptr_t end_any = 0, end_write = 0;
  for (const Part &p : v) {
    if (p.b < end_write || (p.write && p.b < end_any)) return true;
    end_any = std::max(end_any, p.e);
    if (p.write) end_write = std::max(end_write, p.e);
  }
  return false;
}

moe_status moe_query_clip_size(int32_t count, size_t *bytes) {
  if (!bytes || count < 0) return MOE_ERR_INVALID_ARG;
  Taker t;
  t.take(clip_scratch(count));
  *bytes = t.o;
  return MOE_OK;
}

static moe_status run_clip(const moe_grad *g, int32_t count, float max_norm, float *norm, void *ws,
                           size_t ws_bytes, moe_stream_t stream) {
  Taker t;
  const size_t at = t.take(clip_scratch(count));
  const moe_status st = check_dense_ws(ws, ws_bytes, t.o);
  if (st != MOE_OK) return st;
  return dense_status(launch_clip(g, count, max_norm, norm,
                                  reinterpret_cast<double *>(static_cast<char *>(ws) + at),
                                  reinterpret_cast<cudaStream_t>(stream)));
}

moe_status moe_grad_norm(const moe_grad *grads, int32_t count, float *norm, void *ws, size_t ws_bytes,
                         moe_stream_t stream) {
  DenseRange range("moe_grad_norm");
  const moe_status st = validate_grads(grads, count, false);
  if (st != MOE_OK) return st;
  if (!norm || !aligned_to(norm, 4)) return MOE_ERR_INVALID_ARG;
  return run_clip(grads, count, -1.0f, norm, ws, ws_bytes, stream);
}

moe_status moe_clip_grads(const moe_grad *grads, int32_t count, float max_norm, float *norm, void *ws,
                          size_t ws_bytes, moe_stream_t stream) {
  DenseRange range("moe_clip_grads");
  const moe_status st = validate_grads(grads, count, true);
  if (st != MOE_OK) return st;
  if (!(max_norm > 0.0f) || !aligned_to(norm, 4)) return MOE_ERR_INVALID_ARG;
  try {                                  // (the sort's scratch is host memory)
    if (grads_overlap(grads, count, norm)) return MOE_ERR_INVALID_ARG;
  } catch (...) {
    return MOE_ERR_UNSUPPORTED;
  }
  return run_clip(grads, count, max_norm, norm, ws, ws_bytes, stream);
}

}  // extern "C"
