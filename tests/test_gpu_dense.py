"""The dense operators (linear with bias, activation and residual; the gated
feed-forward block; their gradients) against a plain evaluation in 64 bits.

Tolerances are bounds, element by element, evaluated in 64 bits beside the
reference.  With u = half a step of the layer's type (2^-8 bf16, 2^-24 fp32):
  * a product of K terms carries at most c_K sum_k |A||B|, c_K = (K + 32) 2^-23
    (fp32 accumulation: at most 2^-23 of the running sum an addition, whatever
    the order; the bias and residual additions are in the 32);
  * an activation's error is its slope (at most 1.13) times its argument's,
    plus FN max(1, |value|) for the exponential, erf and division (bf16: the fast
    forms), whose arguments stay below 16;
  * a matrix that a second product reads carries u times its magnitude (bf16
    calls of at most 16 rows, backward 4: 2^-17, two planes of 8 bits), and its error
    passes through |other operand|;
  * the output is rounded once: u |y|.
relu' jumps at 0, so backward passes are given pre-activations exactly as
the kernels read them (they are inputs).
"""
import math

import pytest
import torch

from mixture_experts_layer_63_b200 import api

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U = {BF16: 2.0 ** -8, F32: 2.0 ** -24}
SLOPE, FN = 1.13, {BF16: 2.0 ** -18, F32: 2.0 ** -20}


def um(dtype, rows, most=4):
    """Rounding of what one product of a call hands to the next."""
    return 2.0 ** -17 if dtype == BF16 and rows <= most else U[dtype]


def ck(K):
    return (K + 32) * 2.0 ** -23


def act64(z, name):
    import torch.nn.functional as F
    return {"identity": lambda v: v, "relu": F.relu, "silu": F.silu, "gelu": F.gelu,
            "gelu_tanh": lambda v: F.gelu(v, approximate="tanh")}[name](z)


def act64_grad(z, name):
    v = z.detach().clone().requires_grad_(True)
    g, = torch.autograd.grad(act64(v, name).sum(), v) if name != "identity" else (torch.ones_like(v),)
    return g


def rnd(gen, *shape, dtype, std=1.0, pad=0, off=0):
    """Rows of a buffer `pad` columns wider, starting at its column `off`."""
    t = (torch.randn(*shape[:-1], shape[-1] + pad, generator=gen, device="cuda") * std).to(dtype)
    return t[..., off:off + shape[-1]]


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def near(got, ref, bound, what):
    assert got.shape == ref.shape
    assert torch.isfinite(got).all(), what
    over = ((got.double() - ref).abs() / (bound + 1e-300)).max().item() if ref.numel() else 0.0
    assert over <= 1.0, f"{what}: {over:.3f} times the bound"


def d(t):
    return None if t is None else t.double()


# ------------------------------------ linear -----------------------------------

def linear_case(M, K, N, act, dtype, bias, res, save, pad=0, off=0, inplace=False, seed=0):
    g = gen(seed)
    x, w = rnd(g, M, K, dtype=dtype, pad=pad, off=off), rnd(g, N, K, dtype=dtype, std=K ** -0.5, pad=pad, off=off)
    b = rnd(g, N, dtype=dtype) if bias else None
    r = rnd(g, M, N, dtype=dtype, pad=pad, off=off) if res else None
    r0 = None if r is None else r.clone()
    wide = torch.full((M, N + pad), 7.0, dtype=dtype, device="cuda")
    y = r if inplace else wide[:, off:off + N]
    z = torch.empty(M, N, dtype=dtype, device="cuda") if save else None
    cfg = api.linear_config(M, K, N, act, dtype, K + pad, K + pad, N + pad, N + pad)
    ws = api.new_linear_workspace(cfg)
    api.moe_linear(cfg, x, w, b, r, y, z, ws)
    api.moe_check_device_errors(ws)
    xd, wd = x.double(), w.double()
    zr = xd @ wd.T
    ez = ck(K) * (xd.abs() @ wd.abs().T)
    if bias:
        zr = zr + b.double()
        ez = ez + ck(0) * b.double().abs()
    yr = act64(zr, act)
    ey = SLOPE * ez + FN[dtype] * yr.abs().clamp_min(1) * (act != "identity" and act != "relu")
    if res:
        yr = yr + r0.double()
        ey = ey + 2.0 ** -23 * yr.abs()
    u = U[dtype]
    near(y, yr, ey + u * (yr.abs() + ey), "y")
    if save:
        near(z, zr, ez + u * (zr.abs() + ez), "z")
    if pad and not inplace:                    # the columns beside y are not touched
        assert (wide[:, :off] == 7).all() and (wide[:, off + N:] == 7).all()


SHAPES = [(1, 1, 1), (1, 64, 128), (1, 14336, 130), (2, 200, 72), (3, 129, 65), (5, 4096, 256), (16, 256, 512),
          (17, 72, 1000), (33, 512, 24), (64, 1000, 264), (127, 88, 136), (128, 128, 128), (129, 1024, 257),
          (255, 31, 7), (256, 64, 128), (300, 320, 192), (513, 2048, 130), (1000, 777, 333), (2100, 64, 72)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_linear(M, K, N, dtype):
    acts = list(api.DENSE_ACTS)
    i = (M + K + N) % 5
    linear_case(M, K, N, acts[i], dtype, bias=True, res=True, save=True, seed=M + K)
    linear_case(M, K, N, acts[(i + 1) % 5], dtype, bias=False, res=False, save=False, seed=M + N)


# long contractions over few tiles: tiles cut into pieces between CTA pairs
LONG = [(150, 8192, 130), (300, 16384, 520), (700, 4104, 1000), (130, 20000, 24), (2100, 2048, 2304)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,K,N", LONG)
def test_linear_long_contractions(M, K, N, dtype):
    for again in range(2):                     # the counters are back at zero
        linear_case(M, K, N, "gelu_tanh", dtype, bias=True, res=True, save=True, seed=K + again)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("act", list(api.DENSE_ACTS))
@pytest.mark.parametrize("bias,res,save", [(0, 0, 0), (1, 0, 1), (0, 1, 0), (1, 1, 1)])
def test_linear_epilogues(act, bias, res, save, dtype):
    for M in (4, 150, 600):
        linear_case(M, 192, 328, act, dtype, bool(bias), bool(res), bool(save), seed=5)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M", [1, 7, 40, 400])
@pytest.mark.parametrize("pad,off", [(8, 0), (8, 8), (3, 0), (5, 3), (1, 1)])
def test_linear_strided_rows(M, pad, off, dtype):
    linear_case(M, 264, 200, "gelu", dtype, True, True, True, pad=pad, off=off, seed=pad)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M", [1, 20, 300])
def test_linear_residual_in_place(M, dtype):
    linear_case(M, 256, 384, "identity", dtype, True, True, False, inplace=True)
    linear_case(M, 256, 130, "silu", dtype, False, True, False, pad=3, off=1, inplace=True)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M", [2, 100, 700])
def test_linear_infinite_and_nan_inputs_stay_in_their_rows(M, dtype):
    """A row of x with a NaN gives a NaN row; every other row is as without it."""
    g = gen(2)
    x, w = rnd(g, M, 320, dtype=dtype), rnd(g, 136, 320, dtype=dtype, std=0.05)
    y, y2 = (torch.empty(M, 136, dtype=dtype, device="cuda") for _ in range(2))
    cfg = api.linear_config(M, 320, 136, "relu", dtype)
    ws = api.new_linear_workspace(cfg)
    api.moe_linear(cfg, x, w, None, None, y, None, ws)
    x2 = x.clone()
    x2[M // 2, 319] = float("nan")
    api.moe_linear(cfg, x2, w, None, None, y2, None, ws)
    torch.cuda.synchronize()
    assert y2[M // 2].isnan().all()
    keep = torch.arange(M, device="cuda") != M // 2
    assert torch.equal(y[keep], y2[keep])


@pytest.mark.parametrize("T", [1, 4, 16, 17, 130])
def test_gated_overflow_is_an_infinity(T):
    """A hidden value beyond bf16's range makes the results that read it
    infinite, of the product's sign, however many rows the call has; the same
    backward, for dA, dU and h.  (Powers of two: every product is exact, and the
    other hidden values are too small to matter.)"""
    K, f, inf = 16, 24, math.inf
    x = torch.zeros(T, K, dtype=BF16, device="cuda")
    x[:, 0] = 1.0
    w1, w3 = (torch.zeros(f, K, dtype=BF16, device="cuda") for _ in range(2))
    w1[:, 0], w3[:, 0] = 1.0, 1.0
    w1[5, 0], w3[5, 0] = 2.0 ** 70, 2.0 ** 70
    w2 = torch.ones(K, f, dtype=BF16, device="cuda")
    w2[1::2, 5] = -1.0
    y, dx = (torch.empty(T, K, dtype=BF16, device="cuda") for _ in range(2))
    a, u = (torch.empty(T, f, dtype=BF16, device="cuda") for _ in range(2))
    cfg = api.gated_ffn_config(T, K, f, "relu")
    ws = api.new_gated_ffn_workspace(cfg, backward=True)
    api.moe_gated_ffn(cfg, x, w1, None, w3, None, w2, None, None, y, a, u, ws)
    assert (y[:, ::2] == inf).all() and (y[:, 1::2] == -inf).all()
    # dh = 2^60 everywhere, u = 2^70 in column 5: dA, dU and h overflow there
    dy = torch.zeros(T, K, dtype=BF16, device="cuda")
    dy[:, 0] = 2.0 ** 60
    dw1, dw3, db1 = torch.empty_like(w1), torch.empty_like(w1), torch.empty(f, dtype=BF16, device="cuda")
    dw2, db3 = torch.empty_like(w2), torch.empty_like(db1)
    api.moe_gated_ffn_backward(cfg, x, w1, w3, w2, a, u, dy, dx, dw1, db1, dw3, db3, dw2, None, ws)
    api.moe_check_device_errors(ws)
    for t in (dw1[5, 0], dw3[5, 0], dw2[0, 5], db1[5], db3[5]):
        assert t == inf
    assert (dx[:, 0] == inf).all()
    assert dw1[4, 0] == T * 2.0 ** 60            # (T has at most 8 bits)


def test_activation_gradients_far_out():
    """act' of huge finite pre-activations is its limit, 0 or 1."""
    v = torch.tensor([-3e38, -1e20, -1e4, 1e4, 1e20, 3e38], device="cuda")
    for dtype in (BF16, F32):
        for act in ("silu", "gelu", "gelu_tanh", "relu"):
            for M in (1, 40):
                z = v.to(dtype).repeat(M, 1)
                cfg = api.linear_config(M, 8, 6, act, dtype)
                db = torch.empty(6, dtype=dtype, device="cuda")
                api.moe_linear_backward(cfg, None, None, z, torch.ones_like(z), None, None, db,
                                        api.new_linear_workspace(cfg, backward=True))
                assert db.tolist() == [0, 0, 0, M, M, M], (act, dtype, M)


@pytest.mark.parametrize("off", [1, 4])
@pytest.mark.parametrize("M", [40, 400])
def test_column_slices_that_start_anywhere(M, off):
    """x and dy as column slices of rows that are themselves aligned: the same
    bits as from aligned copies (the same kernels run)."""
    g = gen(21)
    K, N = 264, 200
    x, w, dy = (rnd(g, M, K, dtype=BF16, pad=8, off=off), rnd(g, N, K, dtype=BF16, std=0.06),
                rnd(g, M, N, dtype=BF16, pad=8, off=off))
    w1, w3, w2 = (rnd(g, *s, dtype=BF16, std=0.06) for s in ((N, K), (N, K), (K, N)))
    gy = rnd(g, M, K, dtype=BF16, pad=8, off=off)
    a, u = (rnd(g, M, N, dtype=BF16) for _ in range(2))
    got = []
    for copy in (False, True):
        xs, ys, gs = (t.contiguous() if copy else t for t in (x, dy, gy))
        cfg = api.linear_config(M, K, N, ld_x=xs.stride(0), ld_y=ys.stride(0))
        wide = lambda n, t: torch.zeros(M, t.stride(0), dtype=BF16, device="cuda")[:, :n]  # noqa: E731
        o = [wide(N, ys), wide(K, xs), torch.empty_like(w), wide(K, gs), wide(K, xs)]
        o += [torch.empty_like(t) for t in (w1, w3, w2)]
        ws = api.new_linear_workspace(cfg, backward=True)
        api.moe_linear(cfg, xs, w, None, None, o[0], None, ws)
        api.moe_linear_backward(cfg, xs, w, None, ys, o[1], o[2], None, ws)
        gc = api.gated_ffn_config(M, K, N, ld_x=xs.stride(0), ld_y=gs.stride(0))
        ws = api.new_gated_ffn_workspace(gc, backward=True)
        api.moe_gated_ffn(gc, xs, w1, None, w3, None, w2, None, None, o[3], None, None, ws)
        api.moe_gated_ffn_backward(gc, xs, w1, w3, w2, a, u, gs, o[4], o[5], None, o[6], None, o[7], None, ws)
        api.moe_check_device_errors(ws)
        got.append(o)
    for p, q in zip(*got):
        assert torch.equal(p, q)


def test_linear_without_rows_launches_nothing():
    cfg = api.linear_config(0, 64, 64)
    ws = api.new_linear_workspace(cfg)
    e = torch.empty(0, 64, dtype=BF16, device="cuda")
    w = torch.zeros(64, 64, dtype=BF16, device="cuda")
    n = api.kernel_launches()
    api.moe_linear(cfg, e, w, None, None, e.clone(), None, ws)
    assert api.kernel_launches() == n


def linear_backward_case(M, K, N, act, dtype, pad=0, seed=0, want=(1, 1, 1)):
    g = gen(seed + 50)
    x, w = rnd(g, M, K, dtype=dtype, pad=pad), rnd(g, N, K, dtype=dtype, std=K ** -0.5, pad=pad)
    dy = rnd(g, M, N, dtype=dtype, pad=pad)
    z = rnd(g, M, N, dtype=dtype, std=2.0) if act != "identity" else None
    dx = torch.full((M, K + pad), 7.0, dtype=dtype, device="cuda")[:, :K] if want[0] else None
    dw = torch.full((N, K), 7.0, dtype=dtype, device="cuda") if want[1] else None
    db = torch.full((N,), 7.0, dtype=dtype, device="cuda") if want[2] else None
    cfg = api.linear_config(M, K, N, act, dtype, K + pad, K + pad, 0, N + pad)
    ws = api.new_linear_workspace(cfg, backward=True)
    api.moe_linear_backward(cfg, x, w, z, dy, dx, dw, db, ws)
    api.moe_check_device_errors(ws)
    u = U[dtype]
    xd, wd, dz = x.double(), w.double(), dy.double()
    edz = torch.zeros_like(dz)
    if act != "identity":
        f = act64_grad(z.double(), act)
        edz = dz.abs() * FN[dtype] * f.abs().clamp_min(1) * (act != "relu")
        dz = dz * f
        edz = edz + um(dtype, M) * (dz.abs() + edz)
    if want[0]:
        ref = dz @ wd
        e = ck(N) * (dz.abs() @ wd.abs()) + edz @ wd.abs()
        near(dx, ref, e + u * (ref.abs() + e), "dx")
    if want[1]:
        ref = dz.T @ xd
        e = ck(M) * (dz.abs().T @ xd.abs()) + edz.T @ xd.abs()
        near(dw, ref, e + u * (ref.abs() + e), "dw")
    if want[2]:
        ref = dz.sum(0)
        e = ck(M) * dz.abs().sum(0) + edz.sum(0)
        near(db, ref, e + u * (ref.abs() + e), "db")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_linear_backward(M, K, N, dtype):
    acts = list(api.DENSE_ACTS)
    linear_backward_case(M, K, N, acts[(M + N) % 5], dtype, seed=M)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,K,N", [(8192, 130, 300), (20000, 64, 24), (5000, 520, 264), (300, 256, 9000)])
def test_linear_backward_long_contractions(M, K, N, dtype):
    linear_backward_case(M, K, N, "silu", dtype, seed=M)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("act", list(api.DENSE_ACTS))
@pytest.mark.parametrize("pad", [0, 8, 3])
def test_linear_backward_strided(act, pad, dtype):
    linear_backward_case(300, 264, 200, act, dtype, pad=pad)


@pytest.mark.parametrize("want", [(1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 0, 1), (0, 1, 1)])
def test_linear_backward_of_some(want):
    linear_backward_case(70, 64, 48, "silu", BF16, want=want)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("act", ["identity", "gelu"])
def test_backward_without_rows_gives_zero_gradients(act, dtype):
    linear_backward_case(0, 130, 70, act, dtype)


# ------------------------------------- gated -----------------------------------

def gated_refs(x, w1, b1, w3, b3, act, dtype):
    """a, u, h in 64 bits and bounds of the kernel's h before its rounding."""
    K = x.shape[1]
    a, u = x @ w1.T, x @ w3.T
    ea, eu = ck(K) * (x.abs() @ w1.abs().T), ck(K) * (x.abs() @ w3.abs().T)
    if b1 is not None:
        a, u = a + b1, u + b3
        ea, eu = ea + ck(0) * b1.abs(), eu + ck(0) * b3.abs()
    f = act64(a, act)
    ef = SLOPE * ea + FN[dtype] * f.abs().clamp_min(1) * (act not in ("relu", "identity"))
    h = f * u
    eh = ef * (u.abs() + eu) + f.abs() * eu + 2.0 ** -23 * h.abs()
    return a, ea, u, eu, h, eh


def gated_case(T, K, f, act, dtype, bias, res, save, pad=0, inplace=False, seed=0):
    g = gen(seed)
    x = rnd(g, T, K, dtype=dtype, pad=pad)
    w1, w3 = (rnd(g, f, K, dtype=dtype, std=K ** -0.5) for _ in range(2))
    w2 = rnd(g, K, f, dtype=dtype, std=f ** -0.5)
    b1, b3, b2 = (rnd(g, n, dtype=dtype, std=0.5) for n in (f, f, K)) if bias else (None,) * 3
    r = rnd(g, T, K, dtype=dtype, pad=pad) if res else None
    r0 = None if r is None else r.clone()
    y = r if inplace else torch.full((T, K + pad), 7.0, dtype=dtype, device="cuda")[:, :K]
    a, u = (torch.empty(T, f, dtype=dtype, device="cuda") for _ in range(2)) if save else (None, None)
    cfg = api.gated_ffn_config(T, K, f, act, dtype, ld_x=K + pad, ld_y=K + pad, ld_r=K + pad)
    ws = api.new_gated_ffn_workspace(cfg)
    api.moe_gated_ffn(cfg, x, w1, b1, w3, b3, w2, b2, r, y, a, u, ws)
    api.moe_check_device_errors(ws)
    un = U[dtype]
    ar, ea, ur, eu, h, eh = gated_refs(x.double(), w1.double(), d(b1), w3.double(), d(b3), act, dtype)
    if save:
        near(a, ar, ea + un * (ar.abs() + ea), "a")
        near(u, ur, eu + un * (ur.abs() + eu), "u")
    eh = eh + um(dtype, T, 16) * (h.abs() + eh)
    w2d = w2.double()
    yr = h @ w2d.T
    ey = (eh + ck(f) * h.abs()) @ w2d.abs().T
    if bias:
        yr = yr + b2.double()
    if res:
        yr = yr + r0.double()
    ey = ey + 2.0 ** -22 * yr.abs()
    near(y, yr, ey + un * (yr.abs() + ey), "y")


GATED = [(1, 1, 1), (1, 128, 64), (1, 4096, 136), (3, 200, 333), (8, 256, 512), (16, 72, 136), (31, 64, 1000),
         (65, 320, 192), (130, 264, 72), (257, 512, 129), (300, 31, 40), (600, 1024, 328), (1025, 96, 320)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,K,f", GATED)
def test_gated(T, K, f, dtype):
    acts = list(api.DENSE_ACTS)
    i = (T + K + f) % 5
    gated_case(T, K, f, acts[i], dtype, True, True, True, seed=T)
    gated_case(T, K, f, acts[(i + 2) % 5], dtype, False, False, False, seed=f)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("act", list(api.DENSE_ACTS))
@pytest.mark.parametrize("T", [2, 90, 500])
def test_gated_strided(T, act, dtype):
    gated_case(T, 264, 200, act, dtype, True, True, True, pad=3)
    gated_case(T, 264, 200, act, dtype, False, True, False, pad=8, inplace=True)


def gated_backward_case(T, K, f, act, dtype, bias, pad=0, seed=0, drop=()):
    g = gen(seed + 9)
    x, dy = rnd(g, T, K, dtype=dtype, pad=pad), rnd(g, T, K, dtype=dtype, pad=pad)
    w1, w3 = (rnd(g, f, K, dtype=dtype, std=K ** -0.5) for _ in range(2))
    w2 = rnd(g, K, f, dtype=dtype, std=f ** -0.5)
    a, u = rnd(g, T, f, dtype=dtype, std=1.5), rnd(g, T, f, dtype=dtype)
    o = {"dx": torch.full((T, K + pad), 7.0, dtype=dtype, device="cuda")[:, :K]}
    for n, shape in (("dw1", (f, K)), ("dw3", (f, K)), ("dw2", (K, f)), ("db1", (f,)), ("db3", (f,)), ("db2", (K,))):
        o[n] = torch.full(shape, 7.0, dtype=dtype, device="cuda") if bias or n[1] == "w" else None
    for n in drop:
        o[n] = None
    cfg = api.gated_ffn_config(T, K, f, act, dtype, ld_x=K + pad, ld_y=K + pad)
    ws = api.new_gated_ffn_workspace(cfg, backward=True)
    api.moe_gated_ffn_backward(cfg, x, w1, w3, w2, a, u, dy, o["dx"], o["dw1"], o["db1"], o["dw3"], o["db3"],
                               o["dw2"], o["db2"], ws)
    api.moe_check_device_errors(ws)
    un = U[dtype]
    xd, dyd, w1d, w3d, w2d, ad, ud = (t.double() for t in (x, dy, w1, w3, w2, a, u))
    fa, ga = act64(ad, act), act64_grad(ad, act)
    fn = FN[dtype] * (act not in ("relu", "identity"))
    dh = dyd @ w2d
    eh = ck(K) * (dyd.abs() @ w2d.abs())

    def part(factor, rel):
        """dh * factor, rounded: value and bound; rel: error of the factor."""
        v = dh * factor
        e = eh * (factor.abs() + rel) + dh.abs() * rel + 2.0 ** -22 * v.abs()
        return v, e + um(dtype, T) * (v.abs() + e)
    da, eda = part(ud * ga, ud.abs() * fn * ga.abs().clamp_min(1))
    du, edu = part(fa, fn * fa.abs().clamp_min(1))
    hh = fa * ud
    ehh = ud.abs() * fn * fa.abs().clamp_min(1) + 2.0 ** -23 * hh.abs()
    ehh = ehh + um(dtype, T) * (hh.abs() + ehh)

    def product(name, pairs, n):
        if o[name] is None:
            return
        ref = sum(p @ q for p, _, q in pairs)
        e = sum(ck(n * len(pairs)) * (p.abs() @ q.abs()) + ep @ q.abs() for p, ep, q in pairs)
        near(o[name], ref, e + un * (ref.abs() + e), name)
    product("dx", [(da, eda, w1d), (du, edu, w3d)], f)
    product("dw1", [(da.T, eda.T, xd)], T)
    product("dw3", [(du.T, edu.T, xd)], T)
    if o["dw2"] is not None:
        ref = dyd.T @ hh
        e = ck(T) * (dyd.abs().T @ hh.abs()) + dyd.abs().T @ ehh
        near(o["dw2"], ref, e + un * (ref.abs() + e), "dw2")
    for name, v, ev in (("db1", da, eda), ("db3", du, edu), ("db2", dyd, torch.zeros_like(dyd))):
        if o[name] is not None:
            ref = v.sum(0)
            e = ck(T) * v.abs().sum(0) + ev.sum(0)
            near(o[name], ref, e + un * (ref.abs() + e), name)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,K,f", GATED)
def test_gated_backward(T, K, f, dtype):
    gated_backward_case(T, K, f, list(api.DENSE_ACTS)[(T + f) % 5], dtype, True, seed=T)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,K,f", [(300, 4096, 200), (700, 2056, 1000), (4000, 136, 72), (200, 520, 6000)])
def test_gated_long_contractions(T, K, f, dtype):
    gated_case(T, K, f, "silu", dtype, True, True, True, seed=T)
    gated_backward_case(T, K, f, "gelu", dtype, True, seed=T)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("act", list(api.DENSE_ACTS))
def test_gated_backward_strided(act, dtype):
    gated_backward_case(300, 136, 200, act, dtype, False, pad=3)
    gated_backward_case(70, 64, 72, act, dtype, True, pad=8)


@pytest.mark.parametrize("drop", [("dx",), ("dw1", "dw3"), ("dw2", "db2"), ("dx", "dw1", "dw3", "dw2", "db2"),
                                  ("dx", "dw1", "dw3", "dw2", "db1", "db3")])
def test_gated_backward_of_some(drop):
    gated_backward_case(90, 64, 48, "silu", BF16, True, drop=drop)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gated_without_rows(dtype):
    gated_backward_case(0, 64, 130, "silu", dtype, True)
    cfg = api.gated_ffn_config(0, 64, 130, dtype=dtype)
    assert api.new_gated_ffn_workspace(cfg).numel() >= 4096


# --------------------------- gradients against differences ---------------------------

def test_gradients_against_differences():
    """Central differences of the block's 64-bit forward along random
    directions against the fp32 gradients of the kernels.  Error of the
    difference: O(eps^2) curvature, below 1e-6 of the sum of magnitudes at
    eps = 1e-4; fp32 gradients: 2e-6 relative."""
    g = gen(4)
    T, K, f, act = 40, 36, 52, "gelu"
    p = {"x": rnd(g, T, K, dtype=F32), "w1": rnd(g, f, K, dtype=F32, std=0.2), "w3": rnd(g, f, K, dtype=F32, std=0.2),
         "w2": rnd(g, K, f, dtype=F32, std=0.2), "b1": rnd(g, f, dtype=F32), "b3": rnd(g, f, dtype=F32),
         "b2": rnd(g, K, dtype=F32)}
    dy = rnd(g, T, K, dtype=F32)
    block = api.GatedFFN(p["w1"], p["w3"], p["w2"], p["b1"], p["b3"], p["b2"], act)
    block(p["x"], train=True)
    grads = block.backward(p["x"], dy)

    def loss(q):
        h = act64(q["x"] @ q["w1"].T + q["b1"], act) * (q["x"] @ q["w3"].T + q["b3"])
        return ((h @ q["w2"].T + q["b2"]) * dy.double()).sum()
    q = {k: v.double() for k, v in p.items()}
    for k in q:
        v = torch.randn(q[k].shape, generator=g, device="cuda", dtype=torch.float64)
        eps = 1e-4
        num = (loss({**q, k: q[k] + eps * v}) - loss({**q, k: q[k] - eps * v})) / (2 * eps)
        got = (grads["d" + k].double() * v).sum()
        mag = (grads["d" + k].double() * v).abs().sum()
        assert abs(num - got) <= 5e-6 * mag, k


# ----------------------------- a run of them together ---------------------------------

def test_block_around_the_moe_layer_and_clipping():
    """A GatedFFN with residual, then the MoE layer, its backward through both,
    and one clip over all gradients, fp32 and bf16 together."""
    from dataclasses import replace

    from mixture_experts_layer_63_b200.inputs import WORKLOADS, make_inputs
    w = replace(WORKLOADS["deepseekmoe_tc"], T=300, d_model=256, d_ff=128, E=8, k=2)
    inp = make_inputs(w, seed=3, device="cuda")
    moe = api.MoELayer(api.config_from_workload(w), inp.w_router, inp.w1, inp.w2, inp.w3, inp.bias)
    g = gen(8)
    ffn = api.GatedFFN(rnd(g, 320, 256, dtype=BF16, std=1 / 16), rnd(g, 320, 256, dtype=BF16, std=1 / 16),
                       rnd(g, 256, 320, dtype=BF16, std=320 ** -0.5))
    h = ffn(inp.x, residual=inp.x, train=True)
    moe(h)
    dy = rnd(g, w.T, w.d_model, dtype=BF16)
    gm = moe.backward(h, dy)
    gf = ffn.backward(inp.x, gm["dx"].to(BF16))
    api.moe_check_device_errors(moe.ws)
    flat = [t for q in (gm, gf) for k, t in q.items() if k != "dx" and t is not None]
    before = [t.double() for t in flat]
    norm = api.clip_grads([gm, gf], max_norm=0.5)
    ref = torch.stack([t.square().sum() for t in before]).sum().sqrt()
    assert abs(norm.double() - ref) <= 2.0 ** -23 * ref
    assert ref > 0.5
    for t, b in zip(flat, before):
        c = b * (0.5 / (ref + 1e-6))
        assert ((t.double() - c).abs() <= (U[t.dtype] + 2.0 ** -22) * c.abs() + 1e-44).all()


def test_captured_replay_and_other_streams():
    """A captured graph of forward and backward replays with new inputs; the
    same calls on a side stream give the same bits."""
    g = gen(11)
    T, K, f = 200, 256, 384
    block = api.GatedFFN(*(rnd(g, *s, dtype=BF16, std=0.06) for s in ((f, K), (f, K), (K, f))))
    cfg = api.gated_ffn_config(T, K, f)
    x, dy, y, dx = (rnd(g, T, K, dtype=BF16) for _ in range(4))
    a, u = (torch.empty(T, f, dtype=BF16, device="cuda") for _ in range(2))
    dws = [torch.empty_like(t) for t in (block.w1, block.w3, block.w2)]
    ws, bws = api.new_gated_ffn_workspace(cfg), api.new_gated_ffn_workspace(cfg, backward=True)

    def step():
        api.moe_gated_ffn(cfg, x, block.w1, None, block.w3, None, block.w2, None, x, y, a, u, ws)
        api.moe_gated_ffn_backward(cfg, x, block.w1, block.w3, block.w2, a, u, dy, dx, dws[0], None, dws[1], None,
                                   dws[2], None, bws)
    outs = [y, a, u, dx, *dws]
    step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    x.copy_(rnd(g, T, K, dtype=BF16))
    graph.replay()
    torch.cuda.synchronize()
    replayed = [t.clone() for t in outs]
    for t in outs:
        t.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    for p, q in zip(replayed, outs):
        assert torch.equal(p, q)


def test_two_streams_with_their_own_workspaces():
    g = gen(12)
    M, K, N = 300, 512, 640
    cfg = api.linear_config(M, K, N, "silu")
    w = rnd(g, N, K, dtype=BF16, std=0.05)
    xs = [rnd(g, M, K, dtype=BF16) for _ in range(2)]
    ys = [torch.empty(M, N, dtype=BF16, device="cuda") for _ in range(4)]
    wss = [api.new_linear_workspace(cfg) for _ in range(2)]
    for i in range(2):
        api.moe_linear(cfg, xs[i], w, None, None, ys[i], None, wss[i])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for i in range(2):
            api.moe_linear(cfg, xs[i], w, None, None, ys[2 + i], None, wss[i], streams[i])
    torch.cuda.synchronize()
    assert torch.equal(ys[0], ys[2]) and torch.equal(ys[1], ys[3])


def test_block_and_clip_on_a_side_stream_own_what_they_use():
    """Workspaces and outputs of a call on another stream are not handed out
    again, on the current one, while the call still runs."""
    g = gen(16)
    T, K, f = 64, 256, 320
    x, dy = rnd(g, T, K, dtype=BF16), rnd(g, T, K, dtype=BF16)
    ws = [rnd(g, *s, dtype=BF16, std=0.06) for s in ((f, K), (f, K), (K, f))]
    ref = api.GatedFFN(*ws)
    y0 = ref(x, train=True)
    g0 = ref.backward(x, dy)
    grads = [t.clone() for t in (g0["dw1"], g0["dw2"])]
    n0 = api.clip_grads([t.clone() for t in grads], 1e9)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)              # (about 10 ms)
    block = api.GatedFFN(*ws)
    y1 = block(x, train=True, stream=side)
    g1 = block.backward(x, dy, stream=side)
    n1 = api.clip_grads(grads, 1e9, stream=side)
    small = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (512, 4096, 8192, 1 << 20) for _ in range(8)]
    torch.cuda.synchronize()
    assert torch.equal(y0, y1) and n0 == n1 and all(torch.equal(g0[k], g1[k]) for k in ("dx", "dw1", "dw3", "dw2"))
    assert all((t == 255).all() for t in small)


def test_captured_block_outlives_larger_batches():
    """A graph captured before the workspaces grew replays on the ones it was
    captured with."""
    g = gen(17)
    K, f = 256, 320
    block = api.GatedFFN(*(rnd(g, *s, dtype=BF16, std=0.06) for s in ((f, K), (f, K), (K, f))))
    x, dy = rnd(g, 200, K, dtype=BF16), rnd(g, 200, K, dtype=BF16)
    y0 = block(x, train=True)
    g0 = block.backward(x, dy)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = block(x, train=True)
        q = block.backward(x, dy)
    big = rnd(g, 3000, K, dtype=BF16)
    block(big, train=True)
    block.backward(big, big)
    junk = [torch.full((n << 20,), 255, dtype=torch.uint8, device="cuda") for n in (1, 2, 20, 42, 45, 60) for _ in range(2)]
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, y0) and all(torch.equal(q[k], g0[k]) for k in ("dx", "dw1", "dw3", "dw2"))
    assert all((t == 255).all() for t in junk)


def test_one_workspace_serves_different_calls_in_turn():
    """Cut tiles, copies and partial sums of one call leave nothing that the
    next call on the workspace reads."""
    g = gen(14)
    dtype = BF16
    lc, gc = api.linear_config(300, 8200, 520, "gelu"), api.gated_ffn_config(700, 264, 200)
    n = max(api.new_linear_workspace(lc, backward=True).numel(), api.new_gated_ffn_workspace(gc, backward=True).numel())
    shared = torch.randint(0, 255, (n,), dtype=torch.uint8, device="cuda")
    api.moe_workspace_init(shared)
    x, w, z, dy = (rnd(g, *s, dtype=dtype, std=0.3) for s in ((300, 8200), (520, 8200), (300, 520), (300, 520)))
    gx, w1, w3, w2 = (rnd(g, *s, dtype=dtype, std=0.1) for s in ((700, 264), (200, 264), (200, 264), (264, 200)))
    got = []
    for ws in (None, shared, shared):
        o = [torch.empty(s, dtype=dtype, device="cuda") for s in ((300, 520), (300, 8200), (520, 8200), (520,), (700, 264))]
        api.moe_linear(lc, x, w, None, None, o[0], None, api.new_linear_workspace(lc) if ws is None else ws)
        api.moe_gated_ffn(gc, gx, w1, None, w3, None, w2, None, gx, o[4], None, None,
                          api.new_gated_ffn_workspace(gc) if ws is None else ws)
        api.moe_linear_backward(lc, x, w, z, dy, o[1], o[2], o[3],
                                api.new_linear_workspace(lc, backward=True) if ws is None else ws)
        torch.cuda.synchronize()
        got.append(o)
    api.moe_check_device_errors(shared)
    for o in got[1:]:
        assert all(torch.equal(p, q) for p, q in zip(got[0], o))


@pytest.mark.parametrize("M", [3, 300])
def test_fp32_extremes(M):
    """Huge and tiny fp32 values (beyond bf16's rounding range and next to its
    smallest): the split into bf16 parts keeps them; an infinite element makes
    its row's results non-finite and leaves the others alone."""
    g = gen(15)
    K, N = 640, 200
    w = rnd(g, N, K, dtype=F32, std=1.0)
    cfg = api.linear_config(M, K, N, dtype=F32)
    ws = api.new_linear_workspace(cfg)
    for scale in (1e30, 1e-20):
        x = rnd(g, M, K, dtype=F32, std=scale)
        y = torch.empty(M, N, device="cuda")
        api.moe_linear(cfg, x, w, None, None, y, None, ws)
        ref = x.double() @ w.double().T
        near(y, ref, ck(K) * (x.double().abs() @ w.double().abs().T), f"scale {scale}")
    x = rnd(g, M, K, dtype=F32)
    x[0, 0] = 3.4e38                               # rounds to infinity in bf16
    w2 = w * 1e-3
    api.moe_linear(cfg, x, w2, None, None, y, None, ws)
    near(y, x.double() @ w2.double().T, ck(K) * (x.double().abs() @ w2.double().abs().T), "next to the largest")
    x[1, 5] = math.inf
    y2 = torch.empty_like(y)
    api.moe_linear(cfg, x, w2, None, None, y2, None, ws)
    torch.cuda.synchronize()
    assert not y2[1].isfinite().any()
    keep = torch.arange(M, device="cuda") != 1
    assert torch.equal(y[keep], y2[keep])


def test_binding_refuses_wrong_tensors():
    cfg = api.linear_config(8, 16, 24)
    ws = api.new_linear_workspace(cfg)
    x, w = torch.zeros(8, 16, dtype=BF16, device="cuda"), torch.zeros(24, 16, dtype=BF16, device="cuda")
    y = torch.zeros(8, 24, dtype=BF16, device="cuda")
    for bad in (dict(x=x.float()), dict(x=x[:7]), dict(x=x.repeat(1, 2)[:, ::2]), dict(x=x.T), dict(y=x),
                dict(y=torch.zeros(8, 30, dtype=BF16, device="cuda")[:, :24]), dict(w=w.cpu()), dict(w=w[:, :8])):
        kw = dict(x=x, w=w, y=y) | bad
        with pytest.raises(ValueError):
            api.moe_linear(cfg, kw["x"], kw["w"], None, None, kw["y"], None, ws)
    with pytest.raises(ValueError):
        api.moe_linear(cfg, x, w, torch.zeros(23, dtype=BF16, device="cuda"), None, y, None, ws)


def test_results_repeat_bit_for_bit():
    g = gen(13)
    for dtype in (BF16, F32):
        M, K, N = 700, 1032, 520
        x, w, dy = (rnd(g, *s, dtype=dtype, std=0.1) for s in ((M, K), (N, K), (M, N)))
        cfg = api.linear_config(M, K, N, dtype=dtype)
        ws, bws = api.new_linear_workspace(cfg), api.new_linear_workspace(cfg, backward=True)
        got = []
        for _ in range(2):
            y, dx, dw = (torch.empty(s, dtype=dtype, device="cuda") for s in ((M, N), (M, K), (N, K)))
            db = torch.empty(N, dtype=dtype, device="cuda")
            api.moe_linear(cfg, x, w, None, None, y, None, ws)
            api.moe_linear_backward(cfg, x, w, None, dy, dx, dw, db, bws)
            got.append((y, dx, dw, db))
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(*got))


# ------------------------------- offsets past 32 bits ---------------------------------

@pytest.mark.parametrize("dtype,M,K,N", [(BF16, 140000, 64, 16384), (BF16, 1, 16384, 140000), (BF16, 70, 16384, 140000),
                                         (F32, 2, 16384, 140000)])
def test_linear_offsets_past_32_bits(dtype, M, K, N):
    """The last rows and columns of a result or a weight matrix of more than
    2^31 elements, and its gradients."""
    g = gen(30)
    big = max(M * N, N * K)
    assert big > 2 ** 31
    x = rnd(g, M, K, dtype=dtype)
    w = torch.empty(N, K, dtype=dtype, device="cuda")
    w.normal_(std=K ** -0.5, generator=g)
    y = torch.empty(M, N, dtype=dtype, device="cuda")
    cfg = api.linear_config(M, K, N, "relu", dtype)
    ws = api.new_linear_workspace(cfg)
    api.moe_linear(cfg, x, w, None, None, y, None, ws)
    api.moe_check_device_errors(ws)
    del ws
    rows, cols = slice(max(0, M - 40), M), slice(N - 300, N)
    ref = x[rows].double() @ w[cols].double().T
    e = ck(K) * (x[rows].double().abs() @ w[cols].double().abs().T)
    ref = ref.clamp_min(0)
    near(y[rows, cols], ref, e + U[dtype] * (ref + e), "y")
    if M * N <= 2 ** 31:
        return
    ws = api.new_linear_workspace(cfg, backward=True)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty(N, dtype=dtype, device="cuda")
    z = y                                        # as pre-activations: the mask is y > 0
    dy = torch.empty_like(y)
    dy.normal_(generator=g)
    api.moe_linear_backward(cfg, x, w, z, dy, dx, dw, db, ws)
    api.moe_check_device_errors(ws)
    dz = dy[rows].double() * (y[rows] > 0)
    ref = dz @ w.double()
    e = ck(N) * (dz.abs() @ w.double().abs())
    near(dx[rows], ref, e + U[dtype] * (ref.abs() + e), "dx")
    dzc = dy[:, cols].double() * (y[:, cols] > 0)
    for got, ref, mag in ((dw[cols], dzc.T @ x.double(), dzc.abs().T @ x.double().abs()),
                          (db[cols], dzc.sum(0), dzc.abs().sum(0))):
        e = ck(M) * mag
        near(got, ref, e + U[dtype] * (ref.abs() + e), "dw, db")


def test_gated_offsets_past_32_bits():
    g = gen(31)
    T, K, f = 140000, 64, 16384
    x = rnd(g, T, K, dtype=BF16)
    w1, w3, w2 = (rnd(g, *s, dtype=BF16, std=s[1] ** -0.5) for s in ((f, K), (f, K), (K, f)))
    y = torch.empty_like(x)
    cfg = api.gated_ffn_config(T, K, f, "relu")
    ws = api.new_gated_ffn_workspace(cfg)
    api.moe_gated_ffn(cfg, x, w1, None, w3, None, w2, None, None, y, None, None, ws)
    api.moe_check_device_errors(ws)
    xs = x[-40:].double()
    _, _, _, _, h, eh = gated_refs(xs, w1.double(), None, w3.double(), None, "relu", BF16)
    eh = eh + U[BF16] * (h.abs() + eh)
    ref = h @ w2.double().T
    e = (eh + ck(f) * h.abs()) @ w2.double().abs().T
    near(y[-40:], ref, e + U[BF16] * (ref.abs() + e), "y")
