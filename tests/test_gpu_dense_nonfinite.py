"""NaN and infinities in the dense operators: which results it reaches is compared with the
formulas' in 64 bits, place by place, and every other result with what the call
gives without it, bit for bit."""
import math

import pytest
import torch

from mixture_experts_layer_63_b200 import api

from .test_gpu_dense import BF16, F32, act64, act64_grad, gen, rnd

pytestmark = pytest.mark.gpu

ACTS = list(api.DENSE_ACTS)


def grad64(z, act):
    """act' with act'(NaN) = NaN (identity: 1)."""
    g = act64_grad(z, act)
    return g if act == "identity" else torch.where(z.isnan(), z, g)


def check(got, clean, ref, what):
    """`got` is NaN where `ref` is, infinite of its sign where `ref` is, and has the bits of `clean` elsewhere."""
    assert torch.equal(got.isnan(), ref.isnan()), what
    assert torch.equal(got == math.inf, ref == math.inf) and torch.equal(got == -math.inf, ref == -math.inf), what
    ok = ref.isfinite()
    assert torch.equal(got[ok], clean[ok]), what


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("act", [a for a in ACTS if a != "identity"])
@pytest.mark.parametrize("M", [1, 3, 40, 300])
def test_nan_pre_activation_of_a_linear_backward(M, act, dtype):
    g = gen(60)
    K, N = 136, 200
    x, w, dy = rnd(g, M, K, dtype=dtype), rnd(g, N, K, dtype=dtype, std=0.1), rnd(g, M, N, dtype=dtype)
    z = rnd(g, M, N, dtype=dtype)
    cfg = api.linear_config(M, K, N, act, dtype)
    ws = api.new_linear_workspace(cfg, backward=True)

    def run(z):
        o = [torch.empty_like(t) for t in (x, w)] + [torch.empty(N, dtype=dtype, device="cuda")]
        api.moe_linear_backward(cfg, x, w, z, dy, *o, ws)
        return o
    clean = run(z)
    z2 = z.clone()
    z2[M // 2, 77] = math.nan
    got = run(z2)
    api.moe_check_device_errors(ws)
    dz = dy.double() * grad64(z2.double(), act)
    for p, q, r, n in zip(got, clean, (dz @ w.double(), dz.T @ x.double(), dz.sum(0)), ("dx", "dw", "db")):
        check(p, q, r, n)
    assert got[0][M // 2].isnan().all() and got[1][77].isnan().all() and got[2][77].isnan()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T", [1, 3, 40, 300])
@pytest.mark.parametrize("where", ["a", "u"])
def test_nan_pre_activation_of_a_gated_backward(where, T, act, dtype):
    g = gen(61)
    K, f = 72, 136
    x, dy = rnd(g, T, K, dtype=dtype), rnd(g, T, K, dtype=dtype)
    w1, w3, w2 = (rnd(g, *s, dtype=dtype, std=0.1) for s in ((f, K), (f, K), (K, f)))
    p = {"a": rnd(g, T, f, dtype=dtype), "u": rnd(g, T, f, dtype=dtype)}
    cfg = api.gated_ffn_config(T, K, f, act, dtype)
    ws = api.new_gated_ffn_workspace(cfg, backward=True)

    def run(a, u):
        o = {n: torch.empty(s, dtype=dtype, device="cuda") for n, s in
             (("dx", (T, K)), ("dw1", (f, K)), ("db1", (f,)), ("dw3", (f, K)), ("db3", (f,)), ("dw2", (K, f)),
              ("db2", (K,)))}
        api.moe_gated_ffn_backward(cfg, x, w1, w3, w2, a, u, dy, *o.values(), ws)
        return o
    clean = run(**p)
    p[where] = p[where].clone()
    p[where][T // 2, 101] = math.nan
    got = run(**p)
    api.moe_check_device_errors(ws)
    xd, dyd, w1d, w3d, w2d, a, u = (t.double() for t in (x, dy, w1, w3, w2, p["a"], p["u"]))
    dh, h = dyd @ w2d, act64(a, act) * u
    da, du = dh * u * grad64(a, act), dh * act64(a, act)
    ref = {"dx": da @ w1d + du @ w3d, "dw1": da.T @ xd, "db1": da.sum(0), "dw3": du.T @ xd, "db3": du.sum(0),
           "dw2": dyd.T @ h, "db2": dyd.sum(0)}
    for n in ref:
        check(got[n], clean[n], ref[n], n)
    assert got["dw2"][:, 101].isnan().all()


def spots(t, places, values):
    t = t.clone()
    for (i, j), v in zip(places, values):
        t[i, j] = v
    return t


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M", [1, 3, 12, 20, 40, 150, 300])
@pytest.mark.parametrize("side", ["x", "w", "both"])
def test_infinite_elements_of_a_linear_forward(side, M, dtype):
    """inf v = +-inf, inf 0 = NaN, inf - inf = NaN, inf inf = inf, whatever the
    rows: sizes on every kernel."""
    g = gen(62)
    for K, N in ((136, 200), (4096, 264)):
        x, w = rnd(g, M, K, dtype=dtype), rnd(g, N, K, dtype=dtype, std=0.1)
        w[3, 5] = 0.0
        clean, got = (torch.empty(M, N, dtype=dtype, device="cuda") for _ in range(2))
        cfg = api.linear_config(M, K, N, "identity", dtype)
        ws = api.new_linear_workspace(cfg)
        api.moe_linear(cfg, x, w, None, None, clean, None, ws)
        if side != "w":
            x = spots(x, [(M - 1, 5), (M // 2, 7), (M // 2, 100)], [math.inf, -math.inf, math.inf])
        if side != "x":
            w = spots(w, [(9, 5), (9, 131), (N - 1, 7)], [math.inf, math.inf, -math.inf])
        api.moe_linear(cfg, x, w, None, None, got, None, ws)
        api.moe_check_device_errors(ws)
        check(got, clean, x.double() @ w.double().T, f"{K} x {N}")


@pytest.mark.parametrize("M", [6, 40, 300])
def test_infinite_elements_of_an_fp32_linear_backward(M):
    g = gen(63)
    K, N = 264, 392
    x, w, dy = rnd(g, M, K, dtype=F32), rnd(g, N, K, dtype=F32, std=0.1), rnd(g, M, N, dtype=F32)
    cfg = api.linear_config(M, K, N, "identity", F32)
    ws = api.new_linear_workspace(cfg, backward=True)

    def run():
        o = [torch.empty_like(x), torch.empty_like(w), torch.empty(N, device="cuda")]
        api.moe_linear_backward(cfg, x, w, None, dy, *o, ws)
        return o
    clean = run()
    x, w = spots(x, [(1, 200)], [-math.inf]), spots(w, [(300, 17), (301, 17)], [math.inf, -math.inf])
    dy = spots(dy, [(M - 1, 2), (1, 3)], [math.inf, -math.inf])
    got = run()
    api.moe_check_device_errors(ws)
    for p, q, r, n in zip(got, clean, (dy.double() @ w.double(), dy.double().T @ x.double(), dy.double().sum(0)),
                          ("dx", "dw", "db")):
        check(p, q, r, n)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [1, 7, 16, 17, 130, 300])
def test_infinite_weights_of_a_gated_block(T, dtype):
    """The second product's: h is handed on in planes, of few rows too."""
    g = gen(64)
    K, f = 136, 328
    x = rnd(g, T, K, dtype=dtype)
    w1, w3, w2 = (rnd(g, *s, dtype=dtype, std=0.1) for s in ((f, K), (f, K), (K, f)))
    clean, got = (torch.empty(T, K, dtype=dtype, device="cuda") for _ in range(2))
    cfg = api.gated_ffn_config(T, K, f, "silu", dtype)
    ws = api.new_gated_ffn_workspace(cfg)
    api.moe_gated_ffn(cfg, x, w1, None, w3, None, w2, None, None, clean, None, None, ws)
    w2 = spots(w2, [(5, 300), (60, 0), (60, 9)], [math.inf, -math.inf, -math.inf])
    api.moe_gated_ffn(cfg, x, w1, None, w3, None, w2, None, None, got, None, None, ws)
    api.moe_check_device_errors(ws)
    h = act64(x.double() @ w1.double().T, "silu") * (x.double() @ w3.double().T)
    check(got, clean, h @ w2.double().T, "y")
