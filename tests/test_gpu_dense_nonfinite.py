"""NaN in the dense operators: which results it reaches is compared with the
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
