"""What the dense operators' results are worth as a whole, and the forms that no
other test's operands reach.

fp32 products of tensor-core size: ||result - reference|| <= 5e-7 ||reference||.
The operands are split in three bf16 parts and six of the nine products of
parts kept; what is left out is below 5e-8 of the norm (the CPU test evaluates
it).  A chunk of 128 terms takes eight additions of its leading products into
the accumulator, each cut towards zero: half a unit of the last place on
average, 0.36 * 2^-23 of the sum so far, which grows over the chunk to its end
and is 0.7 of it on average: 8 * 0.36 * 0.7 * 2^-23 = 2.4e-7 of a chunk, and, as
chunks have either sign, of the result.  The chunks are added with roundings to
nearest, 2^-24 of a running sum at most, of either sign.  The bound is twice the
expectation.  Without any one of the six products the error is over it, with
products of two parts only (4e-6) eight times, as the CPU test shows.
"""
import pytest
import torch

from mixture_experts_layer_63_b200 import api

from .test_gpu_dense import BF16, F32, act64, act64_grad, ck, gen, near, rnd, U

NORM = 5e-7


def parts(v, n):
    out = []
    for _ in range(n):
        h = v.to(BF16).float()
        out.append(h)
        v = v - h
    return out


@pytest.mark.parametrize("M,K,N", [(300, 640, 200), (130, 4096, 136), (64, 16384, 72)])
def test_fewer_products_of_parts_are_over_the_bound(M, K, N):
    """The bound tells three parts from two, and the six products from five."""
    g = torch.Generator().manual_seed(K)
    x, w = torch.randn(M, K, generator=g), torch.randn(N, K, generator=g)
    ref = x.double() @ w.double().T
    a, b = parts(x, 3), parts(w, 3)

    def off(pairs):
        got = sum(a[i].double() @ b[j].double().T for i, j in pairs)
        return ((got - ref).norm() / ref.norm()).item()
    six = [(0, 0), (0, 1), (1, 0), (1, 1), (0, 2), (2, 0)]
    assert off(six) < NORM / 10
    for gone in six:
        assert off([p for p in six if p != gone]) > NORM, gone
    assert off([(0, 0), (0, 1), (1, 0), (1, 1)]) > 5 * NORM


def whole(got, ref, what):
    e = ((got.double() - ref).norm() / ref.norm()).item()
    assert e <= NORM, f"{what}: {e:.2e} of the norm"


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,N", [(300, 256, 264), (520, 640, 200), (256, 4096, 1024), (40, 4096, 2048), (2100, 2048, 2304),
                                   (300, 16384, 520), (1000, 4104, 700)])
def test_fp32_linear_and_its_gradients(M, K, N):
    g = gen(70)
    x, w, dy = rnd(g, M, K, dtype=F32), rnd(g, N, K, dtype=F32, std=K ** -0.5), rnd(g, M, N, dtype=F32)
    y, dx, dw = torch.empty(M, N, device="cuda"), torch.empty_like(x), torch.empty_like(w)
    cfg = api.linear_config(M, K, N, dtype=F32)
    ws = api.new_linear_workspace(cfg, backward=True)
    api.moe_linear(cfg, x, w, None, None, y, None, ws)
    api.moe_linear_backward(cfg, x, w, None, dy, dx, dw, None, ws)
    api.moe_check_device_errors(ws)
    xd, wd, dyd = x.double(), w.double(), dy.double()
    whole(y, xd @ wd.T, "y")
    whole(dx, dyd @ wd, "dx")
    whole(dw, dyd.T @ xd, "dw")


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,f", [(300, 640, 520), (700, 2056, 1000), (40, 4096, 1024)])
def test_fp32_gated_block_products(T, K, f):
    """Each product of the block by itself: a and u; dw2 (h is elementwise); y, dx
    and the other weight gradients carry two products, one after another."""
    g = gen(71)
    x, dy = rnd(g, T, K, dtype=F32), rnd(g, T, K, dtype=F32)
    w1, w3, w2 = (rnd(g, *s, dtype=F32, std=s[1] ** -0.5) for s in ((f, K), (f, K), (K, f)))
    y, a, u = torch.empty_like(x), torch.empty(T, f, device="cuda"), torch.empty(T, f, device="cuda")
    cfg = api.gated_ffn_config(T, K, f, "silu", F32)
    ws = api.new_gated_ffn_workspace(cfg, backward=True)
    api.moe_gated_ffn(cfg, x, w1, None, w3, None, w2, None, None, y, a, u, ws)
    dx, d1, d3, d2 = torch.empty_like(x), torch.empty_like(w1), torch.empty_like(w3), torch.empty_like(w2)
    api.moe_gated_ffn_backward(cfg, x, w1, w3, w2, a, u, dy, dx, d1, None, d3, None, d2, None, ws)
    api.moe_check_device_errors(ws)
    xd, dyd, w1d, w3d, w2d = (t.double() for t in (x, dy, w1, w3, w2))
    whole(a, xd @ w1d.T, "a")
    whole(u, xd @ w3d.T, "u")
    ad, ud = a.double(), u.double()               # (inputs of what follows)
    fa, h = act64(ad, "silu"), act64(ad, "silu") * ud
    dh = dyd @ w2d
    da, du = dh * ud * act64_grad(ad, "silu"), dh * fa

    def two(got, ref, what):
        """Two products in a row, and the elementwise steps between (2^-20 of
        the factors' scale): twice the bound and 1e-6."""
        e = ((got.double() - ref).norm() / ref.norm()).item()
        assert e <= 2 * NORM + 1e-6, f"{what}: {e:.2e} of the norm"
    two(y, h @ w2d.T, "y")
    two(dx, da @ w1d + du @ w3d, "dx")
    two(d1, da.T @ xd, "dw1")
    two(d3, du.T @ xd, "dw3")
    two(d2, dyd.T @ h, "dw2")


# ------------------- bf16 weights whose base is not 16-byte aligned -------------------

def at_offset(t, off):
    """The same matrix, packed, from element `off` of a buffer on."""
    flat = torch.zeros(t.numel() + 16, dtype=t.dtype, device="cuda")
    v = flat[off:off + t.numel()].view(t.shape)
    return v.copy_(t)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["gelu", "silu"])
@pytest.mark.parametrize("M", [1, 4, 11, 40, 150, 400])
@pytest.mark.parametrize("off", [1, 4])
def test_weights_at_unaligned_addresses(off, M, act):
    """Slices of a flat parameter buffer: rows apart by a multiple of 16 bytes
    from a base that is not one (what no copy has room for)."""
    g = gen(72)
    K, N = 264, 200
    x, w, dy = rnd(g, M, K, dtype=BF16), at_offset(rnd(g, N, K, dtype=BF16, std=K ** -0.5), off), rnd(g, M, N, dtype=BF16)
    b, r = rnd(g, N, dtype=BF16), rnd(g, M, N, dtype=BF16)
    y, z = (torch.empty(M, N, dtype=BF16, device="cuda") for _ in range(2))
    dx, dw, db = torch.empty_like(x), torch.empty(N, K, dtype=BF16, device="cuda"), torch.empty_like(b)
    cfg = api.linear_config(M, K, N, act)
    ws = api.new_linear_workspace(cfg, backward=True)
    api.moe_linear(cfg, x, w, b, r, y, z, ws)
    xd, wd, u = x.double(), w.double(), U[BF16]
    zr = xd @ wd.T + b.double()
    ez = ck(K) * (xd.abs() @ wd.abs().T) + ck(0) * b.double().abs()
    near(z, zr, ez + u * (zr.abs() + ez), "z")
    yr = act64(zr, act)
    ey = 1.13 * ez + 2.0 ** -18 * yr.abs().clamp_min(1)
    yr = yr + r.double()
    ey = ey + 2.0 ** -23 * yr.abs()
    near(y, yr, ey + u * (yr.abs() + ey), "y")
    api.moe_linear_backward(cfg, x, w, z, dy, dx, dw, db, ws)
    api.moe_check_device_errors(ws)
    fg = act64_grad(z.double(), act)
    dz = dy.double() * fg
    edz = dy.double().abs() * 2.0 ** -18 * fg.abs().clamp_min(1)
    edz = edz + (2.0 ** -17 if M <= 4 else u) * (dz.abs() + edz)
    for got, ref, e, n in ((dx, dz @ wd, ck(N) * (dz.abs() @ wd.abs()) + edz @ wd.abs(), "dx"),
                           (dw, dz.T @ xd, ck(M) * (dz.abs().T @ xd.abs()) + edz.T @ xd.abs(), "dw"),
                           (db, dz.sum(0), ck(M) * dz.abs().sum(0) + edz.sum(0), "db")):
        near(got, ref, e + u * (ref.abs() + e), n)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 4, 11, 40, 300])
@pytest.mark.parametrize("which", ["w1", "w3", "w2", "all"])
def test_gated_weights_at_unaligned_addresses(which, T):
    """Against the same call with aligned weights: the two differ by how their
    sums are ordered and by the roundings that this moves, one step of h, dA
    and dU and one of the result."""
    g = gen(73)
    K, f = 136, 200
    x, dy = rnd(g, T, K, dtype=BF16), rnd(g, T, K, dtype=BF16)
    a, u = rnd(g, T, f, dtype=BF16), rnd(g, T, f, dtype=BF16)
    w = {n: rnd(g, *s, dtype=BF16, std=s[1] ** -0.5) for n, s in (("w1", (f, K)), ("w3", (f, K)), ("w2", (K, f)))}
    v = {n: at_offset(t, 3) if which in (n, "all") else t for n, t in w.items()}
    cfg = api.gated_ffn_config(T, K, f, "silu")
    ws = api.new_gated_ffn_workspace(cfg, backward=True)
    got = []
    for q in (w, v):
        o = [torch.empty_like(x)]
        api.moe_gated_ffn(cfg, x, q["w1"], None, q["w3"], None, q["w2"], None, x, o[0], None, None, ws)
        o += [torch.empty_like(x)] + [torch.empty(t.shape, dtype=BF16, device="cuda") for t in w.values()]
        api.moe_gated_ffn_backward(cfg, x, q["w1"], q["w3"], q["w2"], a, u, dy, o[1], o[2], None, o[3], None, o[4],
                                   None, ws)
        got.append(o)
    api.moe_check_device_errors(ws)
    xd, dyd, ad, ud, w1, w3, w2 = (t.double() for t in (x, dy, a, u, w["w1"], w["w3"], w["w2"]))
    fa, ga, dh = act64(ad, "silu"), act64_grad(ad, "silu"), dyd.abs() @ w2.abs()
    h = act64(xd @ w1.T, "silu").abs() * (xd @ w3.T).abs()
    eh = (1.13 * ck(K) + 2.0 ** -18) * ((xd.abs() @ w1.abs().T).clamp_min(1) * (xd.abs() @ w3.abs().T).clamp_min(1))
    da, du, hh = dh * (ud * ga).abs(), dh * fa.abs(), (fa * ud).abs()
    step = 2 * U[BF16]
    mags = [((h * step + 2 * eh) @ w2.abs().T, xd.abs() + h @ w2.abs().T),
            (step * (da @ w1.abs() + du @ w3.abs()), da @ w1.abs() + du @ w3.abs()),
            (step * (da.T @ xd.abs()), da.T @ xd.abs()), (step * (du.T @ xd.abs()), du.T @ xd.abs()),
            (step * (dyd.abs().T @ hh), dyd.abs().T @ hh)]
    for p, q, (inner, mag), n in zip(*got, mags, ("y", "dx", "dw1", "dw3", "dw2")):
        bound = inner + 2 * ck(K + f + T) * mag + step * (p.double().abs() + inner)
        over = ((p.double() - q.double()).abs() / (bound + 1e-30)).max().item()
        assert over <= 1.0, f"{n}: {over:.2f} times the bound"
