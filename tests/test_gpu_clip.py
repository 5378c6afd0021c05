"""Global gradient norm and clipping against 64 bits.  The norm is one fp32
rounding of a 64-bit value (2^-24; 2^-23 is allowed for the sum's order); a
clipped element carries the fp32 rounding of the factor and of the product
and the tensor's own: (2^-23 + u) |value|, u = 2^-8 (bf16) or 2^-24."""
import math

import pytest
import torch

from mixture_experts_layer_63_b200 import api

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U = {BF16: 2.0 ** -8, F32: 2.0 ** -24}


def make(sizes, seed=0, std=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return [(torch.randn(n, generator=g, device="cuda") * std).to(dt) for n, dt in sizes]


def norm64(ts):
    return math.sqrt(math.fsum(float(t.double().square().sum()) for t in ts))


def check(src, got, norm, max_norm):
    ref = norm64(src)
    assert abs(float(norm) - ref) <= 2.0 ** -23 * ref
    c = min(1.0, max_norm / (ref + 1e-6))
    for s, t in zip(src, got):
        want = s.double() * c
        assert t.shape == s.shape and t.dtype == s.dtype
        assert ((t.double() - want).abs() <= (U[t.dtype] + 2.0 ** -23) * want.abs() + 1e-44).all()
        if c == 1.0:
            assert torch.equal(t, s)


LISTS = {
    "one_element": [(1, F32)],
    "one_bf16": [(1, BF16)],
    "empty_between": [(0, F32), (5, BF16), (0, BF16), (7, F32)],
    "odd": [(4095, F32), (4097, BF16), (12289, F32), (31, BF16)],
    "mixed": [(1 << 20, F32), (999_999, BF16), (64, F32), (300_001, F32)],
    "long": [(33_333_333, BF16), (20_000_003, F32)],
    "many": [(17 * i + 1, F32 if i % 3 else BF16) for i in range(700)],
}


@pytest.mark.parametrize("name", list(LISTS))
@pytest.mark.parametrize("clip", [True, False])
@pytest.mark.parametrize("inplace", [True, False])
def test_clip(name, clip, inplace):
    src = make(LISTS[name], seed=len(name))
    keep = [t.clone() for t in src]
    max_norm = norm64(src) * (0.3 if clip else 2.0)
    out = None if inplace else [torch.full_like(t, 7.0) for t in src]
    norm, ws = torch.empty((), device="cuda"), api.new_clip_workspace(src)
    api.moe_clip_grads(src, max_norm, norm, ws, out=out)
    torch.cuda.synchronize()
    check(keep, src if inplace else out, norm, max_norm)
    if not inplace:
        assert all(torch.equal(p, q) for p, q in zip(src, keep))
    api.moe_grad_norm(keep, norm, ws)
    ref = norm64(keep)
    assert abs(float(norm) - ref) <= 2.0 ** -23 * ref


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("off", [1, 2, 3, 5, 8])
def test_views_at_any_alignment(dt, off):
    """Slices that start anywhere, read and written; what lies beside them stays."""
    g = torch.Generator(device="cuda")
    g.manual_seed(off)
    a, b = (torch.randn(50_000, generator=g, device="cuda").to(dt) for _ in range(2))
    ka, kb = a.clone(), b.clone()
    src, out = [a[off:off + 20_001]], [b[2 * off + 1:2 * off + 20_002]]
    keep = [t.clone() for t in src]
    norm, ws = torch.empty((), device="cuda"), api.new_clip_workspace(src)
    api.moe_clip_grads(src, 1.0, norm, ws, out=out)
    torch.cuda.synchronize()
    check(keep, out, norm, 1.0)
    assert torch.equal(a, ka)
    assert torch.equal(b[:2 * off + 1], kb[:2 * off + 1]) and torch.equal(b[2 * off + 20_002:], kb[2 * off + 20_002:])
    api.moe_clip_grads(src, 1.0, norm, ws)
    torch.cuda.synchronize()
    check(keep, src, norm, 1.0)
    assert torch.equal(a[:off], ka[:off]) and torch.equal(a[off + 20_001:], ka[off + 20_001:])


def test_extreme_values():
    """Squares beyond fp32's range, values below its normal range, zeros."""
    norm = torch.empty((), device="cuda")
    for scale in (1e30, 1e-30):
        src = make([(10_000, F32)], seed=1)
        src = [t * scale for t in src]
        keep = [t.clone() for t in src]
        ws = api.new_clip_workspace(src)
        api.moe_clip_grads(src, 1e-3 * scale, norm, ws)
        torch.cuda.synchronize()
        ref = norm64(keep)
        assert abs(float(norm) - ref) <= 2.0 ** -23 * ref
        c = min(1.0, float(torch.tensor(1e-3 * scale, dtype=F32)) / (ref + 1e-6))
        want = keep[0].double() * c
        assert ((src[0].double() - want).abs() <= 2.0 ** -22 * want.abs() + 1e-44).all()
    z = [torch.zeros(100, device="cuda")]
    api.moe_clip_grads(z, 1.0, norm, ws)
    assert float(norm) == 0.0 and not z[0].any()


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_infinite_and_nan_gradients(bad):
    src = make([(5000, F32), (300, BF16)], seed=2)
    src[0][4321] = bad
    norm, ws = torch.empty((), device="cuda"), api.new_clip_workspace(src)
    api.moe_clip_grads(src, 1.0, norm, ws)
    if math.isnan(bad):
        assert math.isnan(float(norm)) and all(t.isnan().all() for t in src)
    else:
        assert float(norm) == math.inf
        assert src[0][4321].isnan() and src[0].isnan().sum() == 1
        assert (src[0].nan_to_num() == 0).all() and (src[1] == 0).all()


def test_infinite_max_norm_leaves_every_bit():
    src = make([(70_000, F32), (333, BF16)], seed=3, std=1e3)
    keep = [t.clone() for t in src]
    norm, ws = torch.empty((), device="cuda"), api.new_clip_workspace(src)
    api.moe_clip_grads(src, math.inf, norm, ws)
    torch.cuda.synchronize()
    check(keep, src, norm, math.inf)
    api.moe_clip_grads(src, 1.0, None, ws)                 # no norm wanted
    torch.cuda.synchronize()
    check(keep, src, norm, 1.0)


def test_empty_list_and_repeatability():
    norm = torch.full((), 5.0, device="cuda")
    ws = api.new_clip_workspace([])
    api.moe_grad_norm([], norm, ws)
    assert float(norm) == 0.0
    api.moe_clip_grads([None], 1.0, norm, ws)
    assert float(norm) == 0.0
    src = make([(1_234_567, F32), (7_654_321, BF16)], seed=4)
    ws = api.new_clip_workspace(src)
    got = []
    for _ in range(3):
        api.moe_grad_norm(src, norm, ws)
        got.append(float(norm))
    assert len(set(got)) == 1


def test_captured_clip_reads_new_gradients():
    src = make([(40_000, F32), (999, BF16)], seed=5)
    norm, ws = torch.empty((), device="cuda"), api.new_clip_workspace(src)
    out = [torch.empty_like(t) for t in src]
    api.moe_clip_grads(src, 1.0, norm, ws, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.moe_clip_grads(src, 1.0, norm, ws, out=out)
    for t, n in zip(src, make([(40_000, F32), (999, BF16)], seed=6, std=3.0)):
        t.copy_(n)
    graph.replay()
    torch.cuda.synchronize()
    check(src, out, norm, 1.0)


def test_refusals():
    t = torch.ones(100, device="cuda")
    norm, ws = torch.empty((), device="cuda"), api.new_clip_workspace([t])
    for bad in ([t, t], [t, t[50:]]):
        with pytest.raises(api.MoeError):
            api.moe_clip_grads(bad, 1.0, norm, ws)
    api.moe_grad_norm([t, t], norm, ws)                    # reading twice is fine
    assert abs(float(norm) - math.sqrt(200)) < 1e-5
    for bad in (dict(max_norm=0.0), dict(max_norm=math.nan)):
        with pytest.raises(api.MoeError):
            api.moe_clip_grads([t], bad["max_norm"], norm, ws)
    for g, out in (([t[::2]], None), ([t], [t[:50]]), ([t], [t.to(BF16)]), ([t.to(torch.float16)], None),
                   ([t.cpu()], None), ([t, t], [t])):
        with pytest.raises(ValueError):
            api.moe_clip_grads(g, 1.0, norm, ws, out=out)
    assert (t == 1).all()


def test_offsets_past_32_bits():
    """Three elements behind the first 2^31 of a tensor, zeros before them."""
    t = torch.zeros(2 ** 31 + 5, dtype=BF16, device="cuda")
    t[-3:] = torch.tensor([3.0, 4.0, 12.0], dtype=BF16)
    norm, ws = torch.empty((), device="cuda"), api.new_clip_workspace([t])
    api.moe_clip_grads([t], 6.5, norm, ws)
    assert norm.item() == 13.0
    assert t[-3:].tolist() == [1.5, 2.0, 6.0]         # c = 0.5 (1 - 1e-7), rounded to bf16
    assert not t[:-3].any()
