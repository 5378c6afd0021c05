"""Clipping without a limit (an infinite max_norm: the norm alone is wanted, and
every gradient keeps its bits, whatever it holds)."""
import math

import pytest
import torch

from mixture_experts_layer_63_b200 import api

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("inplace", [True, False])
def test_infinite_limit_leaves_every_bit_of_an_infinite_or_nan_gradient(bad, inplace):
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    src = [torch.randn(70_001, generator=g, device="cuda"), torch.randn(333, generator=g, device="cuda").to(BF16)]
    src[0][4321] = bad
    src[1][7] = bad
    keep = [t.clone() for t in src]
    out = None if inplace else [torch.full_like(t, 7.0) for t in src]
    norm, ws = torch.empty((), device="cuda"), api.new_clip_workspace(src)
    api.moe_clip_grads(src, math.inf, norm, ws, out=out)
    torch.cuda.synchronize()
    assert math.isnan(float(norm)) if math.isnan(bad) else float(norm) == math.inf
    for t, k in zip(src if inplace else out, keep):
        ok = k.isfinite()
        assert torch.equal(t[ok], k[ok]) and torch.equal(t.isnan(), k.isnan()) and torch.equal(t == bad, k == bad)
