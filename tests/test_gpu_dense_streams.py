"""Calls of different sizes at once, on streams of their own with workspaces of
their own: few-row products, the gated block, large products and the MoE layer
share the SMs, their shared memory and tensor memory.  Every result has the
bits that the call gives alone."""
from dataclasses import replace

import pytest
import torch

from mixture_experts_layer_63_b200 import api

from .test_gpu_dense import BF16, gen, rnd

pytestmark = pytest.mark.gpu


def linear(g, M, K, N):
    cfg = api.linear_config(M, K, N)
    x, w, y = rnd(g, M, K, dtype=BF16), rnd(g, N, K, dtype=BF16, std=0.03), torch.empty(M, N, dtype=BF16, device="cuda")
    ws = api.new_linear_workspace(cfg)
    return lambda: api.moe_linear(cfg, x, w, None, None, y, None, ws), [y], ws


def gated(g, T, K, f):
    cfg = api.gated_ffn_config(T, K, f)
    x, y = rnd(g, T, K, dtype=BF16), torch.empty(T, K, dtype=BF16, device="cuda")
    w = [rnd(g, *s, dtype=BF16, std=0.03) for s in ((f, K), (f, K), (K, f))]
    ws = api.new_gated_ffn_workspace(cfg)
    return lambda: api.moe_gated_ffn(cfg, x, w[0], None, w[1], None, w[2], None, x, y, None, None, ws), [y], ws


def layer():
    from mixture_experts_layer_63_b200.inputs import WORKLOADS, make_inputs
    w = replace(WORKLOADS["deepseekmoe_tc"], T=300, d_model=256, d_ff=128, E=8, k=2)
    inp = make_inputs(w, seed=3, device="cuda")
    moe = api.MoELayer(api.config_from_workload(w), inp.w_router, inp.w1, inp.w2, inp.w3, inp.bias)
    out = torch.empty_like(inp.x)
    return lambda: out.copy_(moe(inp.x)), [out], moe.ws


SETS = {
    "gated and linear of 80 rows": lambda g: [gated(g, 80, 2048, 5632), linear(g, 80, 4096, 4096), gated(g, 72, 1024, 4096)],
    "a token beside batches": lambda g: [linear(g, 1, 4096, 4096), gated(g, 80, 2048, 5632), gated(g, 128, 1024, 4096),
                                         linear(g, 12, 2048, 9000)],
    "decoding beside the layer": lambda g: [layer(), linear(g, 1, 4096, 4096), gated(g, 16, 2048, 5632)],
    "prompts beside decoding": lambda g: [linear(g, 700, 2048, 2048), gated(g, 300, 1024, 2048), gated(g, 4, 2048, 5632),
                                          linear(g, 100, 4096, 1024)],
}


@pytest.mark.parametrize("name", list(SETS))
def test_calls_at_once(name):
    calls = SETS[name](gen(80))
    for call, _, _ in calls:
        call()
    torch.cuda.synchronize()
    alone = [[t.clone() for t in out] for _, out, _ in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(40):
        for s, (call, _, _) in zip(streams, calls):
            with torch.cuda.stream(s):
                call()
    torch.cuda.synchronize()
    for (_, out, ws), want in zip(calls, alone):
        api.moe_check_device_errors(ws)
        assert all(torch.equal(p, q) for p, q in zip(out, want))
