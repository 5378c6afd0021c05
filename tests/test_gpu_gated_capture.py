"""A GatedFFN whose first use, or whose growth, is inside a capture: eager calls
before the first replay, a second graph replayed first, and a graph of the
backward pass alone (sizes whose tiles are cut, so that the control block's
counters matter).  Every result is compared bit for bit with another object's
that never saw a capture."""
import pytest
import torch

from mixture_experts_layer_63_b200 import api

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
T, K, F = 300, 4096, 520


def data(seed=40):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s, std=1.0: (torch.randn(*s, generator=g, device="cuda") * std).to(BF16)  # noqa: E731
    ws = [r(F, K, std=K ** -0.5), r(F, K, std=K ** -0.5), r(K, F, std=F ** -0.5)]
    return ws, r(T, K), r(T, K)


def step(block, x, dy):
    y = block(x, train=True)
    return [y, *(v for v in block.backward(x, dy).values() if v is not None)]


def same(p, q):
    torch.cuda.synchronize()
    return all(torch.equal(a, b) for a, b in zip(p, q, strict=True))


def junk(block):
    """Memory that a capture allocated holds anything before the first replay."""
    for t in block.graph_ws.values():
        t.fill_(171)
    torch.cuda.synchronize()


@pytest.mark.parametrize("warm", [0, 3])
def test_eager_calls_and_a_second_graph_before_the_first_replay(warm):
    ws, x, dy = data()
    ref = step(api.GatedFFN(*ws), x, dy)
    torch.cuda.synchronize()
    block = api.GatedFFN(*ws)
    if warm:
        step(block, x[:warm], dy[:warm])
    graphs, outs = [], []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(step(block, x, dy))
        junk(block)
    assert same(step(block, x, dy), ref)
    junk(block)
    for i in (1, 0, 1):
        for t in outs[i]:
            t.fill_(7.0)
        graphs[i].replay()
        assert same(outs[i], ref)
    assert same(step(block, x, dy), ref)
    for t in (block.ws, block.bws):
        api.moe_check_device_errors(t)


def test_graph_of_the_backward_alone_outlives_the_next_forward():
    ws, x, dy = data(41)
    ref = step(api.GatedFFN(*ws), x, dy)[1:]
    block = api.GatedFFN(*ws)
    step(block, x, dy)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g = block.backward(x, dy)
    block(dy, train=True)                          # replaces a and u
    other = [torch.full((T, F), 3.0, dtype=BF16, device="cuda") for _ in range(4)]
    graph.replay()
    assert same([v for v in g.values() if v is not None], ref)
    assert all((t == 3).all() for t in other)
