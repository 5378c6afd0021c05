"""Workspaces and pre-activations of a GatedFFN across captures.  What a
capture records runs at the replay, the clearing of a workspace's control
block too: the counters of cut tiles and the wait limit in it must not be
taken for cleared before.  Here a capture is a flag and the launches are
noted; test_gpu_gated_capture.py runs the same on a GPU."""
import pytest
import torch

from mixture_experts_layer_63_b200 import api

K, F = 64, 96


@pytest.fixture
def fake(monkeypatch):
    """capturing: whether a capture is under way; seen: each launch's workspace
    and whether its control block was clear; buffers come filled with other bytes."""
    from mixture_experts_layer_63_b200 import build
    build.build()

    class Fake:
        capturing = False
        seen = []
    f = Fake()
    f.seen = []
    empty = torch.empty

    def dirty(*a, **kw):
        t = empty(*a, **kw)
        return t.fill_(171) if t.dtype is torch.uint8 else t

    def note(*args):
        ws = args[-1]
        f.seen.append((ws, not ws[:4096].any()))
        if f.capturing:                     # nothing of it has run yet
            ws.fill_(171)
    monkeypatch.setattr(torch, "empty", dirty)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: f.capturing)
    monkeypatch.setattr(api, "moe_gated_ffn", note)
    monkeypatch.setattr(api, "moe_gated_ffn_backward", note)
    return f


def block():
    t = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    return api.GatedFFN(t(F, K), t(F, K), t(K, F))


def rows(n):
    return torch.zeros(n, K, dtype=torch.bfloat16)


def run(b, n, backward):
    x = rows(n)
    if backward:
        b.backward(x, x)
    else:
        b(x, train=True)


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("warm", [0, 8])
def test_eager_call_after_a_capture_finds_a_cleared_block(fake, backward, warm):
    """First use inside a capture, or a capture of a larger batch than before."""
    b = block()
    if warm:
        run(b, warm, False)
        run(b, warm, backward)
    elif backward:
        run(b, 4000, False)
    fake.capturing = True
    if backward and warm:
        run(b, 4000, False)
    run(b, 4000, backward)
    assert fake.seen[-1][1]                 # cleared within the graph itself
    graph = fake.seen[-1][0]
    fake.capturing = False
    for n in (4000, 300):
        if backward:
            run(b, n, False)
        run(b, n, backward)
        ws, clear = fake.seen[-1]
        assert clear and ws is not graph


@pytest.mark.parametrize("backward", [False, True])
def test_second_graph_clears_for_itself(fake, backward):
    """Two graphs on one object: either may be replayed first."""
    b = block()
    fake.capturing = True
    for _ in range(2):
        run(b, 500, False)
        run(b, 500, backward)
        assert fake.seen[-1][1]
    assert any(fake.seen[-1][0] is t for t in b.captured)


def test_capture_uses_a_cleared_workspace_that_is_there(fake):
    b = block()
    run(b, 500, False)
    ws = fake.seen[-1][0]
    fake.capturing = True
    run(b, 400, False)
    assert fake.seen[-1][0] is ws and any(ws is t for t in b.captured)


def test_captured_backward_keeps_what_it_reads(fake):
    """A graph of backward alone reads the a and u of an eager forward, which
    the next training forward replaces."""
    b = block()
    run(b, 200, False)
    run(b, 200, True)
    a, u = b.a, b.u
    fake.capturing = True
    run(b, 200, True)
    fake.capturing = False
    run(b, 200, False)
    assert b.a is not a and all(any(t is k for k in b.captured) for t in (a, u))
