"""The list of gradients that the binding hands to the C entry points, from
whatever holds the tensors.  (Addresses and sizes only: no GPU.)"""
import struct

import pytest
import torch

from mixture_experts_layer_63_b200 import api


@pytest.fixture(autouse=True)
def any_device(monkeypatch):
    monkeypatch.setattr(api, "_on_device", lambda t: None)


def entries(packed):
    raw, n = packed
    v = struct.unpack("=" + "QQqii" * n, raw)
    return [v[5 * i:5 * i + 5] for i in range(n)]


def tensors():
    return [torch.zeros(8), torch.zeros(8), torch.zeros(8, dtype=torch.bfloat16), torch.zeros(3)]


@pytest.mark.parametrize("make", [list, tuple, iter, lambda ts: (t for t in ts),
                                  lambda ts: {str(i): t for i, t in enumerate(ts)}.values()])
def test_any_iterable_lists_each_tensor_once_in_place(make):
    ts = tensors()
    got = entries(api._grad_list(make(ts)))
    want = [(t.data_ptr(), t.data_ptr(), t.numel(), api._DTYPES[t.dtype], 0) for t in ts]
    assert got == want


@pytest.mark.parametrize("make", [list, iter])
def test_outputs_go_with_their_gradients(make):
    ts, out = tensors(), tensors()
    got = entries(api._grad_list(make(ts), make(out)))
    assert [(s, d) for s, d, *_ in got] == [(t.data_ptr(), o.data_ptr()) for t, o in zip(ts, out)]


def test_gradients_without_their_output_are_refused():
    ts = tensors()
    for out in ([*ts[:3], None], ts[:3], iter(ts[:3]), [*ts, ts[0]]):
        with pytest.raises(ValueError):
            api._grad_list(ts, out)
    # no gradient: no output asked for
    assert len(entries(api._grad_list([None, ts[0]], [None, ts[1]]))) == 1
