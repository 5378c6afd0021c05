"""The list of gradients that the binding hands to the C entry points, from
whatever holds the tensors, and sizes that no memory holds.  (Addresses and
sizes only: no GPU.)"""
import ctypes
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


def test_sizes_beyond_any_memory_are_refused():
    """... before their byte counts pass 64 bits or their chunk counts 32."""
    from mixture_experts_layer_63_b200 import build
    build.build()
    L, need = api.lib(), ctypes.c_size_t(0)
    assert L.moe_query_clip_size(300, ctypes.byref(need)) == api.MOE_OK
    ws, norm = 1 << 60, 1 << 59
    big = 1 << 46
    for sizes in ([big + 1], [1 << 62], [(1 << 63) - 1], [3, big - 2], [1 << 62, 1 << 62, 1 << 62, 1 << 62],
                  [big // 128] * 129):
        for dt in (api.MOE_F32, api.MOE_BF16):
            arr = (api.MoeGrad * len(sizes))()
            for i, (e, n) in enumerate(zip(arr, sizes)):
                e.src = e.dst = 256 * (i + 1)
                e.n, e.dtype = n, dt
            raw = bytes(arr)
            assert L.moe_clip_grads(raw, len(sizes), 1.0, norm, ws, need.value, None) == api.MOE_ERR_UNSUPPORTED
            assert L.moe_grad_norm(raw, len(sizes), norm, ws, need.value, None) == api.MOE_ERR_UNSUPPORTED
            arr[0].n = -1                                # (a wrong entry is named first)
            assert L.moe_grad_norm(bytes(arr), len(sizes), norm, ws, need.value, None) == api.MOE_ERR_INVALID_ARG
