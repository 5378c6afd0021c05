"""Host validation of the dense operators (linear, gated feed-forward block,
gradient clipping): every refusal returns before any CUDA call, so this runs
without a GPU.  Pointers are plain numbers here; nothing dereferences them."""
import ctypes

import pytest
import torch

from mixture_experts_layer_63_b200 import api

OK, INVALID, UNSUPPORTED, WORKSPACE = (api.MOE_OK, api.MOE_ERR_INVALID_ARG, api.MOE_ERR_UNSUPPORTED,
                                       api.MOE_ERR_WORKSPACE)
BIG = 1 << 40           # addresses far apart from one another


def A(i):
    """The address of buffer i."""
    return BIG * (i + 1)


@pytest.fixture(scope="module")
def L():
    from mixture_experts_layer_63_b200 import build
    build.build()
    return api.lib()


def lin(**kw):
    c = api.linear_config(10, 24, 40, act="relu")
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def gated(**kw):
    c = api.gated_ffn_config(10, 24, 40)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def size(fn, cfg, backward=0):
    out = ctypes.c_size_t(0)
    return getattr(api.lib(), fn)(ctypes.byref(cfg), backward, ctypes.byref(out)), out.value


@pytest.mark.parametrize("kw,status", [
    (dict(), OK), (dict(M=0), OK), (dict(M=-1), INVALID), (dict(K=0), INVALID), (dict(N=0), INVALID),
    (dict(act=5), INVALID), (dict(act=-1), INVALID), (dict(dtype=2), INVALID), (dict(reserved=1), INVALID),
    (dict(ld_x=23), INVALID), (dict(ld_x=25), OK), (dict(ld_w=-24), INVALID), (dict(ld_y=39), INVALID),
    (dict(ld_r=1), INVALID), (dict(M=1 << 31), UNSUPPORTED)])
def test_linear_configs(L, kw, status):
    assert size("moe_query_linear_size", lin(**kw))[0] == status
    assert size("moe_query_linear_size", lin(**kw), 1)[0] == status
    assert size("moe_query_linear_size", lin(**kw), 2)[0] == INVALID


@pytest.mark.parametrize("kw,status", [
    (dict(), OK), (dict(T=0), OK), (dict(T=-1), INVALID), (dict(d_model=0), INVALID), (dict(d_ff=-2), INVALID),
    (dict(act=9), INVALID), (dict(dtype=-1), INVALID), (dict(reserved=3), INVALID), (dict(ld_x=3), INVALID),
    (dict(ld_y=24), OK), (dict(ld_r=23), INVALID), (dict(T=1 << 31), UNSUPPORTED)])
def test_gated_configs(L, kw, status):
    assert size("moe_query_gated_ffn_size", gated(**kw))[0] == status


def test_sizes_beyond_any_memory_are_refused(L):
    """... before their byte counts pass 64 bits."""
    big = 0x7fffffff
    for c in (lin(M=big, N=big), lin(M=big, K=big), lin(K=big, N=big), lin(M=big, ld_x=big)):
        assert size("moe_query_linear_size", c)[0] == UNSUPPORTED
        assert size("moe_query_linear_size", c, 1)[0] == UNSUPPORTED
    for c in (gated(T=big, d_ff=big), gated(d_model=big, d_ff=big), gated(T=big, d_model=big)):
        assert size("moe_query_gated_ffn_size", c)[0] == UNSUPPORTED
    st, n = size("moe_query_linear_size", lin(M=1 << 20, N=1 << 20))
    assert st == OK and n < 1 << 40


def linear_call(L, c, x=A(0), w=A(1), b=A(2), r=A(3), y=A(4), z=A(5), ws=A(6), nws=None):
    n = size("moe_query_linear_size", c)[1] if nws is None else nws
    return L.moe_linear(ctypes.byref(c), x, w, b, r, y, z, ws, n, None)


def test_linear_refusals(L):
    c = lin()
    for kw in (dict(x=None), dict(w=None), dict(y=None), dict(ws=None), dict(ws=A(6) + 8), dict(x=A(0) + 1),
               dict(b=A(2) + 1), dict(z=A(5) + 1), dict(y=A(4) + 1)):
        assert linear_call(L, c, **kw) == INVALID, kw
    assert linear_call(L, c, nws=100) == WORKSPACE
    assert L.moe_linear(None, A(0), A(1), None, None, A(4), None, A(6), 1 << 20, None) == INVALID
    # y over x, w, b, half of r, z
    for kw in (dict(y=A(0) + 2), dict(y=A(1) + 24 * 40 * 2 - 2), dict(y=A(2) - 10 * 40 * 2 + 2),
               dict(y=A(3) + 2), dict(z=A(4)), dict(z=A(0))):
        assert linear_call(L, c, **kw) == INVALID, kw
    # the residual with another row stride is not the same rows
    assert linear_call(L, lin(ld_r=44), y=A(3)) == INVALID
    # the residual in place, and column slices of one buffer, are accepted
    # (without a GPU the launch itself fails; it is not asked for with one)
    if not torch.cuda.is_available():
        assert linear_call(L, c, y=A(3)) == api.MOE_ERR_CUDA
        assert linear_call(L, lin(ld_x=64, ld_y=64), y=A(0) + 24 * 2) == api.MOE_ERR_CUDA
        assert linear_call(L, lin(ld_x=63, ld_y=63), y=A(0) + 24 * 2) == INVALID
    # no rows: nothing to read or write
    assert linear_call(L, lin(M=0), x=None, y=None) == OK


def test_linear_backward_refusals(L):
    def call(c, x=A(0), w=A(1), z=A(2), dy=A(3), dx=A(4), dw=A(5), db=A(6), ws=A(7), nws=None):
        n = size("moe_query_linear_size", c, 1)[1] if nws is None else nws
        return L.moe_linear_backward(ctypes.byref(c), x, w, z, dy, dx, dw, db, ws, n, None)
    c = lin()
    for kw in (dict(x=None), dict(w=None), dict(z=None), dict(dy=None), dict(dx=None, dw=None, db=None),
               dict(ws=None), dict(dx=A(0)), dict(dx=A(3)), dict(dw=A(1)), dict(db=A(5)), dict(dw=A(4)),
               dict(dx=A(2) + 4), dict(dw=A(5) + 1)):
        assert call(c, **kw) == INVALID, kw
    assert call(c, nws=size("moe_query_linear_size", c, 1)[1] - 1) == WORKSPACE
    # the forward's workspace is smaller: dz and the column sums live here
    assert size("moe_query_linear_size", c, 1)[1] > size("moe_query_linear_size", c)[1]


def test_gated_refusals(L):
    c = gated()
    n = size("moe_query_gated_ffn_size", c)[1]

    def call(x=A(0), w1=A(1), b1=A(2), w3=A(3), b3=A(4), w2=A(5), b2=A(6), r=A(7), y=A(8), a=A(9), u=A(10),
             ws=A(11), nws=n):
        return L.moe_gated_ffn(ctypes.byref(c), x, w1, b1, w3, b3, w2, b2, r, y, a, u, ws, nws, None)
    for kw in (dict(x=None), dict(w1=None), dict(w3=None), dict(w2=None), dict(y=None), dict(b1=None),
               dict(b3=None), dict(a=None), dict(u=None), dict(ws=None), dict(y=A(0)), dict(a=A(10)),
               dict(u=A(8)), dict(y=A(5)), dict(w1=A(1) + 1), dict(y=A(7) + 2)):
        assert call(**kw) == INVALID, kw
    assert call(nws=n - 1) == WORKSPACE
    nb = size("moe_query_gated_ffn_size", c, 1)[1]
    assert nb > n

    def back(x=A(0), w1=A(1), w3=A(2), w2=A(3), a=A(4), u=A(5), dy=A(6), dx=A(7), dw1=A(8), db1=A(9),
             dw3=A(10), db3=A(11), dw2=A(12), db2=A(13), ws=A(14), nws=nb):
        return L.moe_gated_ffn_backward(ctypes.byref(c), x, w1, w3, w2, a, u, dy, dx, dw1, db1, dw3, db3, dw2,
                                        db2, ws, nws, None)
    none = dict(dx=None, dw1=None, db1=None, dw3=None, db3=None, dw2=None, db2=None)
    for kw in (none, dict(dw1=None), dict(db3=None), dict(x=None), dict(w1=None), dict(w2=None), dict(a=None),
               dict(u=None), dict(dy=None), dict(dx=A(0)), dict(dx=A(4)), dict(dw1=A(10)), dict(db2=A(6))):
        assert back(**kw) == INVALID, kw
    assert back(nws=n) == WORKSPACE


def grads(*entries):
    arr = (api.MoeGrad * max(1, len(entries)))()
    for e, (src, dst, n, dt) in zip(arr, entries):
        e.src, e.dst, e.n, e.dtype = src, dst, n, dt
    return bytes(arr), len(entries)


def test_clip_refusals(L):
    need = ctypes.c_size_t(0)
    assert L.moe_query_clip_size(3, ctypes.byref(need)) == OK
    assert L.moe_query_clip_size(-1, ctypes.byref(need)) == INVALID
    f, h = api.MOE_F32, api.MOE_BF16

    def clip(entries, max_norm=1.0, norm=A(20), ws=A(21), nws=need.value):
        arr, n = grads(*entries)
        return L.moe_clip_grads(arr, n, max_norm, norm, ws, nws, None)
    good = (A(0), A(0), 100, f)
    for bad in (dict(entries=[(A(0), A(0), -1, f)]), dict(entries=[(A(0), A(0), 4, 5)]),
                dict(entries=[(None, A(0), 4, f)]), dict(entries=[(A(0), None, 4, f)]),
                dict(entries=[(A(0) + 2, A(0) + 2, 4, f)]),
                dict(entries=[good, good]),                                   # listed twice
                dict(entries=[good, (A(0) + 200, A(0) + 200, 4, h)]),         # inside another
                dict(entries=[(A(0), A(0) + 40, 100, f)]),                    # dst over its own src
                dict(entries=[(A(0), A(1), 100, f), (A(2), A(1) + 396, 4, f)]),
                dict(entries=[(A(0), A(1), 100, f), (A(1) + 396, A(3), 4, f)]),
                dict(entries=[good], max_norm=0.0), dict(entries=[good], max_norm=-1.0),
                dict(entries=[good], max_norm=float("nan")), dict(entries=[good], ws=None),
                dict(entries=[good], norm=A(0) + 4), dict(entries=[good], norm=A(20) + 2)):
        assert clip(**bad) == INVALID, bad
    assert clip([good], nws=16) == WORKSPACE
    arr, n = grads(good)
    assert L.moe_grad_norm(arr, n, None, A(21), need.value, None) == INVALID
    assert L.moe_grad_norm(None, 1, A(20), A(21), need.value, None) == INVALID
    assert L.moe_grad_norm(arr, -1, A(20), A(21), need.value, None) == INVALID


def test_clip_workspace_grows_with_the_list(L):
    n = [ctypes.c_size_t(0) for _ in range(2)]
    assert L.moe_query_clip_size(1, ctypes.byref(n[0])) == OK
    assert L.moe_query_clip_size(5000, ctypes.byref(n[1])) == OK
    assert n[1].value > n[0].value


def test_struct_layout_matches_the_header(tmp_path):
    import os
    import shutil
    import subprocess
    if shutil.which("gcc") is None:
        pytest.skip("gcc not found")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    structs = ((api.MoeLinearConfig, "moe_linear_config"), (api.MoeGatedFfnConfig, "moe_gated_ffn_config"),
               (api.MoeGrad, "moe_grad"))
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "moe.h"', 'int main(void) {']
    for st, cname in structs:
        lines.append(f'printf("{cname} %zu\\n", sizeof({cname}));')
        lines += [f'printf("{cname}.{f} %zu\\n", offsetof({cname}, {f}));' for f, _ in st._fields_]
    lines.append("return 0; }")
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines))
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), str(src), "-o", str(exe)], check=True)
    got = dict(ln.split() for ln in subprocess.run([str(exe)], capture_output=True, text=True,
                                                   check=True).stdout.splitlines())
    for st, cname in structs:
        assert int(got[cname]) == ctypes.sizeof(st)
        for f, _ in st._fields_:
            assert int(got[f"{cname}.{f}"]) == getattr(st, f).offset, f


def test_binding_refuses_cpu_tensors_and_unknown_options(L):
    with pytest.raises(ValueError):
        api.linear_config(1, 2, 3, act="tanh")
    with pytest.raises(ValueError):
        api.gated_ffn_config(1, 2, 3, dtype=torch.float16)
    t = torch.zeros(4, 4)
    with pytest.raises(ValueError):
        api._grad_list([t])
