"""The adapters' entry points on the host: sizes and refusals (nothing is enqueued)."""
import ctypes
import os

import pytest
import torch

from weight_shared_rank_amd import binding

A = 1 << 36          # never dereferenced: every call below is refused, or has no tokens
BIG = 1 << 50


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(binding.LIBPATH):
        from weight_shared_rank_amd import build
        build.build(verbose=False)
    return binding.lib()


def pool(n=4, r=32, K=256, kids=2, rows=(512, 256, 0), vt=A, u=2 * A, scale=3 * A, rank=4 * A):
    return binding.WlAdapters(n, r, K, kids, (ctypes.c_int32 * 3)(*rows), vt, u, scale, rank)


def add(L, p, T=20, x=5 * A, index=6 * A, base=7 * A, y=8 * A, ws=9 * A, wsb=BIG):
    return L.weightless_adapters_add(ctypes.byref(p), x, index, T, base, y, ws, wsb, None)


def back(L, p, T=20, x=5 * A, xb=BIG, dy=6 * A, index=7 * A, base=8 * A, dx=9 * A, du=10 * A, dv=11 * A, ws=12 * A, wsb=BIG):
    g = binding.WlAdapterGrads(base, dx, du, dv)
    return L.weightless_adapters_backward(ctypes.byref(p), x, xb, dy, index, T, ctypes.byref(g), ws, wsb, None)


SHAPES = (dict(n=0), dict(n=4097), dict(r=0), dict(r=8), dict(r=24), dict(r=272), dict(K=0), dict(K=12), dict(K=(1 << 20) + 8),
          dict(kids=0), dict(kids=4), dict(rows=(512, 0, 0)), dict(rows=(-1, 4, 4)), dict(rows=((1 << 20) + 1, 4, 4)))


def test_struct_layout():
    assert binding.WlAdapters.d_vt.offset == 32 and ctypes.sizeof(binding.WlAdapters) == 64


@pytest.mark.parametrize("bad", SHAPES)
def test_shapes_refused(L, bad):
    p = pool(**bad)
    assert L.weightless_adapters_workspace_bytes(ctypes.byref(p), 4) == 0 and binding.last_error()
    assert L.weightless_adapters_backward_workspace_bytes(ctypes.byref(p), 4) == 0
    assert add(L, p) == -2 and back(L, p) == -2


def test_token_counts(L):
    p = pool()
    assert add(L, p, T=-1) == -1 and add(L, p, T=(1 << 20) + 1) == -2
    assert add(L, p, T=0, x=None, index=None, base=None, y=None, ws=None, wsb=0) == 0
    assert L.weightless_adapters_workspace_bytes(None, 4) == 0 and "NULL" in binding.last_error()
    assert L.weightless_adapters_add(None, A, A, 1, A, A, A, BIG, None) == -1
    for T in (0, 1, 16, 256, 257, 4096, 1 << 20):
        n = L.weightless_adapters_workspace_bytes(ctypes.byref(p), T)
        assert n >= 256 and n % 256 == 0


def test_arguments_refused(L):
    need = L.weightless_adapters_workspace_bytes(ctypes.byref(pool()), 20)
    for field, bad, frag in (("vt", None, "vt is NULL"), ("vt", A + 8, "vt must be"), ("u", None, "u is NULL"), ("u", A + 8, "u must be"),
                             ("scale", None, "scale is NULL"), ("scale", A + 2, "scale must"), ("rank", A + 2, "rank must")):
        assert add(L, pool(**{field: bad})) == -1 and frag in binding.last_error(), (field, binding.last_error())
    for bad, status, frag in (
            (dict(x=None), -1, "x is NULL"), (dict(x=A + 2), -1, "x must"), (dict(index=None), -1, "index is NULL"),
            (dict(index=A + 2), -1, "index must"), (dict(base=None), -1, "base is NULL"), (dict(y=None), -1, "y is NULL"),
            (dict(y=8 * A + 1), -1, "y must"), (dict(ws=None), -1, "workspace"), (dict(ws=9 * A + 16), -1, "workspace"),
            (dict(wsb=need - 1), -5, "workspace"), (dict(y=5 * A), -1, "overlap"), (dict(y=A), -1, "overlap"), (dict(y=2 * A), -1, "overlap"),
            (dict(y=7 * A + 2), -1, "overlap"), (dict(y=6 * A), -1, "overlap"), (dict(ws=8 * A), -1, "overlap"), (dict(ws=7 * A), -1, "overlap"),
            (dict(ws=3 * A), -1, "overlap")):
        assert add(L, pool(), **bad) == status and frag in binding.last_error(), (bad, binding.last_error())


def test_backward_arguments_refused(L):
    p = pool()
    need = L.weightless_adapters_backward_workspace_bytes(ctypes.byref(p), 20)
    assert need % 256 == 0 and need > 0
    for bad, status, frag in (
            (dict(dx=None, du=None, dv=None), -1, "no output"), (dict(x=None), -1, "checkpoint is NULL"), (dict(x=5 * A + 64), -1, "256-byte"),
            (dict(xb=64), -5, "checkpoint"), (dict(dy=None), -1, "dy is NULL"), (dict(dy=A + 1), -1, "dy must"), (dict(index=None), -1, "index"),
            (dict(base=None), -1, "base is NULL"), (dict(dx=9 * A + 8), -1, "dx must"), (dict(du=A + 8), -1, "du must"), (dict(dv=A + 8), -1, "dv must"),
            (dict(ws=None), -1, "workspace"), (dict(wsb=need - 1), -5, "workspace"), (dict(dx=8 * A + 16), -1, "overlap"), (dict(du=2 * A), -1, "overlap"),
            (dict(dv=A), -1, "overlap"), (dict(dv=10 * A), -1, "overlap"), (dict(dx=5 * A), -1, "overlap"), (dict(ws=10 * A), -1, "overlap"),
            (dict(ws=6 * A), -1, "overlap"), (dict(du=6 * A), -1, "overlap")):
        assert back(L, p, **bad) == status and frag in binding.last_error(), (bad, binding.last_error())
    assert back(L, p, T=-1) == -1 and back(L, p, T=0, du=None, dv=None, x=None, dy=None, index=None, base=None, ws=None) == 0
    assert L.weightless_adapters_backward(ctypes.byref(p), A, BIG, A, A, 4, None, A, BIG, None) == -1


def test_binding_refuses_host_tensors(L):
    with pytest.raises(binding.WlError, match="device tensor"):
        binding.AdapterPool(torch.zeros(2, 16, 64, dtype=torch.bfloat16), torch.zeros(2, 64, 16, dtype=torch.bfloat16), torch.ones(2), (64,))
