"""The norm's entry points on the host: sizes and refusals (nothing is enqueued)."""
import os

import pytest
import torch

from weight_shared_rank_amd import binding

A = 1 << 32          # never dereferenced: every call below is refused, or has no tokens
BIG = 1 << 40
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(binding.LIBPATH):
        from weight_shared_rank_amd import build
        build.build(verbose=False)
    return binding.lib()


def norm(L, **kw):
    T, K = kw.pop("T", 4), kw.pop("K", 256)
    a = dict(x=A, res=None, w=2 * A, wt=0, offset=0.0, eps=1e-6, h=None, y=3 * A, code=None, cb=0, rstd=None)
    a.update(kw)
    return L.weightless_norm(a["x"], a["res"], T, K, a["w"], a["wt"], a["offset"], a["eps"], a["h"], a["y"], a["code"],
                             a["cb"], a["rstd"], None)


def back(L, **kw):
    T, K = kw.pop("T", 40), kw.pop("K", 256)
    a = dict(dy=A, h=2 * A, rstd=3 * A, dh=None, w=4 * A, wt=0, offset=0.0, dx=5 * A, dw=6 * A, ws=7 * A, wsb=BIG)
    a.update(kw)
    return L.weightless_norm_backward(a["dy"], a["h"], a["rstd"], a["dh"], T, K, a["w"], a["wt"], a["offset"], a["dx"],
                                      a["dw"], a["ws"], a["wsb"], None)


def test_shapes_refused(L):
    for t, k, status in ((1, 0, -2), (1, -8, -2), (1, 12, -2), (1, 32776, -2), (1 << 20, 1 << 15, 0), (-1, 64, -1),
                         ((1 << 20) + 1, 64, -2)):
        n = L.weightless_norm_backward_workspace_bytes(t, k)
        if status:
            assert n == 0 and norm(L, T=t, K=k) == status and back(L, T=t, K=k) == status, (t, k)
        else:
            assert n >= 256 and n % 256 == 0


def test_no_tokens(L):
    assert norm(L, T=0, x=None, w=None, y=None) == 0
    assert back(L, T=0, dw=None, dy=None, h=None, rstd=None, w=None) == 0
    assert back(L, T=0, dx=None, dw=None) == 0


def test_norm_arguments_refused(L):
    cb = L.weightless_act_code_bytes(4, 256)
    rows = 4 * 256 * 2
    for bad, status, frag in (
            (dict(x=None), -1, "x is NULL"), (dict(w=None), -1, "w is NULL"), (dict(x=A + 8), -1, "x must be 16-byte"),
            (dict(w=A + 8), -1, "w must be"), (dict(res=A + 8), -1, "res must be"), (dict(h=A + 8), -1, "h must be"),
            (dict(y=A + 8), -1, "y must be"), (dict(rstd=A + 2), -1, "rstd must be"), (dict(wt=2), -3, "dtype"),
            (dict(eps=0.0), -1, "eps"), (dict(eps=-1.0), -1, "eps"), (dict(eps=NAN), -1, "eps"), (dict(eps=INF), -1, "eps"),
            (dict(offset=NAN), -1, "offset"), (dict(offset=INF), -1, "offset"), (dict(y=None), -1, "no output"),
            (dict(code=A + 128, cb=cb), -1, "256-byte"), (dict(code=9 * A, cb=cb - 1), -5, "code buffer"),
            (dict(y=A), -1, "overlap"),
            (dict(h=A + 16), -1, "overlap"), (dict(h=A + rows - 16), -1, "overlap"), (dict(res=5 * A, h=5 * A + 16), -1, "overlap"),
            (dict(h=3 * A), -1, "overlap"), (dict(y=2 * A), -1, "overlap"), (dict(code=3 * A, cb=cb), -1, "overlap"),
            (dict(rstd=3 * A + 64), -1, "overlap"), (dict(code=A, cb=cb), -1, "overlap")):
        assert norm(L, **bad) == status and frag in binding.last_error(), (bad, binding.last_error())


def test_backward_arguments_refused(L):
    need = L.weightless_norm_backward_workspace_bytes(40, 256)
    for bad, status, frag in (
            (dict(dy=None), -1, "dy is NULL"), (dict(h=None), -1, "h is NULL"), (dict(rstd=None), -1, "rstd is NULL"),
            (dict(w=None), -1, "w is NULL"), (dict(dx=None, dw=None), -1, "no output"), (dict(dx=A + 8), -1, "dx must be"),
            (dict(dw=A + 4), -1, "dw must be"), (dict(dh=A + 2), -1, "dh must be"), (dict(wt=7), -3, "dtype"),
            (dict(offset=NAN), -1, "offset"), (dict(ws=None), -1, "workspace"), (dict(ws=7 * A + 64), -1, "workspace"),
            (dict(wsb=need - 1), -5, "workspace"), (dict(dx=2 * A), -1, "overlap"), (dict(dx=A + 16), -1, "overlap"),
            (dict(dh=9 * A, dx=9 * A + 16), -1, "overlap"), (dict(dw=A), -1, "overlap"), (dict(dw=5 * A), -1, "overlap"),
            (dict(ws=5 * A), -1, "overlap"), (dict(ws=2 * A), -1, "overlap"), (dict(dw=7 * A), -1, "overlap")):
        assert back(L, **bad) == status and frag in binding.last_error(), (bad, binding.last_error())


def test_binding_refuses_host_tensors_and_unknown_outputs(L):
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(64)
    with pytest.raises(binding.WlError, match="device tensor"):
        binding.norm_act(x, w)
    with pytest.raises(binding.WlError, match="device tensor"):
        binding.norm_backward(x, x, torch.zeros(4), w)
    for call, msg in ((lambda: binding._only_wanted(("z",), ("y",), {}), "unknown"), (lambda: binding._only_wanted((), ("y",), {}), "no output"),
                      (lambda: binding._only_wanted(("y",), ("y", "h"), {"h": x}), "not wanted")):
        with pytest.raises(binding.WlError, match=msg):
            call()
