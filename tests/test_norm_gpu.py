"""GPU: the norm with the residual's addition and coded output, and its gradients.

References in float64.  Tolerances, derived before the first run, per element,
with a bf16 rounding 2^-8 and a float32 rounding 2^-24 of the value:

  h      equal: one bf16 rounding of a float32 sum of two bf16
  rstd   2^-23 (float64 rounded to float32)
  y      2^-8 |y| + 2^-22 |y|   (the weight's offset is added in float32: 2^-24; the products, three more)
  code   equal to weightless_act_encode of the y returned
  dx     2^-8 |dx| + 2^-7 smallest normal, and before it, in float32: a (|g| + |n| |mean|) 2^-20
         + a |n| (K + 8) 2^-24 mean_k |g n|
  dw     (T + 8) 2^-23 sum_t |dy n|
"""
import sys

import pytest
import torch

from weight_shared_rank_amd import binding

pytestmark = pytest.mark.gpu
DEV = "cuda"
H, F = 2.0 ** -8, 2.0 ** -24
TINY = 2.0 ** -133          # bf16's smallest step
EPS = 1e-6
ALL = ("y", "code", "h", "rstd")


def announce(msg):
    sys.__stderr__.write(f"[gpu] {msg}\n")
    sys.__stderr__.flush()


def randn(seed, *shape, std=1.0, dtype=torch.bfloat16):
    g = torch.Generator("cpu").manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype).to(DEV)


def check_forward(o, x, w, res, offset, eps=EPS):
    h = x if res is None else (x.float() + res.float()).to(torch.bfloat16)
    if o.h is not None:
        assert torch.equal(o.h.view(torch.int16), h.view(torch.int16))
    hd = h.double()
    a = (hd.square().mean(1) + eps) ** -0.5
    if o.rstd is not None:
        assert ((o.rstd.double() - a).abs() <= 2 * F * a).all()
    if o.y is not None:
        ref = hd * a[:, None] * (offset + w.double())
        err = (o.y.double() - ref).abs()
        assert (err <= (H + 4 * F) * ref.abs() + TINY).all(), err.max()
        if ref.numel() >= 256:
            assert err.norm() <= H * ref.norm()
    if o.code is not None:
        same_code(o.code, binding.encode_act(o.y))


def same_code(a, b):
    n = binding.lib().weightless_act_code_bytes(a.T, a.K)
    at = -(-a.T * a.blocks * 128 // 256) * 256
    assert torch.equal(a.buf[:a.T * a.blocks * 128], b.buf[:a.T * a.blocks * 128])
    run = a.blocks * (-(-a.T // 16) * 16)
    assert at + run <= n and torch.equal(a.buf[at:at + run], b.buf[at:at + run])


SHAPES = [(1, 8), (3, 64), (5, 128), (4, 136), (17, 504), (9, 512), (2, 520), (333, 1152), (6, 1160), (7, 2048),
          (8, 2056), (5, 5376), (16, 8192), (3, 8200), (2, 16384), (15, 21504), (2, 24584), (1, 32768)]


@pytest.mark.parametrize("T,K", SHAPES)
@pytest.mark.parametrize("res,f32,offset", [(True, False, 1.0), (False, True, 0.0)])
def test_forward(gpu_lib, T, K, res, f32, offset):
    announce(f"norm {T} x {K} res={res} f32={f32}")
    x, r = randn(1, T, K, std=3.0), randn(2, T, K) if res else None
    w = randn(3, K, std=0.5, dtype=torch.float32 if f32 else torch.bfloat16)
    check_forward(binding.norm_act(x, w, EPS, residual=r, offset=offset, want=ALL), x, w, r, offset)


@pytest.mark.parametrize("want", [("y",), ("code",), ("h",), ("rstd",), ("y", "rstd"), ("h", "code")])
def test_subsets_are_the_same_bits(gpu_lib, want):
    x, r, w = randn(1, 37, 1160), randn(2, 37, 1160), randn(3, 1160)
    full = binding.norm_act(x, w, residual=r, want=ALL)
    part = binding.norm_act(x, w, residual=r, want=want)
    for name in ALL:
        got = getattr(part, name)
        assert (got is not None) == (name in want)
        if got is not None and name == "code":
            same_code(got, full.code)
        elif got is not None:
            assert torch.equal(got, getattr(full, name))


def test_the_residual_stream_in_place(gpu_lib):
    x, r, w = randn(1, 21, 5376), randn(2, 21, 5376), randn(3, 5376)
    ref = binding.norm_act(x, w, residual=r, want=ALL)
    for target in ("x", "res"):
        x2, r2 = x.clone(), r.clone()
        o = binding.norm_act(x2, w, residual=r2, h=x2 if target == "x" else r2, want=ALL)
        assert torch.equal(o.h, ref.h) and torch.equal(o.y, ref.y) and torch.equal(o.rstd, ref.rstd)
        assert torch.equal(r2 if target == "x" else x2, r if target == "x" else x)


def test_values_that_are_not_finite_stay_in_their_row(gpu_lib):
    x, w = randn(1, 6, 1152), randn(3, 1152)
    clean = binding.norm_act(x, w, want=ALL)
    x[1, 700], x[3, 5] = float("inf"), float("nan")
    x[4] = 0
    o = binding.norm_act(x, w, want=ALL)
    for t in (0, 2, 5):
        assert torch.equal(o.y[t], clean.y[t]) and o.rstd[t] == clean.rstd[t]
    assert o.rstd[1] == 0 and torch.isnan(o.y[1, 700]) and (o.y[1, :700] == 0).all()
    assert torch.isnan(o.rstd[3]) and torch.isnan(o.y[3]).all()
    assert (o.y[4] == 0).all() and abs(o.rstd[4].item() - EPS ** -0.5) < 1e-3
    same_code(o.code, binding.encode_act(o.y))


def test_extreme_magnitudes(gpu_lib):
    """Squares past float32's range on either side."""
    K = 1152
    w = torch.ones(K, device=DEV)
    x = torch.cat([randn(1, 2, K, std=1e30), randn(2, 2, K, std=1e-30)])
    check_forward(binding.norm_act(x, w, 1e-38, want=ALL), x, w, None, 0.0, 1e-38)
    x[0, 0] = 3.3895e38
    w[3] = float("inf")
    o = binding.norm_act(x, w, 1e-38, want=("y",))
    assert torch.isinf(o.y[:, 3]).all() and torch.isfinite(o.y[:, 4:]).all()


def grads_reference(dy, h, a, w, offset, dh):
    n = h.double() * a.double()[:, None]
    g = dy.double() * (offset + w.double())
    mean = (g * n).mean(1, keepdim=True)
    dx = a.double()[:, None] * (g - n * mean) + (0 if dh is None else dh.double())
    K, T = h.shape[1], h.shape[0]
    inner = a.double()[:, None] * (g.abs() + n.abs() * mean.abs()) * 16 * F + \
        a.double()[:, None] * n.abs() * (K + 8) * F * (g * n).abs().mean(1, keepdim=True)
    return dx, (H + 2 * F) * dx.abs() + (1 + H) * inner + TINY, (dy.double() * n).sum(0), (T + 8) * 2 * F * (dy.double() * n).abs().sum(0)


def check_backward(o, dy, h, a, w, offset, dh):
    dx, tx, dw, tw = grads_reference(dy, h, a, w, offset, dh)
    if o.dx is not None:
        assert ((o.dx.double() - dx).abs() <= tx).all()
    if o.dw is not None:
        assert ((o.dw.double() - dw).abs() <= tw + 1e-45).all()


@pytest.mark.parametrize("T,K", SHAPES + [(5000, 128), (1300, 2056)])
@pytest.mark.parametrize("with_dh,f32,offset", [(True, False, 1.0), (False, True, 0.0)])
def test_backward(gpu_lib, T, K, with_dh, f32, offset):
    announce(f"norm backward {T} x {K}")
    dy, h = randn(1, T, K), randn(2, T, K, std=2.0)
    dh = randn(4, T, K) if with_dh else None
    w = randn(3, K, std=0.5, dtype=torch.float32 if f32 else torch.bfloat16)
    a = binding.norm_act(h, w, want=("rstd",)).rstd
    o = binding.norm_backward(dy, h, a, w, offset, dh)
    check_backward(o, dy, h, a, w, offset, dh)
    only = binding.norm_backward(dy, h, a, w, offset, dh, want=("dx",)), binding.norm_backward(dy, h, a, w, offset, dh, want=("dw",))
    assert torch.equal(only[0].dx, o.dx) and torch.equal(only[1].dw, o.dw)
    # dx over the gradient it takes in
    for name in ("dy",) + (("dh",) if with_dh else ()):
        d, r = dy.clone(), None if dh is None else dh.clone()
        got = binding.norm_backward(d, h, a, w, offset, r, dx=d if name == "dy" else r)
        assert torch.equal(got.dx, o.dx) and torch.equal(got.dw, o.dw)


@pytest.mark.parametrize("T,K", [(2, 8), (5, 256), (4, 256), (512, 4096), (513, 4104), (1024, 72), (1025, 72), (1024, 8200), (1100, 17000), (1030, 25000), (40, 32768)])
def test_backward_with_few_and_many_rows(gpu_lib, T, K):
    test_backward(gpu_lib, T, K, True, False, 1.0)


@pytest.mark.parametrize("T,K", [(512, 4096), (513, 4104), (512, 8192), (513, 6152), (3, 16384)])
def test_forward_with_few_and_many_rows(gpu_lib, T, K):
    x, r, w = randn(1, T, K), randn(2, T, K), randn(3, K)
    check_forward(binding.norm_act(x, w, residual=r, want=ALL), x, w, r, 0.0, EPS)


@pytest.mark.parametrize("T,K", [(70000, 512), (36000, 1000), (20000, 2048), (20000, 2056), (9000, 5376), (6000, 8192), (3600, 12000), (2400, 24584)])
def test_rows_past_what_the_caches_hold(gpu_lib, T, K):
    announce(f"norm {T} x {K}")
    x, r, w = randn(1, T, K), randn(2, T, K), randn(3, K)
    o = binding.norm_act(x, w, residual=r, want=ALL)
    check_forward(o, x, w, r, 0.0, EPS)
    g = binding.norm_backward(x, o.h, o.rstd, w, 0.0, r)
    check_backward(g, x, o.h, o.rstd, w, 0.0, r)
    assert torch.equal(binding.norm_backward(x, o.h, o.rstd, w, 0.0, r, dx=r).dx, g.dx)


def test_gradients_against_differences(gpu_lib):
    """<dx, v> and <dw, u> against central differences of the float64 forward.
    With a step of 1e-4 they are off by about 1e-8 of the second derivative's
    scale; dx's own rounding dominates: sum 2^-8 |dx v| with random signs."""
    T, K = 9, 1160
    x, r, w = randn(1, T, K), randn(2, T, K), randn(3, K, std=0.5)
    o = binding.norm_act(x, w, residual=r, offset=1.0, want=("h", "rstd"))
    dy, dh = randn(5, T, K), randn(6, T, K)
    g = binding.norm_backward(dy, o.h, o.rstd, w, 1.0, dh)
    v, u = randn(7, T, K).double(), randn(8, K).double()

    def loss(h, w):
        y = h * (h.square().mean(1, keepdim=True) + EPS) ** -0.5 * (1.0 + w)
        return (y * dy.double()).sum() + (h * dh.double()).sum()
    h, wd, s = o.h.double(), w.double(), 1e-4
    dv = (loss(h + s * v, wd) - loss(h - s * v, wd)) / (2 * s)
    du = (loss(h, wd + s * u) - loss(h, wd - s * u)) / (2 * s)
    assert abs((g.dx.double() * v).sum() - dv) <= 8 * H * (g.dx.double() * v).norm()
    assert abs((g.dw.double() * u).sum() - du) <= 1e-5 * (g.dw.double() * u).abs().sum()


def test_no_tokens(gpu_lib):
    w = randn(3, 64)
    x = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    o = binding.norm_act(x, w, want=ALL)
    assert o.y.shape == (0, 64) and o.rstd.shape == (0,)
    dw = torch.full((64,), 5.0, device=DEV)
    g = binding.norm_backward(x, x, o.rstd, w, dw=dw)
    assert g.dx.shape == (0, 64) and (dw == 0).all()


def test_nothing_else_is_written(gpu_lib):
    """Memory around every output keeps its bytes."""
    T, K = 13, 1160
    x, r, w = randn(1, T, K), randn(2, T, K), randn(3, K)
    pad = 4096
    n = binding.lib().weightless_act_code_bytes(T, K)

    def guarded(nbytes):
        buf = torch.full((nbytes + 2 * pad,), 0x5A, dtype=torch.uint8, device=DEV)
        return buf, buf[pad:pad + nbytes]
    bufs = {"y": guarded(T * K * 2), "h": guarded(T * K * 2), "rstd": guarded(T * 4), "code": guarded(n)}
    out = {"y": bufs["y"][1].view(torch.bfloat16).view(T, K), "h": bufs["h"][1].view(torch.bfloat16).view(T, K),
           "rstd": bufs["rstd"][1].view(torch.float32), "code": binding.ActCode(T, K, buf=bufs["code"][1])}
    o = binding.norm_act(x, w, residual=r, want=ALL, **out)
    dx, dw = guarded(T * K * 2), guarded(K * 4)
    ws = guarded(binding.lib().weightless_norm_backward_workspace_bytes(T, K))
    binding.norm_backward(r, o.h, o.rstd, w, dx=dx[1].view(torch.bfloat16).view(T, K), dw=dw[1].view(torch.float32), ws=ws[1])
    for buf, _ in (*bufs.values(), dx, dw, ws):
        assert (buf[:pad] == 0x5A).all() and (buf[-pad:] == 0x5A).all()


def test_on_another_stream_and_replayed_from_a_graph(gpu_lib):
    T, K = 40, 5376
    x, r, w, dy = randn(1, T, K), randn(2, T, K), randn(3, K), randn(4, T, K)

    def step():
        o = binding.norm_act(x, w, residual=r, want=ALL)
        return o, binding.norm_backward(dy, o.h, o.rstd, w, dh=dy)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, d = step()
    for seed in (11, 12, 13):
        x.copy_(randn(seed, T, K))
        dy.copy_(randn(seed + 50, T, K))
        g.replay()
        torch.cuda.synchronize()
        eo, ed = step()
        assert torch.equal(o.y, eo.y) and torch.equal(o.h, eo.h) and torch.equal(d.dx, ed.dx) and torch.equal(d.dw, ed.dw)
        same_code(o.code, eo.code)


def test_offsets_past_2_to_the_31(gpu_lib):
    T, K = 1 << 20, 2056
    announce(f"norm {T} x {K}")
    x = torch.zeros(T, K, dtype=torch.bfloat16, device=DEV)
    rows = torch.tensor([0, 5, 600000, 1044480, T - 1], device=DEV)
    x[rows] = randn(1, 5, K)
    w = randn(3, K)
    o = binding.norm_act(x, w, want=("y", "code", "rstd"))
    part = binding.norm_act(x[rows].contiguous(), w, want=("y", "code", "rstd"))
    assert torch.equal(o.y[rows], part.y) and torch.equal(o.rstd[rows], part.rstd)
    assert torch.equal(o.code.codes.view(torch.uint8)[rows], part.code.codes.view(torch.uint8))
    assert torch.equal(o.code.scales[rows], part.code.scales)
    g = binding.norm_backward(o.y, x, o.rstd, w)
    want = binding.norm_backward(part.y, x[rows].contiguous(), part.rstd, w)
    assert torch.equal(g.dx[rows], want.dx) and torch.allclose(g.dw, want.dw, rtol=1e-4, atol=1e-4)
