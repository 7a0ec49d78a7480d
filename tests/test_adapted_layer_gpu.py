"""GPU: the pieces together, as a serving step and a training step use them: norm
with the residual's addition -> the bf16 input and its 8-bit checkpoint -> the
stacked projection with the adapters of many requests -> gradients of both -> the
norm's gradients.

The reference runs the same chain in float64 at the checkpoint's values (the
backward pass's own X).  Bounds, derived before the first run, on norms over the
whole output, a bf16 rounding taking 2^-8: y has the shared projection's rounding
and the adapters' (2); what reaches the norm has the shared dx's two and the
adapters' one (3, on the larger of what is added up), which the norm's backward
multiplies by at most m = max a |w| before its own."""
import pytest
import torch

from test_adapters_gpu import DEV, each_slot, make_pool, mixed_index, randn
from weight_shared_rank_amd import binding

pytestmark = pytest.mark.gpu
H, EPS = 2.0 ** -8, 1e-6
K, ROWS, FAMS = 520, (264, 72, 72), ("q", "k", "v")


def make_bundle():
    spec = binding.make_spec(1, 1, {(0, f): (n, K) for f, n in zip(FAMS, ROWS)}, {(0, f): 24 for f in FAMS})
    w0, s = [randn(40 + i, n, K, std=K ** -0.5) for i, n in enumerate(ROWS)], [1 + 0.1 * randn(50 + i, n, dtype=torch.float32) for i, n in enumerate(ROWS)]
    u, v = [randn(60 + i, n, 24, std=0.1) for i, n in enumerate(ROWS)], [randn(70 + i, K, 24, std=0.1) for i in range(3)]
    src = [x for i, f in enumerate(FAMS) for x in (("w0", 0, 0, f, w0[i]), ("s", 0, 0, f, s[i]), ("u", 0, 0, f, u[i]), ("v", 0, 0, f, v[i]))]
    dense = torch.cat([s[i].double()[:, None] * w0[i].double() + u[i].double() @ v[i].double().t().contiguous() for i in range(3)])
    return binding.ThetaBundle(spec, src), dense


def layer(b, p, x, res, w, index):
    o = binding.norm_act(x, w, EPS, residual=res, offset=1.0, want=("y", "code", "h", "rstd"))
    y = b.stacked(0, "qkv", o.y)
    p.add(o.y, index, y, y=y)
    return o, y


def backward(b, p, o, w, dy, dh, index):
    g = b.stacked_backward(0, "qkv", o.code, dy)
    a = p.backward(o.code, dy, index, g.dx, dx=g.dx)
    return g, a, binding.norm_backward(a.dx, o.h, o.rstd, w, 1.0, dh=dh, dx=a.dx)


@pytest.mark.parametrize("T", [1, 9, 48, 400])
def test_forward_and_backward(gpu_lib, T):
    b, dense = make_bundle()
    p = make_pool(4, 16, K, ROWS, ranks=[16, 5, 0, 11])
    x, res, w, index = randn(1, T, K), randn(2, T, K), randn(3, K, std=0.3), mixed_index(T, 4, 5, wild=T > 2)
    o, y = layer(b, p, x, res, w, index)

    h = (x.float() + res.float()).to(torch.bfloat16).double()
    a = (h.square().mean(1, keepdim=True) + EPS) ** -0.5
    n = h * a
    assert ((o.y.double() - n * (1 + w.double())).norm() <= 1.01 * H * (n * (1 + w.double())).norm())

    def project(X, low):
        out = X @ dense.t().contiguous()
        for _, at, kids in each_slot(p, index):
            for n0, m, V, U in kids:
                out[at, n0:n0 + m] += low * ((X[at] @ V.t().contiguous()) @ U.t().contiguous()) * p.scale[index[at].long()].double()[:, None]
        return out
    ref = project(o.y.double(), 1.0)
    assert (y.double() - ref).norm() <= 2 * H * max(ref.norm(), project(o.y.double(), 0.0).norm())

    dy, dh = randn(6, T, sum(ROWS), std=T ** -0.5), randn(7, T, K, std=T ** -0.5)
    g, ad, nb = backward(b, p, o, w, dy, dh, index)
    dshared = dy.double() @ dense
    din = dshared.clone()
    for _, at, kids in each_slot(p, index):
        for n0, m, V, U in kids:
            din[at] += p.scale[index[at].long()].double()[:, None] * ((dy[at, n0:n0 + m].double() @ U) @ V)
    gw = din * (1 + w.double())
    want = a * (gw - n * (gw * n).mean(1, keepdim=True)) + dh.double()
    m = (a.max() * (1 + w.double()).abs().max()).item()
    assert (nb.dx.double() - want).norm() <= H * want.norm() + m * 3 * H * max(din.norm(), dshared.norm())
    dw = (din * n).sum(0)
    assert (nb.dw.double() - dw).norm() <= 4 * H * (din.abs() * n.abs()).norm() * max(1.0, T ** 0.5)
    X = o.code.expand().double()
    for s, at, kids in each_slot(p, index):
        c = float(p.scale[s])
        for i, (n0, rows, V, U) in enumerate(kids):
            d = c * dy[at, n0:n0 + rows].double()
            grad = d.t().contiguous() @ X[at]
            for got, ref in ((ad.du[s, n0:n0 + rows, :U.shape[1]], grad @ V.t().contiguous()), (ad.dv[s, i * 16:i * 16 + V.shape[0]], U.t().contiguous() @ grad)):
                assert (got.double() - ref).norm() <= 1.01 * H * ref.norm()


def test_a_decode_step_replayed_with_other_requests(gpu_lib):
    """One captured step; the requests' adapters and the hidden states change between replays."""
    b, _ = make_bundle()
    p = make_pool(6, 16, K, ROWS)
    T, w = 8, randn(3, K, std=0.3)
    x, res, index = randn(1, T, K), randn(2, T, K), mixed_index(T, 6, 5)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer(b, p, x, res, w, index)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, y = layer(b, p, x, res, w, index)
    for seed in (11, 12, 13):
        x.copy_(randn(seed, T, K))
        index.copy_(mixed_index(T, 6, seed))
        graph.replay()
        torch.cuda.synchronize()
        eo, ey = layer(b, p, x, res, w, index)
        assert torch.equal(y, ey) and torch.equal(o.h, eo.h) and torch.equal(o.y, eo.y)


def test_a_captured_training_step_beside_an_eager_one(gpu_lib):
    b, _ = make_bundle()
    p = make_pool(3, 16, K, ROWS)
    T, w = 70, randn(3, K, std=0.3)
    x, res, index, dy, dh = randn(1, T, K), randn(2, T, K), mixed_index(T, 3, 5), randn(6, T, sum(ROWS)), randn(7, T, K)

    def step():
        o, y = layer(b, p, x, res, w, index)
        return y, *backward(b, p, o, w, dy, dh, index)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, g, ad, nb = step()
    for seed in (21, 22, 23):
        dy.copy_(randn(seed, T, sum(ROWS)))
        index.copy_(mixed_index(T, 3, seed))
        graph.replay()
        torch.cuda.synchronize()
        ey, eg, ead, enb = step()
        assert torch.equal(y, ey) and torch.equal(nb.dx, enb.dx) and torch.equal(nb.dw, enb.dw)
        assert torch.equal(ad.du, ead.du) and torch.equal(ad.dv, ead.dv) and torch.equal(g.ds, eg.ds)
