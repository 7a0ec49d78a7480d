"""GPU: gradients of the adapters, from an 8-bit checkpoint.

Reference in float64 at the checkpoint's own values.  Tolerances, derived before
the first run, per element: a bf16 rounding 2^-8 of the value, a float32 sum of n
terms n * 2^-23 of the sum of their magnitudes; with c the scale, Ta the slot's
tokens and |.| elementwise

  z   e_z = c K 2^-23 |V^T| |X| + 2^-16 |z|       g   e_g = c N 2^-23 |U^T| |dy| + 2^-16 |g|
  dU  2^-8 |dU| + |dy|^T e_z + (2 Ta + 8) 2^-23 |dy|^T |z|
  dV  2^-8 |dV| + e_g^T |X| + (2 Ta + 8) 2^-23 |g|^T |X|
  dx  2^-8 |dx| + sum over children e_g |V^T| + (2 children r + 8) 2^-23 |g| |V^T|

and, one rounding each, the error's norm within 2^-8 of the result's."""
import sys

import pytest
import torch

from test_adapters_gpu import DEV, F, H, check_add, each_slot, make_pool, mixed_index, randn, slots_of
from weight_shared_rank_amd import binding

pytestmark = pytest.mark.gpu
TINY = 2.0 ** -133
ALL = ("dx", "du", "dv")


def announce(msg):
    sys.__stderr__.write(f"[gpu] {msg}\n")
    sys.__stderr__.flush()


def reference(p, X, dy, index, base):
    """(dx, du, dv) in float64 and their tolerances before the final rounding."""
    ref = [base.double(), torch.zeros(p.u.shape, dtype=torch.float64, device=DEV), torch.zeros(p.vt.shape, dtype=torch.float64, device=DEV)]
    tol = [torch.zeros_like(t) for t in ref]
    for a, at, kids in each_slot(p, index):
        c, x = float(p.scale[a]), X[at]
        n2 = (2 * len(at) + 8) * F
        for i, (n0, n, V, U) in enumerate(kids):
            r, d = V.shape[0], dy[at, n0:n0 + n].double()
            dt, Vt = d.t().contiguous(), V.t().contiguous()
            z, g = c * (x @ Vt), c * (d @ U)
            ez = c * p.K * F * (x.abs() @ Vt.abs()) + H * H * z.abs()
            eg = c * n * F * (d.abs() @ U.abs()) + H * H * g.abs()
            ref[0][at] += g @ V
            tol[0][at] += (eg + (2 * len(kids) * r + 8) * F * g.abs()) @ V.abs()
            ref[1][a, n0:n0 + n, :r] = dt @ z
            tol[1][a, n0:n0 + n, :r] = dt.abs() @ (ez + n2 * z.abs())
            gt, row = g.t().contiguous(), i * p.room
            ref[2][a, row:row + r] = gt @ x
            tol[2][a, row:row + r] = (eg + n2 * g.abs()).t().contiguous() @ x.abs()
    return ref, tol


def check(p, code, dy, index, base, g):
    ref, tol = reference(p, code.expand().double(), dy, index, base)
    for name, r, t in zip(ALL, ref, tol):
        got = getattr(g, name)
        if got is None:
            continue
        err = (got.double() - r).abs()
        bound = t + H * r.abs() + TINY
        bad = torch.nonzero(~(err <= bound))
        assert len(bad) == 0, (name, bad[:4].tolist(), [(got[tuple(b)].item(), r[tuple(b)].item()) for b in bad[:4]])
        if r.numel() >= 1024:
            assert err.norm() <= H * r.norm() + TINY, name
    if g.dx is not None:
        none = slots_of(p, index) < 0
        assert torch.equal(g.dx[none].view(torch.int16), base[none].view(torch.int16))


CASES = [  # T, rows, K, r, n
    (1, (1024, 256, 256), 1152, 16, 8), (2, (64,), 64, 16, 1), (3, (1,), 8, 16, 2), (31, (1001,), 712, 48, 3),
    (32, (40, 7, 300), 136, 32, 5), (33, (72, 72), 1160, 64, 2), (77, (513,), 2056, 16, 64), (100, (264,), 520, 256, 4),
    (255, (130,), 64, 128, 300), (257, (130, 66, 2), 320, 112, 6), (333, (1001,), 1160, 32, 5),
    (1000, (256,), 128, 16, 2000), (2500, (96, 96), 256, 64, 12), (9000, (40,), 64, 16, 30), (700, (136, 136, 136), 264, 256, 2)]


@pytest.mark.parametrize("T,rows,K,r,n", CASES)
@pytest.mark.parametrize("ranked", [False, True])
def test_gradients(gpu_lib, T, rows, K, r, n, ranked):
    announce(f"adapters backward T={T} rows={rows} K={K} r={r} n={n} ranked={ranked}")
    ranks = [(r, r // 2, 1, 0, r + 5, -3, max(1, r - 7))[(3 * i) % 7] for i in range(n)] if ranked else None
    p = make_pool(n, r, K, rows, ranks, dirty=ranked)
    code, dy, base = binding.encode_act(randn(7, T, K)), randn(8, T, sum(rows), std=T ** -0.5), randn(10, T, K, std=T ** -0.5)
    index = mixed_index(T, n, 9)
    g = p.backward(code, dy, index, base)
    check(p, code, dy, index, base, g)
    for want in (("dx",), ("du",), ("dv",)):
        one = p.backward(code, dy, index, base if want == ("dx",) else None, want=want)
        assert torch.equal(getattr(one, want[0]), getattr(g, want[0]))
    b2 = base.clone()
    assert torch.equal(p.backward(code, dy, index, b2, want=("dx",), dx=b2).dx, g.dx)


SPLITS = [  # few slots and many tokens; many column tiles; long contractions of z, of g, of both
    (2100, (70, 40), 40, 16, 1), (4500, (130,), 200, 64, 2), (6200, (65, 1), 72, 32, 3), (300, (1001,), 8, 32, 256),
    (300, (520, 130), 264, 16, 260), (200, (700,), 72, 128, 200), (70, (2100, 30), 2056, 32, 3), (40, (1100,), 1160, 48, 2),
    (130, (4100,), 64, 16, 4), (130, (100,), 4104, 64, 4), (250, (1001,), 8, 32, 256), (120, (520, 130), 264, 16, 260),
    (8, (2100, 30), 2056, 32, 3), (12, (4100,), 64, 16, 4), (100, (70,), 2600, 16, 3),
    (300, (1001,), 520, 32, 256), (300, (700,), 520, 128, 200)]


@pytest.mark.parametrize("T,rows,K,r,n", SPLITS)
@pytest.mark.parametrize("ranked", [False, True])
def test_gradients_of_split_sums(gpu_lib, T, rows, K, r, n, ranked):
    test_gradients(gpu_lib, T, rows, K, r, n, ranked)


@pytest.mark.parametrize("T,rows,K,r,n", [(2100, (70, 40), 40, 16, 9), (3000, (200,), 264, 48, 5), (2600, (66, 1, 5), 72, 32, 4), (1000, (1001,), 264, 32, 300),
                                          (900, (700,), 520, 128, 200), (1300, (300, 300), 520, 16, 300), (5000, (40,), 24, 16, 600)])
@pytest.mark.parametrize("uneven", ["one", "half", "last"])
def test_tokens_spread_unevenly(gpu_lib, T, rows, K, r, n, uneven):
    """Slots whose tokens are cut into parts beside slots that are not."""
    announce(f"adapters backward T={T} rows={rows} K={K} r={r} n={n} {uneven}")
    p = make_pool(n, r, K, rows, ranks=[(r, 3, r - 1)[i % 3] for i in range(n)])
    index = mixed_index(T, n, 3)
    index[torch.arange(T, device=DEV) % 8 < {"one": 8, "half": 5, "last": 7}[uneven]] = n - 1 if uneven == "last" else n // 2
    code, dy, base = binding.encode_act(randn(7, T, K)), randn(8, T, sum(rows), std=T ** -0.5), randn(10, T, K, std=T ** -0.5)
    g = p.backward(code, dy, index, base)
    check(p, code, dy, index, base, g)
    for want in ("du", "dv"):
        assert torch.equal(getattr(p.backward(code, dy, index, want=(want,)), want), getattr(g, want))


def test_as_many_tokens_and_slots_as_there_can_be(gpu_lib):
    T, n = 1 << 20, 4096
    announce(f"adapters T={T} n={n}")
    p = make_pool(n, 16, 8, (1, 3))
    x, dy, base, index = randn(1, T, 8), randn(2, T, 4, std=0.1), randn(3, T, 8), mixed_index(T, n, 4)
    code = binding.encode_act(x)
    check(p, code, dy, index, base, p.backward(code, dy, index, base))
    check_add(p, x, index, dy, p.add(x, index, dy))


def test_gradients_past_a_rank_are_zero_for_an_infinite_dy(gpu_lib):
    T = 70
    p = make_pool(2, 48, 136, (70,), ranks=[5, 33])
    dy = randn(2, T, 70)
    dy[3, 7], dy[40] = float("inf"), float("nan")
    g = p.backward(binding.encode_act(randn(1, T, 136)), dy, mixed_index(T, 2, 3), want=("du", "dv"))
    for a, r in enumerate(p.rank.tolist()):
        assert (g.du[a, :, r:] == 0).all() and (g.dv[a, r:] == 0).all()


@pytest.mark.parametrize("T", [1, 32, 65, 700])
@pytest.mark.parametrize("kind", ["none", "one", "last", "sorted"])
def test_index_patterns(gpu_lib, T, kind):
    p = make_pool(6, 32, 264, (200, 56))
    index = {"none": torch.full((T,), -1), "one": torch.full((T,), 2), "last": torch.full((T,), 5),
             "sorted": torch.arange(T) * 7 // T - 1}[kind].to(torch.int32).to(DEV)
    code, dy, base = binding.encode_act(randn(1, T, 264)), randn(2, T, 256), randn(3, T, 264)
    g = p.backward(code, dy, index, base)
    check(p, code, dy, index, base, g)
    if kind == "none":
        assert (g.du == 0).all() and (g.dv == 0).all()


def test_gradients_past_a_rank_are_zero_whatever_lies_there(gpu_lib):
    T = 120
    p = make_pool(5, 48, 136, (70, 33), ranks=[1, 7, 16, 31, 0])
    for a, r in enumerate(p.rank.tolist()):
        p.vt.view(5, 2, 48, 136)[a, :, r:] = float("nan")
        p.u[a, :, r:] = float("inf")
    code, dy, base, index = binding.encode_act(randn(1, T, 136)), randn(2, T, 103), randn(3, T, 136), mixed_index(T, 5, 3)
    g = p.backward(code, dy, index, base)
    check(p, code, dy, index, base, g)
    for a, r in enumerate(p.rank.tolist()):
        assert (g.du[a, :, r:] == 0).all() and (g.dv.view(5, 2, 48, 136)[a, :, r:] == 0).all()


def test_not_finite_stays_where_it_is(gpu_lib):
    T = 90
    p = make_pool(4, 32, 136, (100, 60))
    x, dy, base, index = randn(1, T, 136), randn(2, T, 160), randn(3, T, 136), (torch.arange(T) % 5).to(torch.int32).to(DEV)
    clean = p.backward(binding.encode_act(x), dy, index, base)
    x[6, 3] = float("nan")        # slot 1
    dy[12, 30] = float("inf")     # slot 2
    dy[4], x[4] = float("nan"), float("nan")   # no adapter
    g = p.backward(binding.encode_act(x), dy, index, base)
    keep = torch.ones(T, dtype=torch.bool, device=DEV)
    keep[12] = False
    assert torch.equal(g.dx[keep].view(torch.int16), clean.dx[keep].view(torch.int16)) and not torch.isfinite(g.dx[12]).any()
    for a in (0, 3):
        assert torch.equal(g.du[a], clean.du[a]) and torch.equal(g.dv[a], clean.dv[a])
    assert torch.isnan(g.du[1]).all() and torch.isnan(g.dv[1, :, 3]).all() and torch.equal(g.dv[1, :, 4:], clean.dv[1, :, 4:])
    assert not torch.isfinite(g.du[2, 30]).any() and torch.equal(g.du[2, 31:], clean.du[2, 31:])
    assert not torch.isfinite(g.dv[2, :32]).any() and torch.equal(g.dv[2, 32:], clean.dv[2, 32:])


def test_gradients_against_differences(gpu_lib):
    """<gradient, direction> against central differences of the float64 forward,
    which is bilinear in U and V: exact but for cancellation.  What is left is the
    gradients' own rounding, 2^-8 of each term with random signs."""
    T, K, rows = 60, 264, (100, 36)
    p = make_pool(3, 16, K, rows)
    code, dy, base, index = binding.encode_act(randn(1, T, K)), randn(2, T, 136), randn(3, T, K), mixed_index(T, 3, 4)
    g = p.backward(code, dy, index, base)
    X = code.expand().double()
    of = slots_of(p, index)
    on = of >= 0

    def loss(X, vt, u):
        total = 0.0
        for a in range(3):
            at, n0 = of == a, 0
            for c, n in enumerate(rows):
                z = float(p.scale[a]) * (X[at] @ vt[a, c * 16:(c + 1) * 16].t().contiguous())
                total = total + ((z @ u[a, n0:n0 + n].t().contiguous()) * dy[at, n0:n0 + n].double()).sum()
                n0 += n
        return total
    vt, u, s = p.vt.double(), p.u.double(), 1e-3
    dirs = [randn(5, T, K).double(), randn(6, *vt.shape).double(), randn(7, *u.shape).double()]
    own = [torch.where(on[:, None], g.dx.double() - base.double(), torch.zeros_like(X)), g.dv.double(), g.du.double()]
    noise = [H * g.dx.double() * dirs[0], H * own[1] * dirs[1], H * own[2] * dirs[2]]
    for i, d in enumerate(dirs):
        args = [X, vt, u]
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + s * d, args[i] - s * d
        diff = (loss(*up) - loss(*down)) / (2 * s)
        assert abs((own[i] * d).sum() - diff) <= 8 * noise[i].norm(), i


def test_no_tokens(gpu_lib):
    p = make_pool(3, 16, 64, (40,))
    code = binding.ActCode(0, 64)
    e = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    du, dv = torch.ones_like(p.u), torch.ones_like(p.vt)
    index, dy = torch.empty(0, dtype=torch.int32, device=DEV), torch.empty(0, 40, dtype=torch.bfloat16, device=DEV)
    g = p.backward(code, dy, index, e, du=du, dv=dv)
    assert g.dx.shape == (0, 64) and (du == 0).all() and (dv == 0).all()
    assert p.backward(code, dy, index, e, want=("dx",)).dx.shape == (0, 64)
    assert p.add(e, index, dy).shape == (0, 40)


def test_nothing_else_is_written(gpu_lib):
    T, K, rows = 77, 136, (37, 20)
    p = make_pool(3, 32, K, rows)
    code, dy, base, index = binding.encode_act(randn(1, T, K)), randn(2, T, 57), randn(3, T, K), mixed_index(T, 3, 4)
    pad = 4096

    def guarded(shape):
        n = 2
        for v in shape:
            n *= v
        buf = torch.full((n + 2 * pad,), 0x5A, dtype=torch.uint8, device=DEV)
        return buf, buf[pad:-pad].view(torch.bfloat16).view(shape)
    bufs = {"dx": guarded((T, K)), "du": guarded(tuple(p.u.shape)), "dv": guarded(tuple(p.vt.shape))}
    ws = torch.full((p.backward_workspace_bytes(T) + 2 * pad,), 0x5A, dtype=torch.uint8, device=DEV)
    g = p.backward(code, dy, index, base, ws=ws[pad:-pad], **{k: v for k, (_, v) in bufs.items()})
    check(p, code, dy, index, base, g)
    for b in (ws, *(b for b, _ in bufs.values())):
        assert (b[:pad] == 0x5A).all() and (b[-pad:] == 0x5A).all()


def test_replayed_from_a_graph_and_on_other_streams(gpu_lib):
    T, K, rows = 300, 264, (72, 40)
    p = make_pool(8, 16, K, rows, ranks=[16, 4, 0, 9, 16, 16, 1, 12])
    code, dy, base, index = binding.encode_act(randn(1, T, K)), randn(2, T, 112), randn(3, T, K), mixed_index(T, 8, 3)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        p.backward(code, dy, index, base)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g = p.backward(code, dy, index, base)
    for seed in (4, 5, 6, 7):
        index.copy_(mixed_index(T, 8, seed))
        dy.copy_(randn(seed, T, 112))
        graph.replay()
        torch.cuda.synchronize()
        eager = p.backward(code, dy, index, base)
        assert all(torch.equal(getattr(g, n), getattr(eager, n)) for n in ALL)
        check(p, code, dy, index, base, g)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = [[p.backward(code, dy, index, base, stream=st) for _ in range(8)] for st in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(getattr(x, n), getattr(eager, n)) for xs in got for x in xs for n in ALL)


def test_few_tokens_replayed_with_other_slots_and_ranks(gpu_lib):
    T, K, rows, n = 40, 264, (72, 40), 6
    p = make_pool(n, 32, K, rows, ranks=[32] * n)
    code, dy, base, index = binding.encode_act(randn(1, T, K)), randn(2, T, 112), randn(3, T, K), mixed_index(T, n, 3)
    p.backward(code, dy, index, base)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g = p.backward(code, dy, index, base)
    for seed in (4, 5, 6, 7):
        index.copy_(mixed_index(T, n, seed) if seed < 7 else torch.full((T,), 2, dtype=torch.int32))
        p.rank.copy_(torch.tensor([32, 0, 7, 16, 31, 17], dtype=torch.int32).roll(seed))
        graph.replay()
        torch.cuda.synchronize()
        check(p, code, dy, index, base, g)
        eager = p.backward(code, dy, index, base)
        assert all(torch.equal(getattr(g, name), getattr(eager, name)) for name in ALL)


def test_many_tokens_replayed_between_one_slot_and_many(gpu_lib):
    T, K, rows, n = 2300, 136, (72,), 9
    p = make_pool(n, 16, K, rows)
    code, dy, base, index = binding.encode_act(randn(1, T, K)), randn(2, T, 72, std=0.1), randn(3, T, K), mixed_index(T, n, 3)
    p.backward(code, dy, index, base)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g = p.backward(code, dy, index, base)
    for i in range(5):
        index.copy_(torch.full((T,), i, dtype=torch.int32) if i % 2 else mixed_index(T, n, i))
        graph.replay()
        torch.cuda.synchronize()
        check(p, code, dy, index, base, g)
        eager = p.backward(code, dy, index, base)
        assert all(torch.equal(getattr(g, name), getattr(eager, name)) for name in ALL)


def test_binding_refusals(gpu_lib):
    p = make_pool(2, 16, 64, (32,))
    code, dy, base, index = binding.encode_act(randn(1, 4, 64)), randn(2, 4, 32), randn(3, 4, 64), torch.zeros(4, dtype=torch.int32, device=DEV)
    for bad in (dict(x=randn(1, 4, 64)), dict(x=binding.encode_act(randn(1, 4, 72))), dict(dy=randn(1, 4, 40)), dict(index=index.long()),
                dict(base=None), dict(base=base, want=("du",)), dict(base=base.float()), dict(want=()), dict(want=("dw",)), dict(base=None, want=("du",), dv=p.vt),
                dict(du=p.u.float()), dict(dv=p.vt[:1]), dict(du=p.u), dict(dx=randn(1, 4, 72))):
        with pytest.raises(binding.WlError):
            p.backward(**{**dict(x=code, dy=dy, index=index, base=base), **bad})


def test_offsets_past_2_to_the_31(gpu_lib):
    T, N, K = 66000, 33000, 64
    announce(f"adapters backward T={T} N={N}")
    p = make_pool(3, 16, K, (N,))
    dy = torch.zeros(T, N, dtype=torch.bfloat16, device=DEV)
    rows = torch.tensor([0, 1, 40000, 65070, T - 2, T - 1], device=DEV)
    dy[rows] = randn(2, 6, N)
    x, index = randn(1, T, K), mixed_index(T, 3, 2)
    index[rows] = torch.tensor([0, 1, 2, 0, 1, 2], dtype=torch.int32, device=DEV)
    base = torch.zeros(T, K, dtype=torch.bfloat16, device=DEV)
    g = p.backward(binding.encode_act(x), dy, index, base)
    part = binding.encode_act(x[rows].contiguous())
    ref, tol = reference(p, part.expand().double(), dy[rows], index[rows], base[rows])
    for got, r, t in ((g.dx[rows], ref[0], tol[0]), (g.du, ref[1], tol[1]), (g.dv, ref[2], tol[2])):
        assert ((got.double() - r).abs() <= t + H * r.abs() + TINY).all()
