"""GPU: low-rank adapters of many requests beside one projection.

Reference in float64, token by token's slot.  Tolerance, derived before the first
run, per element: a bf16 rounding 2^-8 of the value, a float32 sum of n terms
n * 2^-23 of the sum of their magnitudes; with c the scale and |.| elementwise

  z   e_z = c K 2^-23 |V^T| |x| + 2^-16 |c z|      (float32 sums; a pair of bf16)
  y   2^-8 |y| + |U| e_z + (2 r + 8) 2^-23 |U| |c z|
"""
import sys

import pytest
import torch

from weight_shared_rank_amd import binding

pytestmark = pytest.mark.gpu
DEV = "cuda"
H, F = 2.0 ** -8, 2.0 ** -23


def announce(msg):
    sys.__stderr__.write(f"[gpu] {msg}\n")
    sys.__stderr__.flush()


def randn(seed, *shape, std=1.0, dtype=torch.bfloat16):
    g = torch.Generator("cpu").manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype).to(DEV)


def make_pool(n, r, K, rows, ranks=None, seed=0, dirty=False):
    """ranks: per slot (None: no rank tensor).  dirty: NaN where nothing may be read."""
    kids = len(rows)
    vt, u = randn(seed + 1, n, kids * r, K, std=K ** -0.5), randn(seed + 2, n, sum(rows), r, std=0.3)
    scale = (0.5 + torch.rand(n, generator=torch.Generator("cpu").manual_seed(seed + 3))).to(DEV)
    rank = None
    if ranks is not None:
        rank = torch.tensor(ranks, dtype=torch.int32, device=DEV)
        live = rank.clamp(0, r)[:, None]
        j = torch.arange(r, device=DEV)[None]
        used = -(-live // 16) * 16
        fill = float("nan") if dirty else 0.0
        v4 = vt.view(n, kids, r, K)
        v4[(j >= live)[:, None, :].expand(n, kids, r)] = 0
        u.masked_fill_((j >= live)[:, None, :], 0)
        v4[(j >= used)[:, None, :].expand(n, kids, r)] = fill
        u.masked_fill_((j >= used)[:, None, :], fill)
    return binding.AdapterPool(vt, u, scale, rows, rank=rank)


def slots_of(p, index):
    """The slot of each token, -1 for none."""
    ok = (index >= 0) & (index < p.slots)
    s = torch.where(ok, index, torch.zeros_like(index)).long()
    if p.rank is not None:
        ok &= p.rank[s] > 0
    return torch.where(ok, s, torch.full_like(s, -1))


def each_slot(p, index):
    """(slot, its tokens, per child (first column, V^T, U) in float64)."""
    of = slots_of(p, index)
    for a in sorted(set(of.tolist()) - {-1}):
        r = p.room if p.rank is None else min(int(p.rank[a]), p.room)
        at, kids = 0, []
        for c, n in enumerate(p.out_dims):
            kids.append((at, n, p.vt[a, c * p.room:c * p.room + r].double(), p.u[a, at:at + n, :r].double()))
            at += n
        yield a, torch.nonzero(of == a)[:, 0], kids


def check_add(p, x, index, base, y):
    ref, tol = base.double(), torch.zeros(base.shape, dtype=torch.float64, device=DEV)
    for a, at, kids in each_slot(p, index):
        c, X = float(p.scale[a]), x[at].double()
        for n0, n, V, U in kids:
            z = c * (X @ V.t().contiguous())
            ez = c * p.K * F * (X.abs() @ V.abs().t().contiguous()) + H * H * z.abs()
            Ut = U.t().contiguous()
            ref[at, n0:n0 + n] += z @ Ut
            tol[at, n0:n0 + n] = (ez + (2 * V.shape[0] + 8) * F * z.abs()) @ Ut.abs()
    tol += H * ref.abs()
    err = (y.double() - ref).abs()
    assert (err <= tol).all(), (err - tol).max()
    if ref.numel() >= 1024:
        assert err.norm() <= H * ref.norm()
    none = slots_of(p, index) < 0
    assert torch.equal(y[none].view(torch.int16), base[none].view(torch.int16))


def mixed_index(T, n, seed, wild=True):
    g = torch.Generator("cpu").manual_seed(seed)
    idx = torch.randint(0, n, (T,), generator=g, dtype=torch.int32)
    if wild and T > 2:
        bad = torch.tensor([-1, n, -2 ** 31, 2 ** 31 - 1, n + 7], dtype=torch.int32)
        at = torch.randperm(T, generator=g)[:max(1, T // 7)]
        idx[at] = bad[torch.arange(len(at)) % 5]
    return idx.to(DEV)


CASES = [  # T, rows, K, r, n
    (1, (1024, 256, 256), 1152, 16, 8), (2, (64,), 64, 16, 1), (3, (1,), 8, 16, 2), (15, (1001,), 712, 48, 3),
    (16, (40, 7, 300), 136, 32, 5), (17, (72, 72), 1160, 64, 2), (64, (513,), 2056, 16, 64), (100, (264,), 520, 256, 4),
    (255, (130,), 64, 128, 300), (256, (48, 48), 72, 80, 3), (257, (130, 66, 2), 320, 112, 6), (333, (1001,), 1160, 32, 5),
    (1000, (256,), 128, 16, 4096), (2500, (96, 96), 256, 64, 12), (9000, (40,), 64, 16, 700)]


@pytest.mark.parametrize("T,rows,K,r,n", CASES)
@pytest.mark.parametrize("ranked", [False, True])
def test_add(gpu_lib, T, rows, K, r, n, ranked):
    announce(f"adapters T={T} rows={rows} K={K} r={r} n={n} ranked={ranked}")
    ranks = [(r, r // 2, 1, 0, r + 5, -3, max(1, r - 7))[(3 * i) % 7] for i in range(n)] if ranked else None
    p = make_pool(n, r, K, rows, ranks, dirty=ranked)
    x, base, index = randn(7, T, K), randn(8, T, sum(rows)), mixed_index(T, n, 9)
    y = p.add(x, index, base)
    check_add(p, x, index, base, y)
    again = base.clone()
    assert p.add(x, index, again, y=again) is again and torch.equal(again.view(torch.int16), y.view(torch.int16))


LONG = [  # enough rows for whole tiles of tokens: K cut into slices, and short
    (2100, (4100,), 1032, 16, 3), (1100, (3000, 4700), 696, 64, 3), (600, (14000,), 520, 128, 2), (1100, (8200,), 520, 256, 2),
    (2100, (4100,), 64, 32, 3), (1100, (8200,), 72, 48, 2), (700, (12000,), 8, 112, 2), (1100, (8200,), 136, 176, 2), (600, (264,), 264, 16, 600), (512, (40, 72), 136, 16, 3), (513, (40, 72), 136, 16, 3),
    (512, (300,), 264, 48, 40), (1, (264,), 8192, 256, 2), (1, (264,), 4096, 64, 2), (60, (264,), 8192, 64, 5), (40, (30000,), 264, 32, 30),
    (40, (30000,), 264, 16, 40), (300, (29999, 9), 264, 16, 40)]


@pytest.mark.parametrize("T,rows,K,r,n", LONG)
@pytest.mark.parametrize("ranked", [False, True])
def test_add_long(gpu_lib, T, rows, K, r, n, ranked):
    test_add(gpu_lib, T, rows, K, r, n, ranked)


TILES_OF_64 = [  # long contractions, high ranks, and outputs large enough for tiles of 64 tokens
    (300, (64,), 40000, 16, 1), (40, (72,), 16384, 32, 2), (1600, (30000,), 64, 16, 1), (1600, (30000,), 72, 32, 1),
    (1600, (30000,), 1032, 16, 1), (1600, (30000,), 1160, 32, 1), (1000, (30000,), 264, 64, 2), (1000, (30000,), 520, 64, 2),
    (1000, (20000,), 264, 128, 2), (1100, (12000,), 264, 256, 2), (60, (264,), 4096, 128, 5), (900, (9000, 300), 2056, 96, 3),
    (450, (4104,), 4096, 48, 2)]


@pytest.mark.parametrize("T,rows,K,r,n", TILES_OF_64)
@pytest.mark.parametrize("ranked", [False, True])
def test_add_in_tiles_of_64(gpu_lib, T, rows, K, r, n, ranked):
    test_add(gpu_lib, T, rows, K, r, n, ranked)


@pytest.mark.parametrize("T", [1, 16, 40, 256, 257, 700])
@pytest.mark.parametrize("kind", ["none", "one", "last", "sorted"])
def test_index_patterns(gpu_lib, T, kind):
    p = make_pool(6, 32, 264, (200, 56))
    index = {"none": torch.full((T,), -1), "one": torch.full((T,), 2), "last": torch.full((T,), 5),
             "sorted": torch.arange(T) * 7 // T - 1}[kind].to(torch.int32).to(DEV)
    x, base = randn(1, T, 264), randn(2, T, 256)
    y = p.add(x, index, base)
    check_add(p, x, index, base, y)
    b2 = base.clone()
    assert torch.equal(p.add(x, index, b2, y=b2), y)


@pytest.mark.parametrize("T", [30, 300])
def test_what_lies_past_a_rank_is_not_used(gpu_lib, T):
    p = make_pool(5, 48, 136, (70, 33), ranks=[1, 7, 16, 31, 48])
    for a, r in enumerate(p.rank.tolist()):
        p.vt.view(5, 2, 48, 136)[a, :, r:] = float("nan")
        p.u[a, :, r:] = float("inf")
    x, base, index = randn(1, T, 136), randn(2, T, 103), mixed_index(T, 5, 3)
    check_add(p, x, index, base, p.add(x, index, base))


@pytest.mark.parametrize("T", [5, 300])
def test_unaligned_base_and_y(gpu_lib, T):
    """base and y at addresses that are only 2-byte aligned, and of different alignment."""
    p = make_pool(3, 16, 128, (64, 8))
    x, index = randn(1, T, 128), mixed_index(T, 3, 4)
    raw = randn(2, T * 72 + 8)
    want = p.add(x, index, raw[:T * 72].view(T, 72))
    base = torch.empty(T * 72 + 8, dtype=torch.bfloat16, device=DEV)
    for i, j in ((1, 0), (0, 1), (3, 5), (8, 8)):
        out = torch.empty(T * 72 + 8, dtype=torch.bfloat16, device=DEV)
        b = base[i:i + T * 72].view(T, 72)
        b.copy_(raw[:T * 72].view(T, 72))
        assert torch.equal(p.add(x, index, b, y=out[j:j + T * 72].view(T, 72)), want)


@pytest.mark.parametrize("T", [20, 400])
def test_not_finite_stays_where_it_is(gpu_lib, T):
    p = make_pool(4, 32, 136, (100, 60))
    x, base, index = randn(1, T, 136), randn(2, T, 160), (torch.arange(T) % 5).to(torch.int32).to(DEV)
    clean = p.add(x, index, base)
    x[6, 3], x[12, 100] = float("inf"), float("nan")
    p.vt[3, 1, 5] = float("nan")
    y = p.add(x, index, base)
    touched = torch.zeros(T, dtype=torch.bool, device=DEV)
    touched[[6, 12]] = True
    touched |= index == 3
    assert torch.equal(y[~touched].view(torch.int16), clean[~touched].view(torch.int16))
    assert torch.isnan(y[12]).all() and not torch.isfinite(y[6]).any() and torch.isnan(y[index == 3][:, :100]).all()
    # an adapter's first output grows past bf16: infinity, not NaN
    p2 = make_pool(1, 16, 8, (4,))
    p2.vt.fill_(0)
    p2.vt[0, 0, 0] = 3e38
    p2.u.fill_(0)
    p2.u[0, :, 0] = 1.0
    p2.scale.fill_(1.0)
    xs = torch.zeros(1, 8, dtype=torch.bfloat16, device=DEV)
    xs[0, 0] = 100.0
    assert torch.isinf(p2.add(xs, torch.zeros(1, dtype=torch.int32, device=DEV), torch.zeros(1, 4, dtype=torch.bfloat16, device=DEV))).all()


@pytest.mark.parametrize("T", [33, 500])
def test_a_token_does_not_depend_on_the_others(gpu_lib, T):
    p = make_pool(5, 48, 256, (130,))
    x, base, index = randn(1, T, 256), randn(2, T, 130), mixed_index(T, 5, 3)
    y = p.add(x, index, base)
    perm = torch.randperm(T, generator=torch.Generator("cpu").manual_seed(1)).to(DEV)
    assert torch.equal(p.add(x[perm].contiguous(), index[perm].contiguous(), base[perm].contiguous()), y[perm])


def test_loading_and_clearing_slots(gpu_lib):
    K, rows = 264, (96, 40)
    p = binding.AdapterPool.empty(4, 32, K, rows)
    x, base = randn(1, 12, K), randn(2, 12, 136)
    index = (torch.arange(12) % 4).to(torch.int32).to(DEV)
    assert torch.equal(p.add(x, index, base), base)
    down, up = [randn(3, 20, K, std=0.1), randn(4, 20, K, std=0.1)], [randn(5, 96, 20), randn(6, 40, 20)]
    p.load(2, down, up, scale=0.75)
    y = p.add(x, index, base)
    check_add(p, x, index, base, y)
    on = index == 2
    want = base[on].double() + 0.75 * torch.cat([(x[on].double() @ a.double().t().contiguous()) @ b.double().t().contiguous() for a, b in zip(down, up)], 1)
    assert (y[on].double() - want).norm() <= 2 * H * want.norm() and not torch.equal(y[on], base[on])
    p.clear(2)
    assert torch.equal(p.add(x, index, base), base)
    for bad in ((4, down, up), (-1, down, up), (0, down[:1], up[:1]), (0, [d[:, :8] for d in down], up), (0, [randn(1, 33, K)] * 2, [randn(1, 96, 33), randn(1, 40, 33)])):
        with pytest.raises(binding.WlError):
            p.load(*bad)


def test_beside_a_shared_projection(gpu_lib):
    """The stacked call and the coded product with adapters on their outputs, in place."""
    K, rows, r = 264, (128, 40, 40), 16
    fams = ("q", "k", "v")
    spec = binding.make_spec(1, 1, {(0, f): (n, K) for f, n in zip(fams, rows)}, {(0, f): 8 for f in fams})
    src = [s for i, (f, n) in enumerate(zip(fams, rows)) for s in
           (("w0", 0, 0, f, randn(10 + i, n, K, std=K ** -0.5)), ("s", 0, 0, f, torch.ones(n, device=DEV)),
            ("u", 0, 0, f, randn(20 + i, n, 8)), ("v", 0, 0, f, randn(30 + i, K, 8, std=0.05)))]
    b = binding.ThetaBundle(spec, src)
    p = make_pool(3, r, K, rows)
    for T in (1, 9, 40, 300):
        x, index = randn(T, T, K), mixed_index(T, 3, T, wild=T > 1)
        base = b.stacked(0, "qkv", x)
        y = base.clone()
        p.add(x, index, y, y=y)
        check_add(p, x, index, base, y)
    w = binding.encode_weight(randn(50, 208, K, std=K ** -0.5))
    base = binding.coded_linear(w, x)
    check_add(p, x, index, base, p.add(x, index, base))


@pytest.mark.parametrize("T", [7, 600])
def test_replayed_from_a_graph_with_other_slots(gpu_lib, T):
    p = make_pool(8, 16, 128, (72,), ranks=[16, 4, 0, 9, 16, 16, 1, 12])
    x, base, index = randn(1, T, 128), randn(2, T, 72), mixed_index(T, 8, 3)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        p.add(x, index, base)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = p.add(x, index, base)
    for seed in (4, 5, 6, 7):
        index.copy_(mixed_index(T, 8, seed))
        x.copy_(randn(seed, T, 128))
        p.rank.copy_(p.rank.roll(1))
        p.rank.clamp_(max=int(seed))   # slots lose ranks: what they hold past them is not zero up to 16 ...
        p.vt.view(8, 1, 16, 128)[:, :, seed:] = 0   # ... until it is
        p.u[:, :, seed:] = 0
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, p.add(x, index, base))
        check_add(p, x, index, base, y)


def test_nothing_else_is_written(gpu_lib):
    for T in (21, 777):
        p = make_pool(3, 32, 136, (37,))
        x, index, base = randn(1, T, 136), mixed_index(T, 3, 2), randn(2, T, 37)
        pad = 4096
        ybuf = torch.full((T * 37 * 2 + 2 * pad,), 0x5A, dtype=torch.uint8, device=DEV)
        ws = torch.full((p.workspace_bytes(T) + 2 * pad,), 0x5A, dtype=torch.uint8, device=DEV)
        y = ybuf[pad:-pad].view(torch.bfloat16).view(T, 37)
        p.add(x, index, base, y=y, ws=ws[pad:-pad])
        check_add(p, x, index, base, y)
        for b in (ybuf, ws):
            assert (b[:pad] == 0x5A).all() and (b[-pad:] == 0x5A).all()


def test_other_streams_have_their_own_workspaces(gpu_lib):
    p = make_pool(4, 32, 1152, (2048,))
    streams = [torch.cuda.Stream() for _ in range(3)]
    data = [(randn(i, 48, 1152), mixed_index(48, 4, i), randn(i + 50, 48, 2048)) for i in range(3)]
    want = [p.add(*d) for d in data]
    torch.cuda.synchronize()
    got = [[p.add(*d, stream=s) for _ in range(20)] for s, d in zip(streams, data)]
    torch.cuda.synchronize()
    assert all(torch.equal(y, w) for ys, w in zip(got, want) for y in ys)


def test_binding_refusals(gpu_lib):
    p = make_pool(2, 16, 64, (32,))
    x, base, index = randn(1, 4, 64), randn(2, 4, 32), torch.zeros(4, dtype=torch.int32, device=DEV)
    for bad in (dict(x=randn(1, 4, 72)), dict(x=x.float()), dict(index=index.long()), dict(index=index[:3]), dict(base=randn(1, 4, 40)),
                dict(base=base.t().contiguous().t()), dict(y=base.float()), dict(y=x[:, :32]), dict(ws=torch.empty(256, dtype=torch.uint8, device=DEV)[:8])):
        with pytest.raises(binding.WlError):
            p.add(**{**dict(x=x, index=index, base=base), **bad})
    for args in ((p.vt, p.u, p.scale, (40,)), (p.vt, p.u, p.scale.double(), (32,)), (p.vt, p.u, p.scale, (32,), index), (p.vt, p.u, p.scale, ()),
                 (p.vt[:, :8].contiguous(), p.u[:, :, :8].contiguous(), p.scale, (32,))):
        with pytest.raises(binding.WlError):
            binding.AdapterPool(*args)


def test_offsets_past_2_to_the_31(gpu_lib):
    """base and y of more than 2^31 elements, and a pool of more."""
    T, N, K = 66000, 33000, 64
    announce(f"adapters T={T} N={N}")
    p = make_pool(3, 16, K, (N,))
    x, index = randn(1, T, K), mixed_index(T, 3, 2)
    y = torch.zeros(T, N, dtype=torch.bfloat16, device=DEV)
    p.add(x, index, y, y=y)
    rows = torch.tensor([0, 1, 40000, 65070, T - 2, T - 1], device=DEV)
    zero = torch.zeros(6, N, dtype=torch.bfloat16, device=DEV)
    check_add(p, x[rows].contiguous(), index[rows].contiguous(), zero, y[rows])
    del y
    n, r, N = 600, 256, 16384
    p = binding.AdapterPool.empty(n, r, K, (N,))
    assert p.u.numel() > 2 ** 31
    p.load(n - 1, [randn(3, r, K, std=0.1)], [randn(4, N, r)])
    for T in (3, 300):
        x, base = randn(5, T, K), randn(6, T, N)
        index = torch.full((T,), n - 1, dtype=torch.int32, device=DEV)
        check_add(p, x, index, base, p.add(x, index, base))
