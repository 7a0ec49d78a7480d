"""GPU: gradients of the weightless linear from an 8-bit checkpoint.

The reference is torch autograd over the forward written out in float64 (on
the GPU), at the checkpoint's own values; a second test holds the results to
differences of that forward.  Tolerances, derived before the first run, per
element: a bf16 rounding 2^-8 of the value, a float32 sum of n terms n * 2^-23
of the sum of their magnitudes; with |.| elementwise and X, D = dy:

  ds   (T + K + 8) 2^-23  sum_k (|D|^T |X|) |W0|
  dW0  |s| (T + 8) 2^-23  |D|^T |X|
  z    e_z = 2^-16 |X V| + K 2^-23 |X| |V|       (a pair of bf16; g likewise with D, U)
  dU   |D|^T e_z + (T + 8) 2^-23 |D|^T |X V| + 2^-8 |dU|
  dV   |X|^T e_g + (T + 8) 2^-23 |X|^T |D U| + 2^-8 |dV|
  dx   (2^-8 + (N + r + 8) 2^-23) (|D| |s|) |W0| + e_g |V|^T
       + (N + r + 8) 2^-23 |D U| |V|^T + 2^-8 |dx|

and, the roundings of many terms being independent, the error's norm within
2 * 2^-8 of the result's for dx (two roundings on the way) and 2^-8 for dU and
dV (one)."""
import sys

import numpy as np
import pytest
import torch

from weight_shared_rank_amd import binding

pytestmark = pytest.mark.gpu
DEV = "cuda"
H, F = 2.0 ** -8, 2.0 ** -23
ALL = ("dx", "ds", "du", "dv", "dw0")


def announce(msg):
    sys.__stderr__.write(f"[gpu] {msg}\n")
    sys.__stderr__.flush()


def randn(seed, *shape, std=1.0, dtype=torch.bfloat16):
    g = torch.Generator("cpu").manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype).to(DEV)


class Layer:
    """One group of families over one K, as a bundle and as float64 tensors."""

    def __init__(self, fams, rows, K, ranks, tied=False, fmt="bf16", seed=0, layers=1):
        self.fams, self.rows, self.K, self.ranks, self.tied = fams, rows, K, ranks, tied
        own = [f for f in fams if not (tied and f == "v")]
        spec = binding.make_spec(layers, 1, {(0, f): (n, K) for f, n in zip(own, rows)},
                                 {(0, f): r for f, r in zip(own, ranks)}, k_eq_v_types=(0,) if tied else (),
                                 w0_format=fmt)
        src, self.w0, self.s, self.u, self.v = [], [], [], [], []
        for i, (f, n, r) in enumerate(zip(own, rows, ranks)):
            at = seed * 100 + i * 10
            self.w0.append(randn(at, n, K, std=K ** -0.5))
            src.append(("w0", 0, 0, f, self.w0[-1]))
            for l in range(layers):
                s = 1 + 0.2 * randn(at + 1 + 1000 * l, n, dtype=torch.float32)
                u, v = randn(at + 2 + 1000 * l, n, r, std=0.2), randn(at + 3 + 1000 * l, K, r, std=0.2)
                src.append(("s", l, 0, f, s))
                if r:
                    src += [("u", l, 0, f, u), ("v", l, 0, f, v)]
            self.s.append(s)
            self.u.append(u)
            self.v.append(v)
        self.layer = layers - 1
        self.bundle = binding.ThetaBundle(spec, src, device=DEV)
        if fmt != "bf16":  # the values of the codes: s = 1, rank 0 materializes them exactly
            plain = binding.ThetaBundle(
                binding.make_spec(1, 1, {(0, f): (n, K) for f, n in zip(own, rows)}, {}, w0_format=fmt),
                [x for f, n, w in zip(own, rows, self.w0)
                 for x in (("w0", 0, 0, f, w), ("s", 0, 0, f, torch.ones(n, device=DEV)))], device=DEV)
            self.w0 = [plain.materialize(0, f) for f in own]

    @property
    def stack(self):
        return {3: "qkv", 2: "gate_up", 1: None}[len(self.fams)]

    @property
    def width(self):
        return sum(self.rows) + (self.rows[-1] if self.tied else 0)

    def backward(self, code, dy, want=ALL, **kw):
        if self.stack:
            return self.bundle.stacked_backward(self.layer, self.stack, code, dy, want=want, **kw)
        g = self.bundle.linear_backward(self.layer, self.fams[0], code, dy, want=want, **kw)
        return g._replace(du=None if g.du is None else (g.du,), dv=None if g.dv is None else (g.dv,))

    def slots(self, dy):
        """dy's columns per child (a tied v slot's as a second block of k's)."""
        edges = np.cumsum([0] + list(self.rows) + ([self.rows[-1]] if self.tied else []))
        parts = [dy[:, a:b] for a, b in zip(edges, edges[1:])]
        return [[p] for p in parts[:-1]][:-1] + [[parts[-2], parts[-1]]] if self.tied else [[p] for p in parts]


def check(lay, x, dy, g):
    """The gradients g against autograd in float64 (and the tolerances above)."""
    X = x.expand().double().requires_grad_(True)
    s, u, v = ([t.double().requires_grad_(True) for t in ts] for ts in (lay.s, lay.u, lay.v))
    w = [t.double().requires_grad_(True) for t in lay.w0]
    D = lay.slots(dy.double())
    loss = 0.0
    for i, ds in enumerate(D):
        y = (X @ w[i].t().contiguous()) * s[i] + (X @ v[i]) @ u[i].t().contiguous()
        for d in ds:
            loss = loss + (y * d).sum()
    loss.backward()
    X = X.detach()
    T, K, N = X.shape[0], lay.K, sum(lay.rows)
    tol = {"dx": torch.zeros_like(X), "ds": [], "dw0": [], "du": [], "dv": []}
    depth = sum(len(ds) * n for ds, n in zip(D, lay.rows)) + 2 * sum(lay.ranks) + 8
    for i, ds in enumerate(D):
        a, b = X.abs(), sum(d.abs() for d in ds)
        n2 = 2 * len(ds) * T + 8  # (z's and g's pairs double the terms)
        wi, si, ui, vi = w[i].detach(), s[i].detach(), u[i].detach(), v[i].detach()
        big = b.t().contiguous() @ a
        tol["ds"].append((n2 + K) * F * (big * wi.abs()).sum(1))
        tol["dw0"].append(si.abs()[:, None] * n2 * F * big)
        z, gg = X @ vi, sum(d @ ui for d in ds)
        ez = H * H * z.abs() + K * F * (a @ vi.abs())
        eg = H * H * gg.abs() + depth * F * (b @ ui.abs())
        tol["du"].append(b.t().contiguous() @ (ez + n2 * F * z.abs()) + H * u[i].grad.abs())
        tol["dv"].append(a.t().contiguous() @ (eg + n2 * F * gg.abs()) + H * v[i].grad.abs())
        tol["dx"] += (H + depth * F) * ((b * si.abs()) @ wi.abs()) + (eg + depth * F * gg.abs()) @ vi.abs().t().contiguous()
    ref = {"dx": x_grad(X, lay, D, s, u, v, w), "ds": torch.cat([t.grad for t in s]),
           "dw0": torch.cat([t.grad for t in w]), "du": [t.grad for t in u], "dv": [t.grad for t in v]}
    tol["dx"] += H * ref["dx"].abs()
    tol["ds"], tol["dw0"] = torch.cat(tol["ds"]), torch.cat(tol["dw0"])

    def one(name, got, want, bound, norm):
        assert got.shape == want.shape, name
        err = (got.double() - want).abs()
        bad = torch.nonzero(~(err <= bound))
        assert len(bad) == 0, (name, bad[:3], got[tuple(bad[0])].item(), want[tuple(bad[0])].item())
        if want.numel() >= 64:  # a norm over a handful of elements averages nothing
            assert err.norm() <= norm * want.norm(), (name, (err.norm() / want.norm()).item())
    for name in ("dx", "ds", "dw0"):
        if getattr(g, name) is not None:
            one(name, getattr(g, name), ref[name], tol[name], 2 * H if name == "dx" else 1e-5)
    for name in ("du", "dv"):
        if getattr(g, name) is not None:
            assert len(getattr(g, name)) == len(D)
            for i, t in enumerate(getattr(g, name)):
                one(f"{name}[{i}]", t, ref[name][i], tol[name][i], H)


def x_grad(X, lay, D, s, u, v, w):
    out = torch.zeros_like(X)
    for i, ds in enumerate(D):
        d = sum(ds)
        out += (d * s[i].detach()) @ w[i].detach() + (d @ u[i].detach()) @ v[i].detach().t().contiguous()
    return out


def same_bits(a, b):
    for x, y in zip(a, b):
        if isinstance(x, tuple):
            same_bits(x, y)
        elif x is not None:
            assert torch.equal(x, y)
        else:
            assert y is None


O, GU, QKV = ("o",), ("gate", "up"), ("q", "k", "v")
CASES = [(O, (16,), 8, (1,), 1), (O, (40,), 64, (4,), 1), (O, (1,), 128, (0,), 3), (O, (128,), 128, (32,), 64),
         (O, (1001,), 712, (20,), 77), (O, (300,), 264, (0,), 130), (O, (64,), 2056, (64,), 17),
         (O, (520,), 136, (130,), 300), (O, (72,), 72, (8,), 3000), (O, (2048,), 1024, (96,), 257),
         (GU, (200, 200), 264, (5, 33), 65), (GU, (513, 513), 520, (64, 0), 40), (GU, (1000, 1000), 904, (70, 40), 513),
         (QKV, (200, 72, 72), 264, (40, 33, 1), 100), (QKV, (33, 7, 9), 40, (5, 2, 3), 2),
         (QKV, (1024, 256, 256), 1152, (64, 64, 64), 600),
         (O, (4090,), 4088, (24,), 4080),  # 256 x 256 tiles
         # few tokens through a large block: one pass over it
         (O, (4100,), 4104, (0,), 1), (O, (1030,), 16392, (129,), 33), (GU, (2101, 2101), 4008, (20, 0), 64),
         (GU, (265, 265), 40000, (3, 40), 50), (QKV, (64000, 130, 63), 264, (33, 16, 8), 17),
         (QKV, (12000, 3000, 2000), 1000, (8, 64, 1), 64), (O, (4100,), 4104, (4,), 65),
         (GU, (2101, 2101), 4008, (20, 0), 128), (QKV, (12000, 3000, 2001), 1000, (8, 64, 1), 97),
         (O, (4100,), 4104, (4,), 129)]


@pytest.mark.parametrize("fams,rows,K,ranks,T", CASES)
def test_gradients_match_autograd(gpu_lib, fams, rows, K, ranks, T):
    lay = Layer(fams, rows, K, ranks, seed=T % 7)
    x = randn(T, T, K)
    x[:, K // 2] *= 24
    announce(f"backward {fams} {rows} K={K} r={ranks} T={T}")
    code = binding.encode_act(x)
    dy = randn(T + 1, T, lay.width, std=T ** -0.5)
    check(lay, code, dy, lay.backward(code, dy))


@pytest.mark.parametrize("rows,T", [((40, 24), 9), ((130, 70), 70), ((256, 128), 400)])
def test_tied_v_adds_to_k(gpu_lib, rows, T):
    """K = V tying: dy has three slots, q, k and v; k's gradients sum both."""
    lay = Layer(QKV, rows, 392, (17, 8), tied=True, seed=3)
    code, dy = binding.encode_act(randn(1, T, 392)), randn(2, T, lay.width, std=T ** -0.5)
    announce(f"tied {rows} T={T}")
    check(lay, code, dy, lay.backward(code, dy))
    # the single call for v runs k's bundle
    g = lay.bundle.linear_backward(0, "v", code, dy[:, -rows[1]:].contiguous(), want=ALL)
    h = lay.bundle.linear_backward(0, "k", code, dy[:, -rows[1]:].contiguous(), want=ALL)
    same_bits(g, h)


@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
@pytest.mark.parametrize("T,N,K", [(5, 136, 264), (90, 136, 264), (30, 2100, 4104)])
def test_coded_shared_blocks(gpu_lib, fmt, T, N, K):
    lay = Layer(GU, (N, N), K, (9, 9), fmt=fmt, seed=4, layers=2)
    code, dy = binding.encode_act(randn(3, T, K)), randn(4, T, lay.width, std=T ** -0.5)
    announce(f"{fmt} T={T}")
    check(lay, code, dy, lay.backward(code, dy))


def test_gradients_match_differences(gpu_lib):
    """Directional central differences of the float64 forward (it is linear in
    each of x, s, W0, U and V, so they are exact up to float64) against the
    inner products of the gradients with the directions."""
    lay = Layer(QKV, (96, 40, 24), 200, (6, 4, 3), seed=5)
    T = 33
    code, dy = binding.encode_act(randn(5, T, 200)), randn(6, T, lay.width)
    g = lay.backward(code, dy)
    base = {"dx": [code.expand().double()], "ds": [t.double() for t in lay.s], "dw0": [t.double() for t in lay.w0],
            "du": [t.double() for t in lay.u], "dv": [t.double() for t in lay.v]}
    D = lay.slots(dy.double())

    def loss(p):
        x = p["dx"][0]
        return sum(((x @ w.t().contiguous()) * s + (x @ v) @ u.t().contiguous()).mul(d[0]).sum().item()
                   for w, s, u, v, d in zip(p["dw0"], p["ds"], p["du"], p["dv"], D))
    for name in ALL:
        got = getattr(g, name)
        got = list(got) if isinstance(got, tuple) else list(torch.split(got, [t.shape[0] for t in base[name]]))
        for i, t in enumerate(base[name]):
            d = randn(70 + i, *t.shape, dtype=torch.float32).double()
            up, dn = (dict(base, **{name: [b + e * d if j == i else b for j, b in enumerate(base[name])]})
                      for e in (0.5, -0.5))
            want, have = loss(up) - loss(dn), (got[i].double() * d).sum().item()
            # <grad, d> is off by at most |error| |d|, the error's norm within 2 * 2^-8 of the gradient's
            assert abs(have - want) <= 2 * H * got[i].double().norm().item() * d.norm().item(), (name, i)


@pytest.mark.parametrize("rows,K,T", [((200, 72, 40), 264, 100), ((6000, 2000, 333), 2104, 60), ((6000, 2000, 333), 2104, 120)])
def test_subsets_give_the_same_bits(gpu_lib, rows, K, T):
    lay = Layer(QKV, rows, K, (40, 33, 8), seed=6)
    code, dy = binding.encode_act(randn(7, T, K)), randn(8, T, lay.width)
    full = lay.backward(code, dy)
    for want in (("dx",), ("ds",), ("du",), ("dv",), ("dw0",), ("dx", "dv"), ("ds", "du"), ()):
        announce(f"want {want}")
        part = lay.backward(code, dy, want=want)
        for name in ALL:
            a, b = getattr(full, name), getattr(part, name)
            assert (b is None) == (name not in want)
            if b is not None:
                same_bits((a,), (b,))


def poisoned(lay, code, dy, want=ALL, dw0=None):
    """The call through the C ABI with every byte of the workspace and of the
    outputs 0xFF (NaN as bf16 and as float32), so that nothing an earlier call
    left can stand in for what this one must write; dw0: accumulated into."""
    import ctypes
    L, T = binding.lib(), code.T

    def nans(*shape, dtype=torch.bfloat16):
        return torch.full((int(np.prod(shape)) * dtype.itemsize,), 0xFF, dtype=torch.uint8, device=DEV).view(dtype).view(shape)
    g, out = binding.WlGrads(), {}
    for name, shape, dtype in (("dx", (T, lay.K), torch.bfloat16), ("ds", (sum(lay.rows),), torch.float32),
                               ("dw0", (sum(lay.rows), lay.K), torch.float32)):
        if name in want:
            out[name] = dw0 if name == "dw0" and dw0 is not None else nans(*shape, dtype=dtype)
            setattr(g, name, out[name].data_ptr())
    g.accumulate_dw0 = dw0 is not None
    for name, heights in (("du", lay.rows), ("dv", [lay.K] * len(lay.rows))):
        if name in want:
            out[name] = tuple(nans(h, r) for h, r in zip(heights, lay.ranks))
            for i, t in enumerate(out[name]):
                getattr(g, name)[i] = t.data_ptr() or None
    need = L.weightless_backward_workspace_bytes(lay.bundle.handle, T)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV)
    fn, which = (L.weightless_stacked_backward, binding.STACKS[lay.stack]) if lay.stack else \
        (L.weightless_linear_backward, binding.FAMILY[lay.fams[0]])
    st = fn(lay.bundle.handle, lay.layer, which, code.buf.data_ptr(), code.buf.numel(), dy.data_ptr(), T,
            ctypes.byref(g), ws.data_ptr(), need, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert st == 0, binding.last_error()
    return binding.Grads(**out)


@pytest.mark.parametrize("T", [1, 16, 64, 65, 128])
@pytest.mark.parametrize("fams,rows,K,ranks,fmt", [
    (O, (4104,), 4104, (8,), "bf16"), (GU, (2104, 2104), 4008, (20, 0), "bf16"),
    (QKV, (6000, 2000, 336), 2104, (40, 33, 8), "bf16"), (O, (4104,), 4104, (8,), "fp8")])
def test_one_pass_without_dx_reads_dy_in_place(gpu_lib, fams, rows, K, ranks, fmt, T):
    """Few tokens through a large block with rows in multiples of 8: dy is read
    where it lies, and what the call then wants of it decides what is prepared."""
    lay = Layer(fams, rows, K, ranks, fmt=fmt, seed=19)
    code, dy = binding.encode_act(randn(80, T, K)), randn(81, T, lay.width, std=T ** -0.5)
    announce(f"all of {rows} {fmt} T={T}")
    full = poisoned(lay, code, dy)
    check(lay, code, dy, full)
    for want in (("ds",), ("dw0",), ("ds", "dw0"), ("ds", "du"), ("dw0", "dv"), ("du", "dv"), ("dx",), ("dx", "dw0")):
        announce(f"want {want}")
        part = poisoned(lay, code, dy, want)
        for name in want:
            same_bits((getattr(part, name),), (getattr(full, name),))
    acc = randn(82, sum(rows), K, dtype=torch.float32)
    total = acc + full.dw0
    poisoned(lay, code, dy, ("dw0",), dw0=acc)
    assert ((acc - total).abs() <= F * (full.dw0.abs() + total.abs())).all()


@pytest.mark.parametrize("T,rows,K,ranks,tied", [(3, (24, 16), 264, (5, 13), False), (70, (21, 13), 136, (4, 0), False),
                                                 (200, (304, 304), 520, (40, 8), False), (90, (64, 32), 264, (16, 8), True)])
def test_every_subset_on_a_poisoned_workspace(gpu_lib, T, rows, K, ranks, tied):
    """All 31 choices of gradients: each writes all it reads of its workspace."""
    lay = Layer(QKV if tied else GU, rows, K, ranks, tied=tied, seed=20)
    code, dy = binding.encode_act(randn(83, T, K)), randn(84, T, lay.width)
    full = poisoned(lay, code, dy)
    check(lay, code, dy, full)
    for bits in range(1, 31):
        want = tuple(n for i, n in enumerate(ALL) if bits >> i & 1)
        announce(f"want {want}")
        part = poisoned(lay, code, dy, want)
        for name in want:
            same_bits((getattr(part, name),), (getattr(full, name),))


@pytest.mark.parametrize("T,rows,K", [(40, 300, 264), (2500, 24, 264), (40, 4100, 4104), (90, 4100, 4104)])
def test_accumulated_block_gradient(gpu_lib, T, rows, K):
    """dw0 += over the layers of a band: the sum of the calls' own gradients,
    one float32 rounding per addition; both with and without a split."""
    lay = Layer(O, (rows,), K, (8,), seed=7)
    code, dy = binding.encode_act(randn(9, T, K)), randn(10, T, rows)
    announce(f"accumulate T={T}")
    one = lay.backward(code, dy, want=("dw0",)).dw0
    acc = randn(11, rows, K, dtype=torch.float32)
    want = acc + one
    got = lay.backward(code, dy, want=("dw0", "ds"), dw0=acc, accumulate=True)
    assert got.dw0 is acc
    assert ((acc - want).abs() <= 2.0 ** -23 * (one.abs() + want.abs())).all()


@pytest.mark.parametrize("N,K", [(136, 264), (4104, 4104)])
def test_unaligned_dy_and_neighbouring_memory(gpu_lib, N, K):
    """dy that starts at an odd element; outputs at odd places in larger
    buffers whose other elements stay as they were."""
    lay = Layer(O, (N,), K, (8,), seed=8)
    T = 50
    code, dy = binding.encode_act(randn(12, T, K)), randn(13, T, N)
    want = lay.backward(code, dy)
    flat = torch.empty(T * N + 1, dtype=torch.bfloat16, device=DEV)
    flat[1:] = dy.flatten()
    announce("unaligned dy")
    same_bits(lay.backward(code, flat[1:].view(T, N)), want)
    # raw call with outputs inside larger buffers
    sizes = {"dx": (T * K, 2, 8), "du": (N * 8, 2, 1), "dv": (K * 8, 2, 1), "ds": (N, 4, 1), "dw0": (N * K, 4, 4)}
    bufs = {k: torch.full((n + 2 * o,), 7.0, dtype=torch.bfloat16 if b == 2 else torch.float32, device=DEV)
            for k, (n, b, o) in sizes.items()}
    g = binding.WlGrads()
    for k, (n, b, o) in sizes.items():
        p = bufs[k].data_ptr() + o * b
        if k in ("du", "dv"):
            getattr(g, k)[0] = p
        else:
            setattr(g, k, p)
    L = binding.lib()
    need = L.weightless_backward_workspace_bytes(lay.bundle.handle, T)
    ws = torch.full((need + 256,), 0x5A, dtype=torch.uint8, device=DEV)
    import ctypes
    st = L.weightless_linear_backward(lay.bundle.handle, 0, binding.FAMILY["o"], code.buf.data_ptr(), code.buf.numel(),
                                      dy.data_ptr(), T, ctypes.byref(g), ws.data_ptr(), need,
                                      ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert st == 0, binding.last_error()
    assert (ws[need:] == 0x5A).all()
    for k, (n, b, o) in sizes.items():
        t = getattr(want, k)
        t = t[0] if isinstance(t, tuple) else t
        assert torch.equal(bufs[k][o:o + n], t.flatten()) and (bufs[k][:o] == 7).all() and (bufs[k][o + n:] == 7).all(), k


@pytest.mark.parametrize("N,K", [(77, 264), (4100, 4104)])
def test_non_finite_values_stay_where_they_belong(gpu_lib, N, K):
    lay = Layer(O, (N,), K, (8,), seed=9)
    T = 40
    x, dy = randn(14, T, K), randn(15, T, N)
    dy[3, N - 1] = float("nan")
    x[5, K - 1] = float("inf")
    announce("non-finite")
    g = lay.backward(binding.encode_act(x), dy)
    nan = torch.isnan(g.dx).any(1)
    assert nan[3] and nan.sum() == 1                       # dx: that token only (x does not enter dx)
    rows = torch.isnan(g.dw0)
    assert rows[N - 1].all() and rows[:, K - 1].all() and rows[:N - 1, :K - 1].sum() == 0
    assert torch.isnan(g.dv[0]).all() and torch.isnan(g.du[0]).all()   # g's and z's token enter every sum
    assert torch.isfinite(lay.backward(binding.encode_act(randn(14, T, K)), randn(15, T, N)).dx).all()


def test_no_tokens_zero_the_sums(gpu_lib):
    lay = Layer(GU, (40, 40), 64, (4, 0), seed=10)
    code = binding.ActCode(0, 64)
    dy = torch.empty(0, 80, dtype=torch.bfloat16, device=DEV)
    g = lay.backward(code, dy)
    assert g.dx.shape == (0, 64) and not g.ds.any() and not g.dw0.any() and not g.du[0].any() and not g.dv[0].any()
    acc = torch.ones(80, 64, device=DEV)
    lay.backward(code, dy, want=("dw0",), dw0=acc, accumulate=True)
    assert (acc == 1).all()


@pytest.mark.parametrize("rows,K,T", [((256, 128, 128), 512, 150), ((6000, 3000, 1900), 1544, 20)])
def test_side_stream_graph_and_two_at_once(gpu_lib, rows, K, T):
    lay = Layer(QKV, rows, K, (32, 16, 16), seed=11)
    codes = [binding.encode_act(randn(20 + i, T, K)) for i in range(3)]
    dys = [randn(30 + i, T, lay.width) for i in range(3)]
    want = [lay.backward(c, d) for c, d in zip(codes, dys)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    announce("two streams")
    got = [[], []]
    for _ in range(4):
        for i in (0, 1):
            got[i].append(lay.backward(codes[i], dys[i], stream=streams[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        for g in got[i]:
            same_bits(g, want[i])
    code, dy = binding.ActCode(T, K, buf=codes[0].buf.clone()), dys[0].clone()
    graph = torch.cuda.CUDAGraph()
    announce("capture")
    with torch.cuda.graph(graph):
        g = lay.backward(code, dy)
    for i in (1, 2, 0, 1):
        code.buf.copy_(codes[i].buf)
        dy.copy_(dys[i])
        graph.replay()
        torch.cuda.synchronize()
        same_bits(g, want[i])
        same_bits(lay.backward(codes[2 - i], dys[2 - i]), want[2 - i])


def test_forward_checkpoint_backward_together(gpu_lib):
    """A training step's calls as they are used: the forward on x, its
    checkpoint, the backward; and the forward's own change when s moves by a
    multiple of ds is what ds says (<y, dy> is linear in s, so up to the
    roundings of the outputs and of the checkpoint)."""
    lay = Layer(GU, (256, 256), 384, (16, 16), seed=12)
    T = 64
    x = randn(40, T, 384)
    dy = randn(41, T, lay.width, std=T ** -0.5)
    announce("forward, checkpoint, backward")
    y0 = lay.bundle.stacked(0, "gate_up", x).double()
    code = binding.encode_act(x)
    g = lay.backward(code, dy)
    check(lay, code, dy, g)
    step = 0.25
    spec = lay.bundle.spec
    src = []
    for i, f in enumerate(GU):
        s = lay.s[i] - step * g.ds[i * 256:(i + 1) * 256]
        src += [("w0", 0, 0, f, lay.w0[i]), ("s", 0, 0, f, s), ("u", 0, 0, f, lay.u[i]), ("v", 0, 0, f, lay.v[i])]
    y1 = binding.ThetaBundle(spec, src, device=DEV).stacked(0, "gate_up", x).double()
    drop = ((y0 - y1) * dy.double()).sum().item()
    # ds at the checkpoint's values against the drop at x itself: E4M3 rounds x by at most 2^-4 of each
    # element, the outputs by 2^-8; the errors' inner products with dy are bounded by their norms
    xe = x.double()
    full = sum((((xe @ lay.w0[i].double().t().contiguous()) * g.ds[i * 256:(i + 1) * 256].double())
                * dy.double()[:, i * 256:(i + 1) * 256]).sum().item() for i in (0, 1))
    assert abs(drop - step * full) <= 2 * H * (y0.norm() * dy.double().norm()).item()
    mass = sum(((xe.abs() @ lay.w0[i].double().abs().t().contiguous()) * g.ds[i * 256:(i + 1) * 256].double().abs()
                * dy.double()[:, i * 256:(i + 1) * 256].abs()).sum().item() for i in (0, 1))
    assert abs(full - (g.ds.double() ** 2).sum().item()) <= 2.0 ** -4 * mass


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_updated_values_are_loaded_into_the_same_arena(gpu_lib, fmt):
    """A step's update as the header describes it: the new values loaded over
    the old on the same stream, behind the calls that read those, with no
    synchronization between; the bits are a fresh bundle's."""
    T, K, rows = 40, 520, (256, 256)
    a, b = (Layer(GU, rows, K, (16, 8), fmt=fmt, seed=i) for i in (21, 22))
    x, dy = randn(90, T, K), randn(91, T, sum(rows), std=T ** -0.5)
    code = binding.encode_act(x)

    def step(bundle):
        g = bundle.stacked_backward(0, "gate_up", code, dy, want=ALL)
        return [bundle.stacked(0, "gate_up", x), g.dx, g.ds, *g.du, *g.dv, g.dw0]

    def sources(lay):
        return [(kind, 0, 0, f, t[i]) for i, f in enumerate(GU)
                for kind, t in (("w0", lay.w0), ("s", lay.s), ("u", lay.u), ("v", lay.v))]
    spec = a.bundle.spec
    want = [step(binding.ThetaBundle(spec, sources(l), device=DEV)) for l in (a, b)]
    arena = torch.empty_like(a.bundle.arena)
    announce(f"load over {fmt}")
    bundles, got = [], []
    for i in range(6):
        bundles.append(binding.ThetaBundle(spec, sources((a, b)[i % 2]), device=DEV, arena=arena))
        got.append(step(bundles[-1]))
    for i, g in enumerate(got):
        for p, q in zip(g, want[i % 2]):
            assert torch.equal(p, q)


@pytest.mark.parametrize("T", [3, 16, 40, 300])
def test_step_of_a_block_in_a_graph(gpu_lib, T):
    """A block's step as a captured graph, replayed on new inputs: the shared
    q|k|v call, a dense projection in 8 bits whose coded input is the checkpoint,
    and both layers' gradients added into the band's one dW0.  Every replay
    equals the calls made one by one."""
    lay = Layer(QKV, (256, 64, 64), 520, (16, 8, 8), seed=18, layers=2)
    wc = binding.encode_weight(randn(70, 200, 520, std=520 ** -0.5))
    ins = [[randn(71 + 2 * i, T, 520), randn(72 + 2 * i, T, lay.width, std=T ** -0.5)] for i in range(3)]

    def step(x, dy, dw0, ws):
        dw0.zero_()
        y = lay.bundle.stacked(1, "qkv", x)
        code = binding.ActCode(T, 520)
        d = binding.coded_linear(wc, x, code=code)
        out = [y, d]
        for l in (0, 1):
            g = lay.bundle.stacked_backward(l, "qkv", code, dy, want=ALL, dw0=dw0, accumulate=True, ws=ws)
            out += [g.dx, g.ds, *g.du, *g.dv]
        return out
    need = binding.lib().weightless_backward_workspace_bytes(lay.bundle.handle, T)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    want = []
    for x, dy in ins:
        dw0 = torch.empty(384, 520, device=DEV)
        want.append([t.clone() for t in step(x, dy, dw0, ws)] + [dw0])
    x, dy, dw0 = ins[0][0].clone(), ins[0][1].clone(), torch.empty(384, 520, device=DEV)
    torch.cuda.synchronize()
    announce(f"captured step T={T}")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(x, dy, dw0, ws)
    for i in (1, 0, 2, 1):
        x.copy_(ins[i][0])
        dy.copy_(ins[i][1])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out + [dw0], want[i]):
            assert torch.equal(a, b)
        again = torch.empty_like(dw0)
        step(ins[2 - i][0], ins[2 - i][1], again, ws)   # eager work between the replays, on the same workspace
        assert torch.equal(again, want[2 - i][-1])
    # the layers' gradients of the shared block add up
    alone = [lay.bundle.stacked_backward(l, "qkv", binding.encode_act(ins[1][0]), ins[1][1], want=("dw0",)).dw0
             for l in (0, 1)]
    total = alone[0] + alone[1]
    assert ((want[1][-1] - total).abs() <= 2 * F * (alone[0].abs() + alone[1].abs())).all()


@pytest.mark.parametrize("T,K", [(1 << 20, 8), (5, 1 << 20)])
def test_most_tokens_and_longest_rows(gpu_lib, T, K):
    lay = Layer(O, (9,), K, (5,), seed=16)
    code, dy = binding.encode_act(randn(64, T, K)), randn(65, T, 9)
    announce(f"T={T} K={K}")
    check(lay, code, dy, lay.backward(code, dy))


@pytest.mark.parametrize("N,K", [(520, 8192), (8200, 136)])
def test_more_than_2_31_elements(gpu_lib, N, K):
    """270000 tokens: x, then dy, hold more than 2^31 elements, and their bytes
    pass 2^32.  Against float64 sums over runs of tokens, by norms: the matrix
    cores round a sum of T terms T / 32 times, each by at most 2^-24 of it, and
    the slices' sums add less than as many again."""
    T, run = 270000, 10000
    lay = Layer(O, (N,), K, (8,), seed=23)
    gen = torch.Generator(DEV).manual_seed(92)

    def rand(width, std):
        t = torch.empty(T, width, dtype=torch.bfloat16, device=DEV)
        for i in range(0, T, run):
            t[i:i + run] = torch.randn(run, width, generator=gen, device=DEV) * std
        return t
    x, dy = rand(K, 1.0), rand(N, T ** -0.5)
    announce(f"T={T} {N} x {K}")
    code = binding.encode_act(x)
    X = code.expand()
    for i in range(0, T, run):
        assert torch.equal(X[i:i + run], binding.encode_act(x[i:i + run]).expand())
    del x
    g = lay.backward(code, dy)
    w, s, u, v = lay.w0[0].double(), lay.s[0].double(), lay.u[0].double(), lay.v[0].double()
    G = torch.zeros(N, K, dtype=torch.float64, device=DEV)
    for i in range(0, T, run):
        d, a = dy[i:i + run].double(), X[i:i + run].double()
        G += d.t().contiguous() @ a
        ref = (d * s) @ w + (d @ u) @ v.t().contiguous()
        assert (g.dx[i:i + run].double() - ref).norm() <= 2 * H * ref.norm(), i
    sums = T / 16 * 2.0 ** -24
    for got, want, tol in ((g.dw0, s[:, None] * G, sums), (g.ds, (G * w).sum(1), 2 * sums),
                           (g.du[0], G @ v, H + sums), (g.dv[0], G.t().contiguous() @ u, H + sums)):
        assert (got.double() - want).norm() <= tol * want.norm()


@pytest.mark.parametrize("T", [20, 200])
def test_a_block_of_more_than_2_31_elements(gpu_lib, T):
    """W0 and dW0 of 2.4e9 elements, in one pass over W0 and as products; the
    tolerances of this file's head over runs of rows."""
    N, K, run = 290000, 8320, 10000
    gen = torch.Generator(DEV).manual_seed(94)
    w0 = torch.empty(N, K, dtype=torch.bfloat16, device=DEV)
    for i in range(0, N, run):
        w0[i:i + run] = torch.randn(run, K, generator=gen, device=DEV) * K ** -0.5
    s = 1 + 0.2 * randn(95, N, dtype=torch.float32)
    bundle = binding.ThetaBundle(binding.make_spec(1, 1, {(0, "o"): (N, K)}, {}),
                                 [("w0", 0, 0, "o", w0), ("s", 0, 0, "o", s)], device=DEV)
    code, dy = binding.encode_act(randn(96, T, K)), randn(97, T, N, std=T ** -0.5)
    announce(f"{N} x {K} T={T}")
    g = bundle.linear_backward(0, "o", code, dy, want=("dx", "ds", "dw0"))
    X = code.expand().double()
    dx, top = torch.zeros_like(X), torch.zeros_like(X)
    for i in range(0, N, run):
        at = slice(i, i + run)
        d, w, si = dy[:, at].double(), w0[at].double(), s[at].double()
        G, mass = d.t().contiguous() @ X, d.t().abs().contiguous() @ X.abs()
        assert ((g.dw0[at] - si[:, None] * G).abs() <= (T + 8) * F * si.abs()[:, None] * mass).all(), i
        assert ((g.ds[at] - (G * w).sum(1)).abs() <= (T + K + 8) * F * (mass * w.abs()).sum(1)).all(), i
        dx += (d * si) @ w
        top += (d * si).abs() @ w.abs()
    assert ((g.dx - dx).abs() <= (H + (N + 8) * F) * top + H * dx.abs()).all()
    assert (g.dx.double() - dx).norm() <= 2 * H * dx.norm()


def test_widest_calls(gpu_lib):
    """More columns than a load can address are refused; just under it (one
    family of 2^20 rows, beyond what 32-bit element offsets of a token reach)
    the last rows are right."""
    n = 1 << 20
    wide = Layer(QKV, (n, n, n), 8, (0, 0, 0), seed=14)
    code, dy = binding.encode_act(randn(60, 3, 8)), randn(61, 3, 3 * n)
    announce("2^20 rows")
    with pytest.raises(binding.WlError, match="WL_ESHAPE"):
        wide.backward(code, dy)
    g = wide.bundle.linear_backward(0, "v", code, dy[:, 2 * n:].contiguous(), want=("dx", "ds", "dw0"))
    D, X, w, s = dy[:, 2 * n:].double(), code.expand().double(), wide.w0[2].double(), wide.s[2].double()
    G = D.t().contiguous() @ X
    mass = D.t().abs().contiguous() @ X.abs()
    assert ((g.dw0 - s[:, None] * G).abs() <= 11 * F * s.abs()[:, None] * mass).all()
    assert ((g.ds - (G * w).sum(1)).abs() <= 19 * F * (mass * w.abs()).sum(1)).all()
    ref, top = (D * s) @ w, (D.abs() * s.abs()) @ w.abs()
    assert ((g.dx - ref).abs() <= (H + (n + 8) * F) * top + H * ref.abs()).all()
    assert (g.dx.double() - ref).norm() <= 2 * H * ref.norm()


def test_dw0_alone_of_a_coded_block_needs_no_block(gpu_lib):
    """dW0 of FP8 and MXFP4 bundles without dx or ds, split over the tokens or
    not, or of few tokens: W0 is not expanded and not read."""
    for fmt in ("fp8", "mxfp4"):
        for T, rows, K in ((40, 300, 264), (2500, 24, 264), (20, 4100, 4104), (70, 4100, 4104)):
            lay = Layer(O, (rows,), K, (8,), fmt=fmt, seed=15)
            code, dy = binding.encode_act(randn(62, T, K)), randn(63, T, rows)
            announce(f"dw0 {fmt} T={T}")
            same_bits(lay.backward(code, dy, want=("dw0",)), lay.backward(code, dy)._replace(dx=None, ds=None, du=None, dv=None))


def test_binding_refusals(gpu_lib):
    lay = Layer(GU, (40, 40), 64, (4, 4), seed=13)
    code, dy = binding.encode_act(randn(50, 6, 64)), randn(51, 6, 80)
    E = binding.WlError
    with pytest.raises(E, match="ActCode"):
        lay.backward(randn(50, 6, 64), dy)
    with pytest.raises(E, match="K = 64"):
        lay.backward(binding.encode_act(randn(50, 6, 72)), dy)
    with pytest.raises(E, match="dy must be"):
        lay.backward(code, dy[:5])
    with pytest.raises(E, match="dy must be"):
        lay.backward(code, dy.float())
    with pytest.raises(E, match="dy must be"):
        lay.backward(code, randn(51, 80, 6).t())
    with pytest.raises(E, match="unknown"):
        lay.backward(code, dy, want=("dq",))
    with pytest.raises(E, match="accumulate"):
        lay.backward(code, dy, want=("dw0",), accumulate=True)
    with pytest.raises(E, match="not wanted"):
        lay.backward(code, dy, want=("dx",), dw0=torch.zeros(80, 64, device=DEV))
    with pytest.raises(E, match="dw0 must be"):
        lay.backward(code, dy, want=("dw0",), dw0=torch.zeros(80, 64, dtype=torch.bfloat16, device=DEV))
    with pytest.raises(E, match="WL_ENOSPACE"):
        lay.backward(code, dy, ws=torch.empty(256, dtype=torch.uint8, device=DEV))
    with pytest.raises(E, match="ws must be"):
        lay.backward(code, dy, ws=torch.empty(1 << 20, dtype=torch.uint8))
    with pytest.raises(E, match="WL_ERANGE"):
        lay.bundle.stacked_backward(1, "gate_up", code, dy)
    with pytest.raises(E, match="WL_ERANGE"):
        lay.bundle.linear_backward(-1, "gate", code, dy)
    with pytest.raises(E, match="WL_ERANGE"):
        lay.bundle.stacked_backward(0, "qkv", code, dy)
    # outputs that overlap an input or each other, and misaligned ones (host checks, nothing runs)
    import ctypes
    L = binding.lib()
    need = L.weightless_backward_workspace_bytes(lay.bundle.handle, 6)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    dx = torch.empty(6, 64, dtype=torch.bfloat16, device=DEV)

    def call(**kw):
        g = binding.WlGrads()
        for k, v in kw.items():
            if k in ("du", "dv"):
                getattr(g, k)[0] = v
            else:
                setattr(g, k, v)
        st = L.weightless_stacked_backward(lay.bundle.handle, 0, 1, code.buf.data_ptr(), code.buf.numel(), dy.data_ptr(),
                                           6, ctypes.byref(g), ws.data_ptr(), need, None)
        return st, binding.last_error()
    for kw, frag in (({"dx": dy.data_ptr()}, "overlap"), ({"dx": code.buf.data_ptr()}, "overlap"),
                     ({"dx": ws.data_ptr()}, "overlap"), ({"ds": lay.bundle.arena.data_ptr()}, "overlap"),
                     ({"dx": dx.data_ptr(), "ds": dx.data_ptr() + 64}, "overlap"),
                     ({"du": dx.data_ptr(), "dv": dx.data_ptr()}, "overlap"),
                     ({"dx": dx.data_ptr() + 2}, "aligned"), ({"ds": dx.data_ptr() + 2}, "aligned"),
                     ({"dw0": dx.data_ptr() + 4}, "aligned"), ({"du": dx.data_ptr() + 1}, "aligned")):
        st, err = call(**kw)
        assert st == -1 and frag in err, (kw, err)
