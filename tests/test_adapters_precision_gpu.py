"""GPU: z and g of the adapters keep float32's 24 bits where they enter the second products.

Two terms that cancel but for 2^-12 of them: a rounding of z to 16 bits then shows as 2^-5
of the result.  The thin products are exact (ones and one 2^-12), so c z and c g are one
float32 rounding from exact, and the scales c are those of 4096 candidates whose c and
c (1 + 2^-12) two bf16 hold worst.

Tolerance, derived before the first run, with m the sum of the magnitudes of the n terms
that enter an element: 2^-8 of the result (bf16), 2^-24 m for c z, and for each of the 3 n
additions of the product 2^-23 m.  With two bf16 for z the error reaches 2^-17.2 m, five
times what is allowed at n = 2."""
import pytest
import torch

from test_adapters_gpu import DEV
from weight_shared_rank_amd import binding

pytestmark = pytest.mark.gpu
H, F, D = 2.0 ** -8, 2.0 ** -24, 2.0 ** -12


def scales(n):
    """n scales whose z is held worst by two bf16."""
    c = 1.0 + torch.rand(4096, generator=torch.Generator("cpu").manual_seed(5))

    def left(v):
        hi = v.to(torch.bfloat16).float()
        return v - hi - (v - hi).to(torch.bfloat16).float()
    worst = ((left(c) - left(c * (1 + D))).abs() / c).topk(n).indices
    return c[worst].to(DEV)


def zeros(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16, device=DEV)


def values(seed, n):
    g = torch.Generator("cpu").manual_seed(seed)
    return (1.0 + torch.rand(n, generator=g)).to(torch.bfloat16).to(DEV)


def check(got, left, right):
    """got [.., ..] is left @ right (float64, every factor c z or c g exact)."""
    ref, m = left @ right, left.abs() @ right.abs()
    n = int((left != 0).sum(1).max())
    err = (got.double() - ref).abs()
    bound = H * ref.abs() + (1 + 6 * n) * F * m
    ok = bool((err <= bound).all())
    assert ok, ((err - H * ref.abs()) / m.clamp_min(1e-30)).max().log2().item()


# a token to a slot and tiles of 16 in one launch, after a grouping, and tiles of 64 whose z
# each workgroup adds up or finish_kernel does; ranks of one chunk of 32 to eight
@pytest.mark.parametrize("T,N,K,r,n", [(3, 40, 8, 16, 3), (3, 40, 8, 64, 3), (40, 40, 8, 16, 3), (40, 40, 8, 256, 3), (600, 40, 8, 16, 3),
                                       (1600, 30000, 72, 32, 1), (1600, 30000, 1160, 32, 1), (1100, 12000, 264, 256, 2), (450, 4104, 4096, 48, 2)])
def test_add(gpu_lib, T, N, K, r, n):
    vt, u = zeros(n, r, K), zeros(n, N, r)
    vt[:, :2, 0], vt[:, 1, 1] = 1.0, D
    u[:, :, 0], u[:, :, 1] = values(2, N), -values(2, N)
    p = binding.AdapterPool(vt, u, scales(n), (N,))
    x, index = zeros(T, K), (torch.arange(T) % n).to(torch.int32).to(DEV)
    x[:, :2] = (2.0 ** (torch.arange(T, device=DEV) % 5))[:, None]
    y = p.add(x, index, zeros(T, N))
    for a in range(n):
        on = index == a
        z = p.scale[a].double() * (x[on].double() @ vt[a].double().t().contiguous())
        check(y[on], z, u[a].double().t().contiguous())


# without the grouping, with it, few slots and many, z and g in slices and whole
SHAPES = [(4, 40, 8, 16, 2), (60, 40, 8, 64, 10), (600, 40, 8, 16, 100), (300, 700, 2600, 32, 50), (1300, 200, 520, 128, 200), (70, 2104, 2056, 32, 12)]


@pytest.mark.parametrize("T,N,K,r,n", SHAPES)
def test_dx(gpu_lib, T, N, K, r, n):
    vt, u = zeros(n, r, K), zeros(n, N, r)
    u[:, 0, :2], u[:, 1, 1] = 1.0, D
    vt[:, 0], vt[:, 1] = values(2, K), -values(2, K)
    p = binding.AdapterPool(vt, u, scales(n), (N,))
    dy, index = zeros(T, N), (torch.arange(T) % n).to(torch.int32).to(DEV)
    dy[:, :2] = (2.0 ** (torch.arange(T, device=DEV) % 5))[:, None]
    dx = p.backward(binding.encode_act(zeros(T, K)), dy, index, zeros(T, K), want=("dx",)).dx
    for a in range(n):
        on = index == a
        check(dx[on], p.scale[a].double() * (dy[on].double() @ u[a].double()), vt[a].double())


@pytest.mark.parametrize("T,N,K,r,n", SHAPES)
@pytest.mark.parametrize("which", ["du", "dv"])
def test_sums_over_tokens(gpu_lib, T, N, K, r, n, which):
    """Pairs of tokens of a slot: z (or g) c and c (1 + 2^-12), dy (or x) of opposite signs."""
    vt, u = zeros(n, r, K), zeros(n, N, r)
    vt[:, 0, :2], u[:, :2, 0] = 1.0, 1.0
    p = binding.AdapterPool(vt, u, scales(n), (N,))
    x, dy, index = zeros(T, K), zeros(T, N), (torch.arange(T) // 2 % n).to(torch.int32).to(DEV)
    thin, wide = (x, dy) if which == "du" else (dy, x)
    thin[:, 0], thin[1::2, 1] = 1.0, D
    # (one magnitude for all columns of x, whose block the checkpoint codes as one)
    wide[:] = values(3, N)[None, :] if which == "du" else 1.75
    wide[1::2] *= -1.0
    code = binding.encode_act(x)
    X = code.expand()
    assert torch.equal(X, x)                                    # the checkpoint holds these values exactly
    g = getattr(p.backward(code, dy, index, want=(which,)), which)
    for a in range(n):
        on = index == a
        if which == "du":
            z = p.scale[a].double() * (X[on].double() @ vt[a].double().t().contiguous())
            check(g[a], dy[on].double().t().contiguous(), z)
        else:
            check(g[a], (p.scale[a].double() * (dy[on].double() @ u[a].double())).t().contiguous(), X[on].double())
