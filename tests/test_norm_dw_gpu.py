"""GPU: the norm's weight gradient, with a bound that a lost row or workgroup breaks.

dw[k] = sum_t dy n, in float32.  Each rounding is 2^-24 of a partial sum of the magnitudes
at most, so the error is at most (depth + 2) 2^-24 sum_t |dy n|, where depth is how many
additions a term passes through and 2 stands for n's and the sum's own:
  more than 1024 rows: a team's rows in turn (of 256 teams or more), 3 additions of a
    workgroup's waves, the partial sums of up to 768 workgroups 16 at a time (48), 15 more
  fewer: 8 rows a wave in turn (2 waves or more, 4 for the shortest rows), 3 within a wave,
    15 between waves
The roundings are independent, each of a partial sum that grows as the square root of its
rows as dw itself does, so the error's norm stays below 4 (sqrt(depth) + 1) 2^-25 of dw's."""
import pytest
import torch

from test_norm_gpu import F, announce, randn
from weight_shared_rank_amd import binding

pytestmark = pytest.mark.gpu


def depth(T):
    return -(-T // 256) + 3 + 48 + 15 if T > 1024 else -(-T // 16) + 3 + 15


def dw_is_near(got, dy, n):
    """got against the sum over rows of dy n (float64)."""
    ref, mag, d = (dy * n).sum(0), (dy * n).abs().sum(0), depth(dy.shape[0])
    err = (got.double() - ref).abs()
    return bool((err <= (d + 2) * F * mag + 1e-45).all()) and \
        (ref.numel() < 64 or bool(err.norm() <= 4 * (d ** 0.5 + 1) * 2.0 ** -25 * ref.norm()))


SHAPES = [(5, 64), (300, 256), (333, 1160), (1000, 5376), (1024, 21504),                # one launch
          (1100, 64), (5000, 256), (4100, 512), (2000, 1000), (2500, 2048), (1100, 2056), (1500, 4096), (1300, 5376), (1200, 8192),
          (1200, 12000), (1030, 21504), (1030, 32768),                                   # a sum of the workgroups' sums
          (70000, 512), (36000, 1000), (20000, 2048), (20000, 2056), (9000, 5376), (6000, 8192), (3600, 12000), (2400, 24584)]  # past the caches


@pytest.mark.parametrize("T,K", SHAPES)
def test_dw(gpu_lib, T, K):
    announce(f"norm dw {T} x {K}")
    dy, h, w = randn(1, T, K), randn(2, T, K, std=2.0), randn(3, K)
    a = binding.norm_act(h, w, want=("rstd",)).rstd
    o = binding.norm_backward(dy, h, a, w, 1.0, dy)
    assert dw_is_near(o.dw, dy.double(), h.double() * a.double()[:, None])
