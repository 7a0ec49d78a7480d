"""The bound of test_norm_dw_gpu.py on the host: float32 sums stay within it, and a sum that
lacks one team's rows, one workgroup's or a single row does not."""
import pytest
import torch

from test_norm_dw_gpu import dw_is_near


def teams_sum(dy, n, teams, lost=None):
    """dw as the kernels add it up: a team's rows in turn, then the teams'."""
    T, K = dy.shape
    part = torch.zeros(teams, K)
    for t0 in range(0, T, teams):
        m = min(teams, T - t0)
        part[:m] += dy[t0:t0 + m] * n[t0:t0 + m]
    if lost is not None:
        part[lost] = 0
    out = torch.zeros(16, K)
    for i in range(0, teams, 16):
        out[:min(16, teams - i)] += part[i:i + 16]
    return out.sum(0)


@pytest.mark.parametrize("T,K,teams,group", [(36000, 64, 768, 1), (20000, 64, 768, 1), (70000, 64, 2560, 4), (2000, 64, 768, 1), (1030, 64, 256, 1), (300, 64, 32, 1)])
def test_a_lost_part_shows(T, K, teams, group):
    g = torch.Generator().manual_seed(T)
    dy, n = torch.randn(T, K, generator=g).bfloat16().float(), torch.randn(T, K, generator=g).bfloat16().float()
    d64, n64 = dy.double(), n.double()
    assert dw_is_near(teams_sum(dy, n, teams), d64, n64)
    lost = list(range(8, 8 + group))
    assert not dw_is_near(teams_sum(dy, n, teams, lost), d64, n64)
    one = (d64 * n64).sum(0) - d64[T // 2] * n64[T // 2]
    assert not dw_is_near(one.float(), d64, n64)
