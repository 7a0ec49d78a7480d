"""GPU: adapters whose rows, or whose dy, are read past the caches, and the same beside them."""
import pytest
import torch

from test_adapters_backward_gpu import check as check_gradients
from test_adapters_gpu import DEV, announce, check_add, make_pool, mixed_index, randn
from weight_shared_rank_amd import binding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [16, 33, 200, 600])
@pytest.mark.parametrize("kind", ["one slot", "two slots", "mixed"])
def test_full_tiles_beside_others(gpu_lib, T, kind):
    """A pool of 40 slots of rank 16 and 30000 rows: its U is larger than what the caches keep."""
    announce(f"adapters past the caches T={T} {kind}")
    p = make_pool(40, 16, 136, (29999, 1), ranks=[(16, 5, 0)[i % 3] for i in range(40)])
    index = {"one slot": torch.full((T,), 3), "two slots": torch.where(torch.arange(T) % 3 == 0, 1, 6)}.get(kind)
    index = mixed_index(T, 40, 2) if index is None else index.to(torch.int32).to(DEV)
    x, base = randn(1, T, 136), randn(2, T, 30000)
    y = p.add(x, index, base)
    check_add(p, x, index, base, y)
    again = base.clone()
    assert torch.equal(p.add(x, index, again, y=again).view(torch.int16), y.view(torch.int16))


# dy past 64 MB (read past the caches where one group of ranks reads it), and below
@pytest.mark.parametrize("T,rows,K,r,n", [(1700, (40001,), 72, 16, 8), (1700, (40000, 9), 72, 32, 7), (1700, (40001,), 72, 64, 8), (1700, (40000,), 72, 128, 4),
                                          (800, (40001,), 72, 16, 8), (800, (40000, 9), 72, 32, 7), (800, (40001,), 72, 64, 8)])
def test_gradients_of_a_large_dy(gpu_lib, T, rows, K, r, n):
    announce(f"adapters backward T={T} rows={rows} K={K} r={r} n={n}")
    p = make_pool(n, r, K, rows, ranks=[(r, r // 2, 1, 0)[i % 4] for i in range(n)])
    code, dy, base = binding.encode_act(randn(7, T, K)), randn(8, T, sum(rows), std=T ** -0.5), randn(10, T, K, std=T ** -0.5)
    index = mixed_index(T, n, 9)
    index[: T // 3] = 0
    g = p.backward(code, dy, index, base)
    check_gradients(p, code, dy, index, base, g)
    assert torch.equal(p.backward(code, dy, index, want=("du",)).du, g.du)
