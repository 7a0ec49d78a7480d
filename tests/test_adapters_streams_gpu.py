"""GPU: adapters whose rows are read past the caches, by tiles that are full and that are not."""
import pytest
import torch

from test_adapters_gpu import DEV, announce, check_add, make_pool, mixed_index, randn

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
