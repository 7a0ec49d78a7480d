"""A workspace sized for more tokens can be too small for fewer, as the header says: the call
refuses it (nothing is enqueued: every call below is refused)."""
import ctypes
import os

import pytest

from weight_shared_rank_amd import binding

A = 1 << 36          # never dereferenced


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(binding.LIBPATH):
        from weight_shared_rank_amd import build
        build.build(verbose=False)
    return binding.lib()


@pytest.mark.parametrize("n,r,K,rows,fewer,more", [(4, 64, 512, (512, 0, 0), 256, 257), (2, 256, 512, (512, 512, 512), 40, 41)])
def test_backward(L, n, r, K, rows, fewer, more):
    p = binding.WlAdapters(n, r, K, sum(v > 0 for v in rows), (ctypes.c_int32 * 3)(*rows), A, 2 * A, 3 * A, None)
    need = [L.weightless_adapters_backward_workspace_bytes(ctypes.byref(p), T) for T in (fewer, more)]
    assert need[0] > need[1]
    g = binding.WlAdapterGrads(8 * A, 9 * A, 10 * A, 11 * A)
    assert L.weightless_adapters_backward(ctypes.byref(p), 5 * A, 1 << 40, 6 * A, 7 * A, fewer, ctypes.byref(g), 12 * A, need[1], None) == -5
    assert "workspace" in binding.last_error()
