"""Calls without tokens write zeros to gradients, so their outputs must not meet an input
either (nothing is enqueued: every call below is refused)."""
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


@pytest.mark.parametrize("out", ["du", "dv"])
@pytest.mark.parametrize("over", [A, 2 * A, 3 * A, 4 * A, 2 * A - 16])
def test_adapter_gradients_over_the_pool(L, out, over):
    p = binding.WlAdapters(4, 32, 256, 2, (ctypes.c_int32 * 3)(512, 256, 0), A, 2 * A, 3 * A, 4 * A)
    g = binding.WlAdapterGrads(None, None, over if out == "du" else 10 * A, over if out == "dv" else 11 * A)
    assert L.weightless_adapters_backward(ctypes.byref(p), None, 0, None, None, 0, ctypes.byref(g), None, 0, None) == -1
    assert "overlap" in binding.last_error()


@pytest.mark.parametrize("over", [4 * A, 4 * A + 512])
def test_norm_gradient_over_the_weight(L, over):
    assert L.weightless_norm_backward(None, None, None, None, 0, 256, 4 * A, 1, 0.0, None, over, None, 0, None) == -1
    assert "overlap" in binding.last_error()
