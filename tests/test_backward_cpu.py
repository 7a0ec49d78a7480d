"""The backward entry points on the host: refusals that need no bundle, and the
layout of the gradient struct.  (Refusals that need a loaded bundle are in the
GPU tests: loading one enqueues work.)"""
import ctypes
import os

import pytest

from weight_shared_rank_amd import binding


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(binding.LIBPATH):
        from weight_shared_rank_amd import build
        build.build(verbose=False)
    return binding.lib()


def test_no_bundle(L):
    g = binding.WlGrads()
    assert L.weightless_backward_workspace_bytes(None, 4) == 0 and "NULL" in binding.last_error()
    for f in (L.weightless_linear_backward, L.weightless_stacked_backward):
        assert f(None, 0, 0, None, 0, None, 4, ctypes.byref(g), None, 0, None) == -1
        assert "bundle is NULL" in binding.last_error()
    assert L.weightless_stacked_backward(None, 0, -1, None, 0, None, 4, ctypes.byref(g), None, 0, None) == -4


def test_grads_struct_layout():
    """The C struct: nine pointers, then an int32 (padded to a pointer)."""
    assert ctypes.sizeof(binding.WlGrads) == 10 * ctypes.sizeof(ctypes.c_void_p)
    assert binding.WlGrads.dw0.offset == 8 * 8 and binding.WlGrads.accumulate_dw0.offset == 9 * 8
