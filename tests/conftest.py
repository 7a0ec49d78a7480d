import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU and the built HIP library")


# Tests of refusals with made-up device addresses: a refusal that got lost would launch a
# kernel on them, so they run only where no GPU is visible.
MADE_UP_ADDRESSES = {"test_coded_cpu.py", "test_norm_cpu.py", "test_adapters_cpu.py", "test_empty_calls_cpu.py",
                     "test_adapter_workspaces_cpu.py"}


def pytest_runtest_setup(item):
    if item.path.name in MADE_UP_ADDRESSES:
        import torch
        if torch.cuda.device_count():      # (counting does not initialise the GPU)
            pytest.skip("made-up device addresses: not where a GPU is visible")


@pytest.fixture(scope="session")
def gpu_lib():
    """The loaded HIP library; GPU tests fail loudly if it is not built."""
    import torch
    if not torch.cuda.is_available():
        pytest.fail("GPU test selected but no GPU is visible")
    from weight_shared_rank_amd import binding
    return binding.lib()
