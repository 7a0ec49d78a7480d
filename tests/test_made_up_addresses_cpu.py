"""Refusal tests with made-up device addresses stay off machines with a GPU."""
import os
import re
import types
from pathlib import Path

import pytest
import torch

import conftest

HERE = os.path.dirname(os.path.abspath(__file__))


def test_every_such_file_is_named():
    """A file says so by a constant A, an address."""
    found = {name for name in os.listdir(HERE) if name.endswith(".py")
             and re.search(r"^A = 1 << \d+", Path(HERE, name).read_text(), re.M)}
    assert found == conftest.MADE_UP_ADDRESSES


@pytest.mark.parametrize("devices", [0, 1])
def test_skipped_where_a_device_is_visible(monkeypatch, devices):
    monkeypatch.setattr(torch.cuda, "device_count", lambda: devices)
    for name in sorted(conftest.MADE_UP_ADDRESSES):
        item = types.SimpleNamespace(path=Path(HERE, name))
        if devices:
            with pytest.raises(pytest.skip.Exception):
                conftest.pytest_runtest_setup(item)
        else:
            conftest.pytest_runtest_setup(item)
    conftest.pytest_runtest_setup(types.SimpleNamespace(path=Path(HERE, "test_norm_gpu.py")))
