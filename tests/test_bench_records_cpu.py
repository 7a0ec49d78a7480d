"""The bench's HBM traffic records (profiles/counters.json) belong to the sources they were
taken on: the bench finds them, or reports no traffic."""
import os
import re

import pytest

import bench


def sources(key):
    """The sources that bench.py names beside traffic_from_profile(key, ...)."""
    text = open(os.path.join(bench.ROOT, "bench.py")).read()
    names = re.search(r"source_sha\(([^)]*)\)\s*\n[^\n]*traffic_from_profile\(\"%s\"" % key, text).group(1)
    return re.findall(r'"([^"]+)"', names)


@pytest.mark.parametrize("key", ["decode", "prefill"])
def test_traffic_is_found(key):
    total, read, written = bench.traffic_from_profile(key, bench.source_sha(*sources(key)))
    assert total and read and written and total == read + written
