"""The committed counters of the GEMM kernel, which the benchmark reports only
while the kernel's sources are those that they were taken on."""
import importlib.util
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("profile", ["COUNTER_PROFILE", "MFMA_PROFILE"])
def test_taken_on_these_sources(profile):
    spec = importlib.util.spec_from_file_location("bench", os.path.join(ROOT, "bench.py"))
    bench = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(bench)
    with open(os.path.join(ROOT, getattr(bench, profile))) as f:
        digest = re.search(r'"source_digest": "(\w+)"', f.read()).group(1)
    assert digest == bench.gemm_source_digest()
