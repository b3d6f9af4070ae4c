"""The DRAM traffic that bench.py reports beside its roofline was measured on the kernel
sources that are in the tree: an edit of them asks for a new capture (the commands stand
in profiles/gemm_prefill_small_ncu.md and profiles/gemm_skewed_small_traffic_ncu.md)."""
import os
import sys

import pytest

from conftest import ROOT

sys.path.insert(0, ROOT)
import bench  # noqa: E402


@pytest.mark.parametrize("workload", ["prefill", "prefill_small", "skewed_small"])
def test_the_record_is_of_these_sources(workload):
    assert bench.ncu_traffic(workload) is not None


def test_profiles_that_are_of_these_sources_say_so():
    for name in ("gemm_prefill_small_ncu.md", "gemm_skewed_small_traffic_ncu.md", "launches_prefill.md"):
        with open(os.path.join(ROOT, "profiles", name)) as f:
            assert bench.kernel_source_hash() in f.read(), name
