"""The benchmark's memory traffic comes from counter runs kept in profiles/: they
have to be runs of the present GEMM source."""
import os
import re

import pytest

import bench
from workloads import gen

CSRC = os.path.join(bench.ROOT, "orthogonalising_matrix_optimizer_amd", "csrc")


def _included(name, seen):
    seen.add(name)
    with open(os.path.join(CSRC, name)) as f:
        for other in re.findall(r'#include "([^"/]+)"', f.read()):
            if other not in seen:
                _included(other, seen)
    return seen


def test_the_source_hash_covers_what_the_kernels_include():
    assert _included("muon_gemm.hip", set()) == set(bench.GEMM_SOURCES)


@pytest.mark.parametrize("workload", sorted(bench.WORKLOADS))
def test_traffic_belongs_to_the_present_source(workload):
    """Counters of another source are retaken, or their file taken out."""
    if not os.path.exists(bench.traffic_file(workload)):
        pytest.skip("no counters kept for this set")
    ms = gen.SETS[workload]
    got = bench._traffic(workload, f"{workload}:{ms.steps}:{ms.coeffs}")
    assert got is not None
    assert got > sum(2 * r * c for r, c in ms.shapes)      # the written matrices alone
