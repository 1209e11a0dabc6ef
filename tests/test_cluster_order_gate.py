"""The gate's kernels read the shared memory of other blocks of their cluster only between cluster barriers (no GPU needed: the
order is read off the sources, as in test_cluster_order.py, for the reads by way of ld_peer)."""
import os
import re

import pytest

from dropless_mixture_experts_top_gb300 import _build
from tests.test_cluster_order import functions

REMOTE, BARRIER = re.compile(r"\bld_peer\s*\("), re.compile(r"\bcluster_(sync|wait)\s*\(\s*\)")


@pytest.mark.parametrize("path,kernel", [("gate.cuh", "gate_select_kernel"), ("gate.cu", "gate_index_kernel")])
def test_remote_reads_lie_between_barriers(path, kernel):
    bodies = [b for n, b in functions(open(os.path.join(_build.CSRC, path)).read()) if n == kernel]
    assert len(bodies) == 1
    remote = [m.start() for m in REMOTE.finditer(bodies[0])]
    barriers = [m.start() for m in BARRIER.finditer(bodies[0])]
    assert remote and barriers[0] < remote[0] and barriers[-1] > remote[-1]
    if "cluster_wait" in bodies[0][barriers[-1]:]:  # the arrival that this wait is for comes after the last read
        assert bodies[0].rindex("cluster_arrive") > remote[-1]
