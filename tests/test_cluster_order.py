"""Every kernel that runs as a cluster passes a cluster barrier before it touches another block's shared memory, and
another one after (no GPU needed: the order is read off the sources).

Until all blocks of a cluster have started, the shared memory of those that have not is not theirs yet; and a block
that has left gives its own back.  Neither __syncthreads nor griddepcontrol.wait orders the blocks of a cluster."""
import glob
import os
import re

import pytest

from dropless_mixture_experts_top_gb300 import _build

REMOTE = re.compile(r"(?:ld|st|red|atom)\.shared::cluster|\bld_cluster_\w+\s*\(|\bst_cluster_\w+\s*\(|"
                    r"\bmbar_arrive_cluster\s*\(|\btma_load_\dd_pair\s*\(|\btc_commit_pair\s*\(")
BARRIER = re.compile(r"\bcluster_(?:sync|wait)\s*\(\s*\)")
FULL = re.compile(r"\bcluster_sync\s*\(\s*\)")


def functions(text):
    """(name, body) of the __device__ and __global__ functions defined in a source."""
    text = re.sub(r"//[^\n]*", "", text)
    text = re.sub(r"__launch_bounds__\((?:[^()]|\((?:[^()]|\([^()]*\))*\))*\)", "", text)
    for m in re.finditer(r"__(?:global__|device__)\b[^;{}]*?\b(\w+)\s*\([^;{}]*\)\s*\{", text):
        depth, i = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
        yield m.group(1), text[m.end():i]


def users():
    found = []
    for path in sorted(glob.glob(os.path.join(_build.CSRC, "*.cu"))):
        for name, body in functions(open(path).read()):
            # (wrappers of a single instruction, and helpers that a kernel calls between its barriers, have none)
            if REMOTE.search(body) and ("cluster_sync" in body or "cluster_wait" in body):
                found.append((os.path.basename(path), name, body))
    return found


def test_the_cluster_kernels_are_found():
    names = {n for _, n, _ in users()}
    assert {"balance_finish_kernel", "block_colsum", "ortho_small_kernel", "ortho_gram_split_kernel",
            "ortho_product_kernel"} <= names


@pytest.mark.parametrize("path,name,body", [pytest.param(*u, id=u[1]) for u in users()])
def test_a_barrier_on_either_side_of_remote_memory(path, name, body):
    remote = [m.start() for m in REMOTE.finditer(body)]
    before = [m.start() for m in BARRIER.finditer(body)]
    after = [m.start() for m in FULL.finditer(body)]
    assert before[0] < remote[0], f"{path}: {name} reaches another block's memory before any cluster barrier"
    assert after[-1] > remote[-1], f"{path}: {name} may leave while another block reaches its memory"
