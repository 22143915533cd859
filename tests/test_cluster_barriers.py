"""Distributed shared memory may be touched only once every CTA of the cluster is known to have started: in each
kernel's source a barrier of the whole cluster stands before the first address in another CTA."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_scaled_mlp_gb300", "csrc")
BARRIER = re.compile(r"\bcluster_(?:sync|wait)\(\)")
REMOTE = re.compile(r"\bcluster_map\(|shared::cluster[.\w:]* \[")


def _kernels():
    """(file, name, body without comments) of every __global__ function."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        src = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"__global__\s+void\s+(?:__launch_bounds__\((?:[^()]|\([^()]*\))*\)\s*)?(\w+)\s*\((?=[^;{]*\{)", src):
            at = src.index("{", m.end())
            depth, i = 0, at
            while True:
                depth += {"{": 1, "}": -1}.get(src[i], 0)
                i += 1
                if depth == 0:
                    break
            yield os.path.basename(path), m.group(1), src[at:i]


USERS = [k for k in _kernels() if REMOTE.search(k[2])]


def test_finds_the_kernels_that_use_clusters():
    assert {(f, n) for f, n, _ in USERS} >= {("norm.cu", "add_rmsnorm_col_kernel"), ("ragged.cu", "ragged_kernel"),
                                             ("gemm.cu", "gemm_kernel")}


@pytest.mark.parametrize("file,name,body", USERS, ids=[n for _, n, _ in USERS])
def test_barrier_before_the_first_remote_access(file, name, body):
    first = BARRIER.search(body)
    assert first and first.start() < REMOTE.search(body).start(), f"{name} in {file}"
