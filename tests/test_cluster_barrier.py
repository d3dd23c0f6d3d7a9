"""Cluster barriers in the kernels' sources, on the host."""
import pathlib
import re

CSRC = pathlib.Path(__file__).resolve().parent.parent / "paged_kv_cache_230_gb300" / "csrc"


def test_warps_converge_before_an_aligned_cluster_barrier():
    """barrier.cluster in its aligned form is undefined where the lanes of a warp do not execute it together, and a lane
    that left a loop early may be ahead of the others: each such barrier follows a __syncwarp()."""
    found = 0
    for path in sorted(CSRC.glob("*.cu*")):
        lines = [line.strip() for line in path.read_text().splitlines()]
        for i, line in enumerate(lines):
            if not re.search(r"barrier\.cluster\.arrive\S*\.aligned", line):
                continue
            found += 1
            assert lines[i - 1] == "__syncwarp();", "%s:%d" % (path.name, i + 1)
    assert found
