"""CPU check of the kernels' sources: a cluster's barrier in its `.aligned` form needs every thread of a warp to reach it together, which
the compiler does not promise behind a branch on the thread's number or on data; the warp meets right before it, or the plain form is used."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dspark_draft_selection_gb300", "csrc")


def test_warps_meet_before_aligned_cluster_barriers():
    used = []
    for path in sorted(glob.glob(os.path.join(CSRC, "*"))):
        lines = [x.split("//")[0].strip() for x in open(path).read().splitlines()]
        lines = [x for x in lines if x]
        for before, line in zip([""] + lines, lines):
            if re.search(r"barrier\.cluster\.", line):
                used.append((os.path.basename(path), "aligned" not in line or before == "__syncwarp();"))
    assert used                                              # the pattern finds the barriers that there are
    assert all(ok for _, ok in used), used
