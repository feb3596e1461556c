"""CPU check of the kernels' sources: a cluster's barrier in its `.aligned` form needs every thread of a warp to reach it together, which
the compiler does not promise behind a branch on the thread's number or on data; the plain form may be reached by each thread for itself."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dspark_draft_selection_gb300", "csrc")


def test_cluster_barriers_ask_for_no_converged_warp():
    used = []
    for path in sorted(glob.glob(os.path.join(CSRC, "*"))):
        for line in open(path).read().splitlines():
            used += [(os.path.basename(path), x) for x in re.findall(r"barrier\.cluster\.\w+[.\w]*", line.split("//")[0])]
    assert used                                              # the pattern finds the barriers that there are
    assert [u for u in used if "aligned" in u[1]] == []
