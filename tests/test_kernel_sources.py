"""Rules that the CUDA sources keep and that no run can show to be broken (a run that breaks one may hang): read from
the sources."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "two_level_sparse_quest_b200", "csrc")


def sources():
    for name in sorted(os.listdir(CSRC)):
        if name.endswith((".cu", ".cuh")):
            with open(os.path.join(CSRC, name)) as f:
                yield name, re.sub(r"//[^\n]*", "", f.read())


def test_aligned_cluster_barriers_converge_the_warp_first():
    """barrier.cluster.*.aligned is executed by whole warps; its callers come from loops over a share of the outputs
    and from predicated loads, so the warp is converged directly before each of them."""
    seen = 0
    for name, text in sources():
        for m in re.finditer(r'asm volatile\(\s*"barrier\.cluster\.[a-z.]*aligned;"', text):
            seen += 1
            assert re.search(r"__syncwarp\(\);\s*$", text[:m.start()]), (name, text[max(0, m.start() - 80):m.end()])
    assert seen >= 3
