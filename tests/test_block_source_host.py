"""Rules of the operators' device code that only show in its source: what a
GPU might answer to code that breaks them is a hang."""
import glob
import os
import re

import pytest

from conftest import ROOT

FILES = sorted(glob.glob(os.path.join(ROOT, "memory_bound_cnn_wtconv2d_gb300", "csrc", "block", "*.cu*")))


def functions_with(src, pattern):
    """(name, body) of the helper around each asm statement that matches: the text
    from the nearest line before it that opens a function at file level."""
    for m in re.finditer(pattern, src):
        head = [h for h in re.finditer(r"^(?:static |template.*\n)?(?:__device__|__global__)[^\n;]*?(\w+)\([^;{]*\)\s*\{", src[:m.start()],
                                       re.M)][-1]
        yield head.group(1), src[head.end():m.start()]


@pytest.mark.parametrize("path", FILES, ids=os.path.basename)
def test_aligned_instructions_follow_a_warp_barrier(path):
    # .aligned forms (bar.sync is one) are undefined on a warp whose lanes have parted
    src = re.sub(r"//[^\n]*", "", open(path).read())
    for name, before in functions_with(src, r'"[^"\n]*(?:\.aligned|bar\.sync)[^"\n]*"'):
        assert re.match(r"\s*__syncwarp\(\);", before), f"{os.path.basename(path)}: {name}"


def test_the_rule_sees_the_helpers():
    found = set()
    for path in FILES:
        src = re.sub(r"//[^\n]*", "", open(path).read())
        found |= {n for n, _ in functions_with(src, r'"[^"\n]*(?:\.aligned|bar\.sync)[^"\n]*"')}
    assert {"cluster_arrive", "cluster_wait", "cluster_sync", "named_sync", "tmem_alloc", "tmem_free", "tmem_load8",
            "tmem_wait_load"} <= found


def test_fences_and_commits_cover_the_elected_lane():
    # which lane elect.sync picks is not promised: what it issues is committed by
    # an elected lane too, and fenced by every lane of its warp
    src = re.sub(r"//[^\n]*", "", open([p for p in FILES if p.endswith("/ns.cu")][0]).read())
    for m in re.finditer(r"mma_commit\(", src):
        guard = src[:m.start()].rsplit("if (", 2)[-1]
        assert "elect_one()" in src[:m.start()][-900:] and "lane == 0" not in guard.split("{")[0]
    barrier = src[src.index("bool grid_barrier"):]
    barrier = barrier[:barrier.index("return !stop")]
    after = barrier[barrier.index("__syncthreads_or"):]
    assert re.search(r"warp == 0 \|\| warp == 10", after) and "threadIdx.x == 0" not in after
