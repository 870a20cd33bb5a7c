"""Rules of the gated product's device code that only show in its source: what a
GPU might answer to code that breaks them is a write to the shared memory of a CTA
that has left."""
import os
import re

from conftest import ROOT

PATH = os.path.join(ROOT, "memory_bound_cnn_wtconv2d_gb300", "csrc", "block", "gated_kernels.cuh")


def source():
    return re.sub(r"//[^\n]*", "", open(PATH).read())


def body(src, name):
    """The text between the braces of the function `name`."""
    at = src.index("{", re.search(r"\b" + name + r"\([^;{]*\)\s*\{", src).start())
    depth = 0
    for i in range(at, len(src)):
        depth += {"{": 1, "}": -1}.get(src[i], 0)
        if not depth:
            return src[at:i]
    raise AssertionError(name)


def test_every_barrier_that_a_commit_arrives_at_is_waited_for_in_both_ctas():
    # a pair's commits arrive at the barriers of both CTAs, and neither may leave before
    src = source()
    multiply = body(src, "multiply")
    at = set(re.findall(r"commit\((?:smem_addr\(&sh\.)?(\w+)", multiply)) - {"bar"}
    assert at == {"empty", "acc_full", "drain"}
    # the products' last k blocks: by the warp of the copies, whatever its rank
    produce = body(src, "produce")
    end = produce[produce.rindex("if (w.rank == 0) {"):]
    end = end[end.index("}") + 1:]  # behind what is the first CTA's alone
    assert re.search(r"for \([^)]*\)\s*drain\(a, &sh\.empty\[s\]", end)
    assert "else" not in end and re.search(r"if \(!ok \|\| sh\.dead\) linger\(a\);", end)
    # the last commit: the second CTA's by that warp too, the first one's by the MMAs' warp
    assert re.search(r"linger\(a\);\s*if \(w\.rank\) drain\(a, &sh\.drain, 0\);\s*$", end)
    assert re.search(r"commit\(smem_addr\(&sh\.drain\)\);\s*drain\(a, &sh\.drain, 0\);\s*\}\s*__syncwarp\(\);\s*$", multiply)
    # the tiles: by every epilogue warp
    assert "wait(sh, a, &sh.acc_full[acc], phase)" in body(src, "epilogue")
    # and the two meet before either leaves
    kernel = body(src, "gated_gemm")
    assert re.search(r"__syncthreads\(\);\s*if constexpr \(PAIR\) cluster_meet\(\);", kernel[kernel.index("epilogue<"):])
