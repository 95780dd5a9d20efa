"""Linear attention without a GPU: what its source has to keep to, and the limits
of its sizes in the C ABI."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = os.path.join(ROOT, "linear_recurrence_scan_affine_gb300", "csrc", "seq_linear.cu")


def code():
    text = open(SOURCE).read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def test_no_wait_between_warps_is_without_a_limit():
    # After a wait that ran out the warps of a block may leave units at different
    # places: a barrier that counts on all of them would never open. Only the
    # barriers that every thread of a block comes to stand outside a unit's work.
    src = code()
    assert not re.search(r"\b(bar|barrier)\.(cta\.)?(sync|arrive|red)", src)
    assert "mbar_try_wait" not in src and "mbarrier.try_wait" not in src
    walk = src[src.index("linear_walk_kernel(const"):src.index("struct SumArgs")]
    work = walk[walk.index("if (warp == 16) {"):walk.rindex("tc::fence_before_sync();")]
    assert "__syncthreads" not in work
