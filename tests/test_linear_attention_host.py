"""Linear attention without a GPU: what its source has to keep to, and the limits
of its sizes in the C ABI."""
import ctypes
import os
import re

from linear_recurrence_scan_affine_gb300 import binding, sequence  # noqa: F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = os.path.join(ROOT, "linear_recurrence_scan_affine_gb300", "csrc", "seq_linear.cu")
INVALID, BF16 = 1, 1
lib = binding.lib()


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


def test_token_counts_past_whole_chunks_are_refused():
    # a segment's length, whole chunks of 128 tokens, has to fit an int
    most = 2 ** 31 - 128
    need = lib.rlcs_linear_attention_scratch_bytes
    assert need(1, most, 1, 1, 8) > 0 and need(300, most, 2, 1, 8) > 0
    for n in (most + 1, 2 ** 31 - 1, 2 ** 31):
        assert need(1, n, 1, 1, 8) == 0
        q, k, v, ld, cu, out, scratch = (ctypes.c_void_p(0x7f0000000000 + (i << 36))
                                         for i in range(7))
        views = (q, 8, 8, k, 8, 8, v, 8, 8, ld, cu, None)
        assert lib.rlcs_linear_attention(*views, out, None, 1, n, 1, 1, 8, 1.0, BF16, scratch,
                                         1 << 30, None) == INVALID
        dq, dk, dv = (ctypes.c_void_p(0x7f0000000000 + (i << 36)) for i in range(7, 10))
        assert lib.rlcs_linear_attention_backward(out, *views, None, dq, dk, dv, None, 1, n, 1, 1,
                                                  8, 1.0, BF16, scratch, 1 << 30, None) == INVALID
