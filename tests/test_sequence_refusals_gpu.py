"""Refusals of the sequence operators that need tensors on a GPU to reach."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rl():
    assert torch.cuda.is_available(), "the -m gpu tests need a CUDA device"
    import linear_recurrence_scan_affine_gb300 as m
    return m


def test_heads_of_no_width_are_refused(rl):
    q = torch.zeros(4, 2, 0, dtype=torch.bfloat16).cuda()
    cache = torch.zeros(4, 3, 2, 0, dtype=torch.bfloat16).cuda()
    cu = torch.tensor([0, 4], dtype=torch.int32).cuda()
    with pytest.raises(rl.RlcsError):
        rl.rlcs_attention(q, q, q, cu)
    with pytest.raises(rl.RlcsError):
        rl.rlcs_attention_backward(q, q, q, q, q, torch.zeros(2, 4).cuda(), cu)
    with pytest.raises((rl.RlcsError, ValueError)):
        rl.rlcs_attention_step(q, cache, cache, torch.ones(4, dtype=torch.int32).cuda())


def test_sizes_that_need_no_scratch_are_refused_by_the_library(rl):
    q = torch.zeros(4, 0, 64, dtype=torch.bfloat16).cuda()
    k = torch.zeros(4, 1, 64, dtype=torch.bfloat16).cuda()
    cu = torch.tensor([0, 4], dtype=torch.int32).cuda()
    with pytest.raises(rl.RlcsError):
        rl.rlcs_attention(q, k, k, cu)
    wide = torch.zeros(2, 1, 1032).cuda()
    w, table = torch.ones(1032).cuda(), torch.ones(4, 2).cuda()
    pos = torch.zeros(2, dtype=torch.int32).cuda()
    with pytest.raises(rl.RlcsError):
        rl.rlcs_qk_norm_rope_backward(wide, wide, wide, wide, w, w, table, table, pos)
