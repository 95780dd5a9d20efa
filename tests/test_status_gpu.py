"""The checks of device-side status wait for every stream before they read it."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rl():
    assert torch.cuda.is_available(), "the -m gpu tests need a CUDA device"
    import linear_recurrence_scan_affine_gb300 as m
    return m


def test_check_scratch_waits_for_other_streams(rl):
    g = torch.Generator().manual_seed(0)
    q, k = (torch.randn(300, h, 64, generator=g).bfloat16().cuda() for h in (4, 2))
    cu = torch.tensor([0, 300], dtype=torch.int32).cuda()
    big = torch.zeros(1 << 28, device="cuda")
    side = torch.cuda.Stream()
    rl.rlcs_attention(q, k, k, cu, stream=side)  # loads the kernel
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(100):  # some tens of milliseconds
            big.add_(1.0)
        rl.rlcs_attention(q, k, k, cu)
        done = side.record_event()
    assert not done.query()
    rl.check_scratch()
    assert done.query()


def test_check_all_workspaces_waits_for_other_streams(rl):
    r = torch.zeros(2, 40000, device="cuda")
    big = torch.zeros(1 << 28, device="cuda")
    side = torch.cuda.Stream()
    rl.rlcs_gae(r, r, r, stream=side)  # loads the kernel
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(100):
            big.add_(1.0)
        rl.rlcs_gae(r, r, r)
        done = side.record_event()
    assert not done.query()
    rl.check_all_workspaces()
    assert done.query()
