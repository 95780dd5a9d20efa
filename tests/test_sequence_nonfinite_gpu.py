"""A state or a gradient of the gated linear recurrence that is not finite
stays so to the end of its episode, however the call's steps are shared out
and however small the product of its gates has become."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rl():
    assert torch.cuda.is_available(), "the -m gpu tests need a CUDA device"
    import linear_recurrence_scan_affine_gb300 as m
    return m


# walks by a cluster's blocks (several windows of them too), by one block, by warps alone
SHAPES = [(1, 20000, 64), (1, 5000, 40), (2, 4099, 520), (1, 700, 34), (30, 1500, 65),
          (800, 1500, 3)]


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("B,T,D", SHAPES)
def test_a_state_that_is_not_finite_stays(rl, B, T, D, bad):
    g = torch.Generator().manual_seed(T + D)
    x, dh = (torch.randn(B, T, D, generator=g) for _ in range(2))
    gate = torch.randn(B, T, D, generator=g) * 0.5 + 1.0  # about 0.7 carried each step
    cx, cg, cd = x.cuda(), gate.cuda(), dh.cuda()
    clean, clean_last = rl.rlcs_gated_scan(cx, cg)
    dx0, dg0, dh00 = rl.rlcs_gated_scan_backward(cd, cx, cg, clean)

    x2 = cx.clone()
    x2[0, 2, 1] = bad  # one channel of one sequence, near the start
    h, last = rl.rlcs_gated_scan(x2, cg)
    want = clean.clone()
    want[0, 2:, 1] = bad
    assert torch.equal(torch.nan_to_num(h, nan=7e9), torch.nan_to_num(want, nan=7e9))
    want_last = clean_last.clone()
    want_last[0, 1] = bad
    assert torch.equal(torch.nan_to_num(last, nan=7e9), torch.nan_to_num(want_last, nan=7e9))

    h0 = torch.zeros(B, D).cuda()
    h0[0, 1] = bad
    h, last = rl.rlcs_gated_scan(cx, cg, h0=h0)
    want[0, :, 1] = bad
    assert torch.equal(torch.nan_to_num(h, nan=7e9), torch.nan_to_num(want, nan=7e9))
    assert torch.equal(torch.nan_to_num(last, nan=7e9), torch.nan_to_num(want_last, nan=7e9))

    d2 = cd.clone()
    d2[0, T - 3, 1] = bad  # near the end: every step before it
    dx, dg, dh0 = rl.rlcs_gated_scan_backward(d2, cx, cg, clean)
    want = dx0.clone()
    want[0, :T - 2, 1] = bad
    assert torch.equal(torch.nan_to_num(dx, nan=7e9), torch.nan_to_num(want, nan=7e9))
    assert not torch.isfinite(dg[0, :T - 2, 1]).any() and torch.isfinite(dg[0, :, 0]).all()
    assert not torch.isfinite(dh0[0, 1]) and torch.equal(dh0[:, 0], dh00[:, 0])
    last_grad = torch.zeros(B, D).cuda()
    last_grad[0, 1] = bad
    dx, _, dh0 = rl.rlcs_gated_scan_backward(cd, cx, cg, clean, dh_last=last_grad)
    want[0, :, 1] = bad
    assert torch.equal(torch.nan_to_num(dx, nan=7e9), torch.nan_to_num(want, nan=7e9))
    assert not torch.isfinite(dh0[0, 1])


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("B,T,D", SHAPES)
def test_a_cut_still_ends_it(rl, B, T, D, bad):
    g = torch.Generator().manual_seed(T + D)
    x, dh = (torch.randn(B, T, D, generator=g) for _ in range(2))
    gate = torch.randn(B, T, D, generator=g) * 0.5 + 1.0
    reset = torch.zeros(B, T, dtype=torch.bool)
    at = T - 9  # long after what is carried has shrunk to nothing
    reset[:, at] = True
    cx, cg, cd, cr = (t.cuda() for t in (x, gate, dh, reset))
    clean, clean_last = rl.rlcs_gated_scan(cx, cg, reset=cr)
    grads = rl.rlcs_gated_scan_backward(cd, cx, cg, clean, reset=cr)
    x2, d2 = cx.clone(), cd.clone()
    x2[:, 2] = bad
    h, last = rl.rlcs_gated_scan(x2, cg, reset=cr)
    assert torch.equal(h[:, at:], clean[:, at:]) and torch.equal(last, clean_last)
    assert torch.equal(h[:, :2], clean[:, :2]) and not torch.isfinite(h[:, 2:at]).any()
    d2[:, T - 2] = bad
    got = rl.rlcs_gated_scan_backward(d2, cx, cg, clean, reset=cr)
    for a, b in zip(got[:2], grads[:2]):
        assert torch.equal(a[:, :at], b[:, :at]) and not torch.isfinite(a[:, at:T - 1]).any()
    assert torch.equal(got[2], grads[2])
