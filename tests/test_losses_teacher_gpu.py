"""Distillation from teachers whose logits are far from 0, or at the type's lowest
value, against its definition in 64 bits (tests/loss_reference.py), on every way
that rows are laid out.

Bounds. As in tests/test_losses_gpu.py: F of the larger of a result's size and the
array's root mean square. log q and log p are differences of logits over the
temperature, less a logarithm: 2^-21 of their size for the roundings of each. p
and its target cancel in the gradient, 2^-19 of what they are before that.
"""
import pytest
import torch

from tests import loss_reference as ref
from tests.test_losses_gpu import close, cuda, gen
from tests.test_losses_range_gpu import LAYOUTS

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rl():
    assert torch.cuda.is_available(), "the -m gpu tests need a CUDA device"
    import linear_recurrence_scan_affine_gb300 as m
    return m


@pytest.mark.parametrize("K", [3, 20, 70])
@pytest.mark.parametrize("n,V", LAYOUTS)
def test_a_teachers_lowest_value(rl, n, V, K):
    # a teacher's entry at the type's lowest value has no weight, wherever it
    # stands and whatever the temperature makes of it; where all of them are
    # there, they are alike
    K = min(K, V)
    g = gen(V + K)
    x = torch.randn(n, V, generator=g) * 2.0
    ids = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(n)]).int()
    low = {d: torch.finfo(d).min for d in (torch.float32, torch.bfloat16)}
    for t in (0.5, 0.7, 1.0, 3.0):
        for value in low.values():
            top = torch.randn(n, K, generator=g)
            top[0, 0] = value
            top[1, K // 2:] = value
            top[2, :K - 1] = value
            if n > 3:
                top[3] = value
            w = torch.randn(n, generator=g)
            for whole in (False, True):
                lse = torch.logsumexp(top.double() / t, 1).clamp(min=-50.0).float() + 0.4
                cl = lse.cuda() if whole else None
                dx, loss = rl.rlcs_distill_loss_backward(*cuda(w, x, ids, top), temperature=t,
                                                         teacher_lse=cl, return_loss=True)
                x64 = x.double().requires_grad_()
                plain = top.clone()
                if n > 3 and not whole:  # the same q: -3.4e38 + log K is beyond 64 bits too
                    plain[3] = 0.0
                want = ref.distill(x64, ids, plain, lse if whole else None, temperature=t)
                size = 20.0 / t + 12.0  # of log p
                close("loss", loss, want, 2.0 ** -21 * size)
                wdx, = torch.autograd.grad((want * w.double()).sum(), x64)
                close("dlogits", dx, wdx, 2.0 ** -19 * (w.abs().double() / t)[:, None])


@pytest.mark.parametrize("K", [3, 70])
@pytest.mark.parametrize("n,V", LAYOUTS)
def test_a_teachers_common_offset(rl, n, V, K):
    # q depends on differences of the teacher's logits alone: an offset that is
    # exact moves the loss by nothing, and its roundings (4096 * 2^-24) by 2.4e-4
    K = min(K, V)
    g = gen(V + K)
    x = torch.randn(n, V, generator=g) * 2.0
    ids = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(n)]).int()
    top = (torch.randn(n, K, generator=g) * 16).round() / 8
    for t in (1.0, 0.7, 3.0):
        for off in (4096.0, -4096.0, 0.0):
            dx, loss = rl.rlcs_distill_loss_backward(*cuda(torch.ones(n), x, ids, top + off),
                                                     temperature=t, return_loss=True)
            x64 = x.double().requires_grad_()
            want = ref.distill(x64, ids, top, temperature=t)
            size = 20.0 / t + 12.0
            close("loss", loss, want, 2.0 ** -21 * size)
            wdx, = torch.autograd.grad(want.sum(), x64)
            close("dlogits", dx, wdx, 2.0 ** -20 / t)
