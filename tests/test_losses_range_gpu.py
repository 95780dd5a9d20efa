"""The losses where logits are large, against their definitions in 64 bits
(tests/loss_reference.py), on every way that rows are laid out: a thread, lanes or
a warp to a row, a block, a cluster, a row read twice.

Bounds. As in tests/test_losses_gpu.py: F of the larger of a result's size and
the array's root mean square. A log probability is a difference of logits, each
exact, over the temperature: 2^-22 of its size, for the difference, the
reciprocal of the temperature and its product, and 2^-20 for log z. An entropy
is log z less a mean exponent, both off by a few roundings, 8 of 2^-24 in all, of
what a row's exponents are from 0: up to 2^-24 of the logits' own size in powers
of two, 32 at most.
"""
import math

import pytest
import torch

from tests import loss_reference as ref
from tests.test_losses_gpu import DT, F, close, cuda, gen

pytestmark = pytest.mark.gpu

# (tokens, V): a thread, 8 lanes, a warp, a block, a cluster, twice (float32, bfloat16)
LAYOUTS = [(400, 6), (5, 20), (6, 700), (6, 5000), (4, 70000), (3, 140001), (3, 270001)]


@pytest.fixture(scope="module")
def rl():
    assert torch.cuda.is_available(), "the -m gpu tests need a CUDA device"
    import linear_recurrence_scan_affine_gb300 as m
    return m


def crowd(g, n, V, at, dtype):
    """Logits [n, V] whose largest are `at` and up to a few places of the type
    below it, others far below, and which of them are near the top."""
    top = torch.tensor(float(at), dtype=torch.float64).to(DT[dtype])
    step = torch.finfo(DT[dtype]).eps * 2.0 ** math.floor(math.log2(abs(float(top))))
    places = torch.randint(0, 4, (n, V), generator=g).double()
    near = torch.rand(n, V, generator=g) < max(0.3, 3.0 / V)
    near[torch.arange(n), torch.randint(0, V, (n,), generator=g)] = True
    x = float(top) - places * step
    x = torch.where(near, x, x - abs(float(top)) * (0.5 + torch.rand(n, V, generator=g)))
    return x.to(DT[dtype]), near


def some(g, near, k=1):
    """k columns of each row among those near its top."""
    return torch.stack([r.nonzero()[:, 0][torch.randint(0, int(r.sum()), (k,), generator=g)]
                        for r in near]).int()


SIZES = [1e7, 2e7, -2e7, 1e8, -3e8, 7e8, 3e9, -3e9, 5e9, -1e10, 1e20, -1e20, 1e30, -1e30, 1e38,
         -2e38]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,V", LAYOUTS)
def test_policy_of_large_logits(rl, n, V, dtype):
    for i, at in enumerate(SIZES if V < 100000 else SIZES[::3]):
        g = gen(V + i)
        x, near = crowd(g, n, V, at, dtype)
        a = some(g, near)[:, 0]
        l = ref.logs(x).gather(1, a.long()[:, None])[:, 0]
        old = torch.where(l > -1e4, l - 0.05, l).float()
        adv, w = torch.randn(n, generator=g), torch.randn(n, generator=g)
        dx, got = rl.rlcs_policy_loss_backward(*cuda(w, x, a, old, adv), entropy_coef=0.1,
                                               return_loss=True)
        x64 = x.double().requires_grad_()
        want = ref.policy(x64, a, old, adv, ent=0.1)
        off = (got.logp.double().cpu() - l).abs()
        assert bool((off <= 2.0 ** -20 + 2.0 ** -22 * l.abs()).all()), (at, float(off.max()))
        from_0 = min(32.0, abs(at) * 1.45 * 2.0 ** -24)
        close("entropy %g" % at, got.entropy, want[2], 2.0 ** -20 + 2.0 ** -21 * from_0)
        # what a ratio moves by: the log probability's error, and with |l| past
        # 2^10 `old` itself stands for no distance any more
        fine = (l > -1e3) | (l - old.double() == 0)
        lost = (2.0 ** -20 + 2.0 ** -22 * l.abs()) * 2.0
        close("loss %g" % at, got.loss[fine.cuda()], want[0][fine], (lost * adv.abs())[fine])
        wdx, = torch.autograd.grad((want[0] * w.double()).sum(), x64)
        slope = ((lost + F) * w.abs() * (adv.abs() + 0.1))[:, None]
        close("dlogits %g" % at, dx[fine.cuda()], wdx[fine], slope[fine])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,V", LAYOUTS)
def test_an_action_far_below(rl, n, V, dtype):
    # a log probability is as exact as the logits' difference, whatever z is made with
    for at in (3e7, -1e10, 1e30):
        g = gen(V)
        x, near = crowd(g, n, V, at, dtype)
        x[:, V // 2], near[:, V // 2] = -3.0 * abs(at), False
        a = torch.full((n,), V // 2, dtype=torch.int32)
        want = ref.logs(x)[:, V // 2]
        one = torch.ones(n)
        got = rl.rlcs_policy_loss(*cuda(x, a, want.float(), one)).logp.double().cpu()
        assert bool(((got - want).abs() <= 2.0 ** -22 * want.abs()).all()), at


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,V", LAYOUTS)
def test_rows_filled_with_a_mask_value(rl, n, V, dtype):
    # all alike, whatever the value; and one left above it
    for fill in (-1e9, -1e10, -1e20, -1e30, 5e9):
        x = torch.full((n, V), fill).to(DT[dtype])
        a = torch.zeros(n, dtype=torch.int32)
        a[1::2] = V - 1
        x[1::2, V - 1] = abs(fill) if fill < 0 else 2 * fill
        one, old = torch.ones(n), ref.logs(x).gather(1, a.long()[:, None])[:, 0].float()
        dx, got = rl.rlcs_policy_loss_backward(*cuda(one, x, a, old, one), entropy_coef=0.1,
                                               return_loss=True)
        x64 = x.double().requires_grad_()
        want = ref.policy(x64, a, old, one, ent=0.1)
        close("logp", got.logp, want[1], 2.0 ** -20 + 2.0 ** -22 * want[1].abs().detach())
        close("entropy", got.entropy, want[2], 2.0 ** -20)
        close("loss", got.loss, want[0], 2.0 ** -18)
        close("dlogits", dx, torch.autograd.grad(want[0].sum(), x64)[0],
              2.0 ** -18 * torch.softmax(x.double(), 1))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,V", LAYOUTS)
def test_distill_of_large_logits(rl, n, V, dtype):
    # large by themselves, or by the temperature
    for i, (at, t) in enumerate([(5e9, 1.0), (-1e10, 1.0), (1e20, 2.0), (-1e30, 1.0), (3e38, 0.5),
                                 (3e7, 0.7), (3000.0, 1e-4), (-3000.0, 1e-6), (2e5, 1e-3)]):
        g = gen(V + i)
        x, near = crowd(g, n, V, at, dtype)
        K = 5
        ids, top = some(g, near, K), torch.randn(n, K, generator=g) * t
        w = torch.randn(n, generator=g)
        dx, loss = rl.rlcs_distill_loss_backward(*cuda(w, x, ids, top), temperature=t,
                                                 return_loss=True)
        x64 = x.double().requires_grad_()
        want = ref.distill(x64, ids, top, temperature=t)
        l = ref.logs(x, t).gather(1, ids.long()).abs().amax(1)
        close("loss %g %g" % (at, t), loss, want, 2.0 ** -20 + 2.0 ** -21 * l)
        wdx, = torch.autograd.grad((want * w.double()).sum(), x64)
        close("dlogits %g %g" % (at, t), dx, wdx, F * (w.abs().double() / t)[:, None])
