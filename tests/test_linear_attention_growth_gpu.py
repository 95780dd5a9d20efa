"""Linear attention with decays that grow (log_decay above 0), against its
definition in 64 bits.

Bounds are those of tests/linear_reference.py. A growing head's tokens differ by
up to 10^35 in size, so the float32 part of a bound is taken from each token's
own root mean square, not from the whole array's.
"""
import math

import pytest
import torch

from tests import linear_reference as ref
from tests.test_linear_attention_gpu import bounds, case, cuda, gen, rand

pytestmark = pytest.mark.gpu

F, U = 2e-5, ref.U
LARGEST = 80.0  # of log_decay times length: e^80 is 5.5e34, sums of D terms stay in range


@pytest.fixture(scope="module")
def rl():
    assert torch.cuda.is_available(), "the -m gpu tests need a CUDA device"
    import linear_recurrence_scan_affine_gb300 as m
    return m


def close(name, got, want, slack):
    want = want.detach().double()
    rms = want.square().flatten(1).mean(1).sqrt()
    rms = rms.view(-1, *[1] * (want.dim() - 1))
    tol = F * torch.maximum(want.abs(), rms) + slack
    if got.dtype == torch.bfloat16:
        tol = tol + U * want.abs()
    off = (got.double().cpu() - want).abs()
    assert bool((off <= tol).all()), "%s: %.3g times the bound" % (
        name, (off / tol.clamp(min=1e-300)).max())


def check(rl, lens, args):
    q, k, v, ld, S, do, dl = args
    cq, ck, cv, cl, cS, cdo, cdl, cu = cuda(q, k, v, ld, S, do, dl, bounds(lens))
    out = rl.rlcs_linear_attention(cq, ck, cv, cl, cu, state=cS)
    leaves = [t.double().requires_grad_() for t in (q, k, v)]
    want, wlast = ref.linear(*leaves, ld, lens, S)
    close("out", out, want, ref.slack(q, k, v, ld, lens, S))
    grads = rl.rlcs_linear_attention_backward(cdo, cq, ck, cv, cl, cu, state=cS, dlast=cdl)
    loss = (want * do.double()).sum()
    if dl is not None:
        loss = loss + (wlast * dl.double()).sum()
    wants = torch.autograd.grad(loss, leaves)
    for name, got, w, s in zip(("dq", "dk", "dv"), grads, wants,
                               ref.backward_slack(do, q, k, v, ld, lens, S, dl)):
        close(name, got, w, s)
    rl.check_scratch()


@pytest.mark.parametrize("states", [False, True])
@pytest.mark.parametrize("Hk,G,D", [(4, 1, 64), (4, 2, 128), (4, 3, 40)])
@pytest.mark.parametrize("lens", [[1], [10], [33], [60], [128], [129], [140], [10, 0, 60, 3],
                                  [128, 10]], ids=str)
def test_growth(rl, lens, Hk, G, D, states):
    # as fast as the longest sequence allows, and slower
    most = min(1.5, LARGEST / max(lens))
    decays = [most, 0.6 * most, 0.1 * most, -0.1]
    check(rl, lens, case(sum(lens) + D, lens, Hk * G, Hk, D, states, decays))


@pytest.mark.parametrize("D", [64, 128])
def test_ten_tokens(rl, D):
    # weights no longer than e^9 are needed, e^127 would not be in range
    check(rl, [10], case(D, [10], 2, 2, D, False, [1.0, 0.7]))


@pytest.mark.parametrize("D", [64, 128])
def test_a_power_past_the_last_weight(rl, D):
    # The largest weight, a^59 = e^87.9, is in range and a^60 = e^89.4 is not:
    # without a state nothing is multiplied by it.
    lens, n, g = [60], 60, gen(D)
    q, k, v, do = (rand(g, n, 1, D, scale=s) for s in (2.0 ** -9, 0.25, 0.25, 2.0 ** -9))
    ld = torch.tensor([1.49])
    assert 59 * 1.49 < math.log(torch.finfo(torch.float32).max) < 60 * 1.49
    check(rl, lens, (q, k, v, ld, None, do, None))
