"""The token policy's operators as they are used together: the gradients of both
losses through the layer against the same model in 64 bits, and acting by
single steps against the whole pass."""
import importlib.util
import math
import os

import pytest
import torch

from tests import linear_reference, loss_reference

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
U = 2.0 ** -8


@pytest.fixture(scope="module")
def ex():
    assert torch.cuda.is_available(), "the -m gpu tests need a CUDA device"
    spec = importlib.util.spec_from_file_location(
        "token_policy", os.path.join(ROOT, "examples", "token_policy.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def plain(ex, p, tokens, lens):
    """The learner's logits and values in 64 bits, from its float32 parameters."""
    z = p["embed"][tokens]
    q, k, v = (z @ p["qkv"]).view(-1, ex.HQ + 2 * ex.HK, ex.D).split([ex.HQ, ex.HK, ex.HK], 1)
    mixed, _ = linear_reference.linear(q, k, v, ex.decays().cpu(), lens)
    z = z + mixed.reshape(-1, ex.HQ * ex.D) @ p["out"]
    return z @ p["head"], (z @ p["value"])[:, 0]


@pytest.mark.parametrize("which", ["distill", "policy"])
def test_gradients(ex, which):
    lens = [130, 40, 1, 65]
    p = ex.init(3)
    tokens, actions, rewards, last, ids, top, cu = ex.episodes(lens, 4)
    mask = last == 0.0
    n = len(tokens)
    weights = torch.full((n,), 1.0 / n, device="cuda")
    p64 = {k: t.detach().double().cpu().requires_grad_() for k, t in p.items()}
    x64, v64 = plain(ex, p64, tokens.cpu(), lens)
    logits, values = ex.learner(p, tokens, cu)
    if which == "distill":
        loss = ex.distill_loss(logits, weights, ids, top, mask)
        want = loss_reference.distill(x64, ids.cpu(), top.cpu(), mask=mask.cpu()).sum() / n
    else:
        logp = loss_reference.logs(x64.detach()).gather(1, actions.cpu().long()[:, None])[:, 0]
        # ratios of 0.9 and 1.1, away from the bounds, whatever the logits' rounding
        off = torch.where(torch.arange(n) % 2 == 0, math.log(0.9), math.log(1.1))
        old = (logp - off).float()
        adv = rewards - 0.5
        loss = ex.policy_loss(logits, weights, actions, old.cuda(), adv, old.cuda(), mask)
        want = loss_reference.policy(x64, actions.cpu(), old, adv.cpu(), old, mask.cpu(),
                                     kl_coef=0.05, ent=0.01)[0].sum() / n
    loss = loss + 0.1 * values.square().mean()
    want = want + 0.1 * v64.square().mean()
    grads = torch.autograd.grad(loss, list(p.values()))
    wants = torch.autograd.grad(want, list(p64.values()))
    # Each array on the way is rounded to bfloat16 (embedding, projections, the
    # layer's result, the sum, logits, and as many gradients back): about twelve
    # roundings, each off by U / sqrt(3) of its array's norm in the mean, half
    # of which could add up: the norm of the difference stays below 8 U.
    for name, g, w in zip(p, grads, wants):
        off = float((g.double().cpu() - w).norm() / w.norm())
        assert off <= 8 * U, (name, off)


def test_example_runs_and_acts(ex):
    lines = []
    p, apart, size = ex.main(updates=3, lens=(140, 20, 1, 60), report=lines.append)
    assert all(bool(torch.isfinite(t).all()) for t in p.values())
    # bfloat16 activations through one layer: a few roundings of U
    assert apart <= 16 * U * size, lines
