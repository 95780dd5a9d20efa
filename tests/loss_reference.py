"""The losses of a policy's logits in 64 bits, row by row, for the tests.

Values and gradients come from their formulas as torch writes them down, with
automatic differentiation for the gradients."""
import math

import torch


def logs(x, temperature=1.0):
    return torch.log_softmax(x.double() / temperature, 1)


def policy(x, actions, old, adv, ref=None, mask=None, low=0.2, high=0.2, kl_coef=0.0, ent=0.0):
    """(loss, logp, entropy, kl) of [tokens, V] logits in 64 bits; differentiable."""
    lp = logs(x)
    p = lp.exp()
    H = -(p * torch.where(p > 0, lp, torch.zeros_like(lp))).sum(1)
    l = lp.gather(1, actions.long()[:, None])[:, 0]
    ratio, A = (l - old.double()).exp(), adv.double()
    # float32 bounds, as the library holds them
    lo, hi = (float(torch.tensor(b, dtype=torch.float32)) for b in (1.0 - low, 1.0 + high))
    free, held = ratio * A, ratio.clamp(lo, hi) * A
    loss = -torch.where(free > held, held.detach(), free)
    kl = None
    if ref is not None:
        d = ref.double() - l
        kl = torch.expm1(d) - d
        loss = loss + (kl_coef * kl if kl_coef else 0.0)
    if ent:
        loss = loss - ent * H
    out = [loss, l, H, kl]
    if mask is not None:
        out = [None if t is None else torch.where(mask.bool(), t, torch.zeros_like(t))
               for t in out]
    return out


def distill(x, ids, top, lse=None, mask=None, temperature=1.0):
    """loss [tokens] in 64 bits; differentiable in x."""
    n, V = x.shape
    there = (ids >= 0) & (ids < V) & (top > -math.inf)
    t = (top.double() / temperature).masked_fill(~there, -math.inf)
    none = ~there.any(1, keepdim=True)
    total = torch.logsumexp(t.masked_fill(none, 0.0), 1) if lse is None else lse.double()
    lq = t - total[:, None]
    q = torch.where(there, lq.exp(), torch.zeros_like(lq))
    lp = logs(x, temperature).gather(1, ids.clamp(0, V - 1).long())
    loss = torch.where(q > 0, q * (lq - lp), torch.zeros_like(q)).sum(1)
    keep = ~none[:, 0] if mask is None else ~none[:, 0] & mask.bool()
    return torch.where(keep, loss, torch.zeros_like(loss))
