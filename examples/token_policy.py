"""A policy over a vocabulary: linear attention, distillation, clipped updates.

The operators that a token policy is made of and learns from, as they are used
together. A linear-attention layer mixes packed episodes of tokens; the policy
is first distilled from the top logits of a teacher, then updated by the
clipped policy loss on advantages from GAE, held near the distilled policy by
a KL term. Both losses take the logits once and give back their gradient; the
layer's gradients come from its backward call. The policy then acts one token
at a time over its recurrent states and reaches the learner's logits.

    python examples/token_policy.py [--updates 20]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import linear_recurrence_scan_affine_gb300 as rl  # noqa: E402

VOCAB, WIDTH, HQ, HK, D, TOP = 500, 128, 4, 2, 64, 16
QKV = (HQ + 2 * HK) * D


class LinearAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, log_decay, cu):
        ctx.save_for_backward(q, k, v, log_decay, cu)
        return rl.rlcs_linear_attention(q, k, v, log_decay, cu)

    @staticmethod
    def backward(ctx, dout):
        dq, dk, dv, _ = rl.rlcs_linear_attention_backward(dout, *ctx.saved_tensors)
        return dq, dk, dv, None, None


class WeighedLoss(torch.autograd.Function):
    """sum(weights * loss) from one reading of the logits: `call(weights, logits)`
    gives (dlogits, losses)."""

    @staticmethod
    def forward(ctx, logits, weights, call):
        dlogits, loss = call(weights, logits)
        ctx.save_for_backward(dlogits)
        return (loss * weights).sum()

    @staticmethod
    def backward(ctx, upstream):
        return ctx.saved_tensors[0] * upstream.to(ctx.saved_tensors[0].dtype), None, None


def distill_loss(logits, weights, ids, top, mask):
    return WeighedLoss.apply(logits, weights, lambda w, x: rl.rlcs_distill_loss_backward(
        w, x, ids, top, mask=mask, return_loss=True))


def policy_loss(logits, weights, actions, old, advantages, reference, mask):
    def call(w, x):
        dx, got = rl.rlcs_policy_loss_backward(w, x, actions, old, advantages, ref_logp=reference,
                                               mask=mask, kl_coef=0.05, entropy_coef=0.01,
                                               return_loss=True)
        return dx, got.loss
    return WeighedLoss.apply(logits, weights, call)


def init(seed):
    g = torch.Generator().manual_seed(seed)

    def weight(n_in, n_out, scale=1.0):
        return (torch.randn(n_in, n_out, generator=g) * scale * n_in ** -0.5).cuda().requires_grad_()

    return {"embed": weight(VOCAB, WIDTH, VOCAB ** 0.5), "qkv": weight(WIDTH, QKV),
            "out": weight(HQ * D, WIDTH, 0.3), "head": weight(WIDTH, VOCAB),
            "value": weight(WIDTH, 1, 0.1)}


def decays():
    return torch.log(1.0 - 2.0 ** -torch.linspace(2.0, 6.0, HK)).cuda()


def linear(x, w):
    return x @ w.to(torch.bfloat16)


def layer(p, z, mix):
    """The layer's residual sum; `mix` is attention over q, k and v."""
    q, k, v = linear(z, p["qkv"]).view(-1, HQ + 2 * HK, D).split([HQ, HK, HK], 1)
    return z + linear(mix(q, k, v).reshape(-1, HQ * D), p["out"])


def learner(p, tokens, cu):
    """Logits [n, VOCAB] and values [n] of packed episodes."""
    z = p["embed"][tokens].to(torch.bfloat16)
    z = layer(p, z, lambda q, k, v: LinearAttention.apply(q, k, v, decays(), cu))
    return linear(z, p["head"]), (z @ p["value"].to(z.dtype)).float()[:, 0]


def actor(p, tokens, lens):
    """The same logits one token at a time: a state per episode."""
    at = torch.tensor([0] + lens).cumsum(0)
    state = torch.zeros(len(lens), HK, D, D, device="cuda")
    logits = torch.zeros(sum(lens), VOCAB, device="cuda", dtype=torch.bfloat16)
    for t in range(max(lens)):
        going = [i for i, n in enumerate(lens) if n > t]
        rows = (at[going] + t).cuda()
        own = torch.tensor(going, device="cuda")

        def mix(q, k, v):
            o, state[own] = rl.rlcs_linear_attention_step(q, k, v, decays(), state[own])
            return o
        z = layer(p, p["embed"][tokens[rows]].to(torch.bfloat16), mix)
        logits[rows] = linear(z, p["head"])
    return logits


def episodes(lens, seed):
    """Tokens, the actions taken (the next token), rewards and a teacher's top logits."""
    g = torch.Generator().manual_seed(seed)
    n = sum(lens)
    tokens = torch.randint(0, VOCAB, (n,), generator=g)
    actions = torch.roll(tokens, -1).to(torch.int32)
    rewards = torch.randn(n, generator=g) * 0.1 + (actions.long() % 7 == tokens % 7).float()
    ids = torch.stack([torch.randperm(VOCAB, generator=g)[:TOP] for _ in range(n)]).int()
    top = torch.randn(n, TOP, generator=g) * 2.0
    cu = torch.tensor([0] + lens).cumsum(0)
    last = torch.zeros(n)
    last[cu[1:] - 1] = 1.0  # an episode's last token ends it
    return [t.cuda() for t in (tokens, actions, rewards, last, ids, top, cu.int())]


def main(updates=20, lens=(300, 77, 150, 1, 222), report=print):
    lens = list(lens)
    p = init(0)
    opt = torch.optim.Adam(list(p.values()), lr=1e-3)
    tokens, actions, rewards, last, ids, top, cu = episodes(lens, 1)
    mask = last == 0.0  # (what follows an episode's end is no action of its own)
    weights = torch.full((len(tokens),), 1.0 / int(mask.sum()), device="cuda")
    for i in range(updates):
        logits, _ = learner(p, tokens, cu)
        loss = distill_loss(logits, weights, ids, top, mask)
        opt.zero_grad()
        loss.backward()
        opt.step()
    report("distilled: loss %.4f" % float(loss.detach()))
    with torch.no_grad():
        start = rl.rlcs_policy_loss(learner(p, tokens, cu)[0], actions, torch.zeros_like(rewards),
                                    torch.zeros_like(rewards)).logp
    for i in range(updates):
        logits, values = learner(p, tokens, cu)
        with torch.no_grad():
            fixed = values.detach()
            # one row of steps, cut at the episodes' ends
            advantages = rl.rlcs_gae(rewards[None], fixed[None], last[None])[0]
            targets = advantages + fixed
        loss = policy_loss(logits, weights, actions, start, advantages, start, mask)
        loss = loss + 0.5 * (values - targets).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
    report("updated: loss %.4f" % float(loss.detach()))
    with torch.no_grad():
        whole, steps = learner(p, tokens, cu)[0].float(), actor(p, tokens, lens).float()
    apart, size = float((whole - steps).abs().max()), float(whole.abs().max())
    report("learner and actor apart by %.4f of %.4f" % (apart, size))
    rl.check_scratch()
    rl.check_all_workspaces()
    return p, apart, size


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--updates", type=int, default=20)
    main(ap.parse_args().updates)
