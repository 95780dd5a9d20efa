"""A recurrent-attention policy and critic on rollouts, trained by V-trace.

The sequence operators and the estimators together, as an actor-learner uses
them. The learner sees a batch of rollouts [N, T] cut into episodes by their
dones: a gated linear recurrence mixes each row (resets at the cuts), causal
attention with normed, rotated queries and keys mixes each episode (the
episodes of all rows packed one after another), V-trace turns the critic's
values into targets and advantages, and the gradients come back through the
operators' backward calls. The actor then walks the same rollouts one step at
a time, with a recurrent state and a key/value cache per row, and reaches the
learner's outputs.

    python examples/sequence_policy.py [--updates 30]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import linear_recurrence_scan_affine_gb300 as rl  # noqa: E402

WIDTH, HQ, HK, D, ACTIONS, OBS = 256, 4, 2, 64, 6, 16
QKV = (HQ + 2 * HK) * D


class GatedScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gate, reset):
        h, _ = rl.rlcs_gated_scan(x, gate, reset=reset)
        ctx.save_for_backward(x, gate, h, reset)
        return h

    @staticmethod
    def backward(ctx, dh):
        x, gate, h, reset = ctx.saved_tensors
        dx, dgate, _ = rl.rlcs_gated_scan_backward(dh, x, gate, h, reset=reset)
        return dx, dgate, None


class NormRope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, qw, kw, cos, sin, positions):
        ctx.save_for_backward(q, k, qw, kw, cos, sin, positions)
        return rl.rlcs_qk_norm_rope(q, k, qw, kw, cos, sin, positions)

    @staticmethod
    def backward(ctx, dq, dk):
        return (*rl.rlcs_qk_norm_rope_backward(dq, dk, *ctx.saved_tensors), None, None, None)


class Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, cu):
        out, lse = rl.rlcs_attention(q, k, v, cu, return_lse=True)
        ctx.save_for_backward(q, k, v, out, lse, cu)
        return out

    @staticmethod
    def backward(ctx, dout):
        q, k, v, out, lse, cu = ctx.saved_tensors
        return (*rl.rlcs_attention_backward(dout, q, k, v, out, lse, cu), None)


def init(seed):
    g = torch.Generator().manual_seed(seed)

    def weight(n_in, n_out, scale=1.0):
        w = torch.randn(n_in, n_out, generator=g) * scale * n_in ** -0.5
        return w.cuda().requires_grad_()

    return {"inp": weight(OBS, WIDTH), "x": weight(WIDTH, WIDTH), "gate": weight(WIDTH, WIDTH),
            "qkv": weight(WIDTH, QKV), "out": weight(HQ * D, WIDTH),
            "qw": torch.ones(D).cuda().requires_grad_(), "kw": torch.ones(D).cuda().requires_grad_(),
            "value": weight(WIDTH, 1, 0.1), "policy": weight(WIDTH, ACTIONS, 0.1)}


def linear(x, w):
    return x @ w.to(torch.bfloat16)


def episodes(dones):
    """Resets [N, T], and the packed episodes' bounds and positions."""
    N, T = dones.shape
    reset = torch.zeros(N, T, dtype=torch.bool, device=dones.device)
    reset[:, 1:] = dones[:, :-1] > 0
    starts = reset.clone()
    starts[:, 0] = True
    first = starts.flatten().nonzero().flatten()
    end = torch.tensor([N * T], device=first.device)
    cu = torch.cat([first, end]).to(torch.int32)
    positions = torch.arange(N * T, device=first.device) - first.repeat_interleave(
        torch.diff(torch.cat([first, end])))
    return reset, cu, positions.to(torch.int32)


def learner(p, obs, reset, cu, positions, tables):
    """Values [N, T] and logits [N, T, ACTIONS] of whole rollouts."""
    N, T, _ = obs.shape
    z = linear(obs.to(torch.bfloat16), p["inp"])
    z = z + GatedScan.apply(linear(z, p["x"]), linear(z, p["gate"]) + 2.0, reset)
    qkv = linear(z, p["qkv"]).view(N * T, HQ + 2 * HK, D)
    q, k, v = qkv.split([HQ, HK, HK], 1)
    q, k = NormRope.apply(q, k, p["qw"], p["kw"], *tables, positions)
    mixed = Attention.apply(q, k, v, cu)
    z = z + linear(mixed.reshape(N, T, HQ * D), p["out"])
    return (z @ p["value"].to(z.dtype)).float()[..., 0], (z @ p["policy"].to(z.dtype)).float()


def actor(p, obs, dones, tables):
    """The same outputs one step at a time: a state and a cache per row."""
    N, T, _ = obs.shape
    state = torch.zeros(N, WIDTH, device="cuda")
    cache = torch.zeros(2, N, T, HK, D, dtype=torch.bfloat16, device="cuda")
    length = torch.zeros(N, dtype=torch.int32, device="cuda")
    rows = torch.arange(N, device="cuda")
    fresh = torch.ones(N, dtype=torch.bool, device="cuda")
    values, logits = [], []
    for t in range(T):
        z = linear(obs[:, t].to(torch.bfloat16), p["inp"])
        h, _ = rl.rlcs_gated_step(linear(z, p["x"]), linear(z, p["gate"]) + 2.0, state,
                                  reset=fresh, new_state=state)
        z = z + h
        length = torch.where(fresh, torch.zeros_like(length), length)
        qkv = linear(z, p["qkv"]).view(N, HQ + 2 * HK, D)
        q, k, v = qkv.split([HQ, HK, HK], 1)
        q, k = rl.rlcs_qk_norm_rope(q, k, p["qw"], p["kw"], *tables, length)
        cache[0, rows, length.long()], cache[1, rows, length.long()] = k, v
        length = length + 1
        mixed = rl.rlcs_attention_step(q, cache[0], cache[1], length)
        z = z + linear(mixed.reshape(N, HQ * D), p["out"])
        values.append((z @ p["value"].to(z.dtype)).float()[:, 0])
        logits.append((z @ p["policy"].to(z.dtype)).float())
        fresh = dones[:, t] > 0
    return torch.stack(values, 1), torch.stack(logits, 1)


def rollouts(N, T, seed):
    """Synthetic rollouts whose reward is for repeating the last observation's sign."""
    g = torch.Generator().manual_seed(seed)
    obs = torch.randn(N, T, OBS, generator=g).cuda()
    dones = (torch.rand(N, T, generator=g) < 0.02).float().cuda()
    actions = torch.randint(0, ACTIONS, (N, T), generator=g).cuda()
    want = (torch.roll(obs[..., 0], 1, 1) > 0).long()
    rewards = (actions == want).float()
    return obs, dones, actions, rewards


def main(updates=30, N=32, T=256, report=print):
    p = init(0)
    opt = torch.optim.Adam(list(p.values()), lr=1e-3)
    tables = rl.rlcs_rope_table(T, D)
    obs, dones, actions, rewards = rollouts(N, T, 1)
    reset, cu, positions = episodes(dones)
    behaviour = torch.full((N, T), -torch.log(torch.tensor(float(ACTIONS))).item(), device="cuda")
    losses = []
    for i in range(updates):
        values, logits = learner(p, obs, reset, cu, positions, tables)
        logp = torch.log_softmax(logits, -1)
        taken = logp.gather(-1, actions[..., None])[..., 0]
        with torch.no_grad():
            targets, advantages = rl.rlcs_vtrace(rewards, values.detach().contiguous(),
                                                 (taken.detach() - behaviour).contiguous(), dones,
                                                 gamma=0.9)
        loss = (0.5 * (values - targets).square().mean() - (taken * advantages).mean()
                + 0.01 * (logp.exp() * logp).sum(-1).mean())
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(float((0.5 * (values - targets).square().mean()).detach()))
        if i % 10 == 0 or i + 1 == updates:
            report("update %d: value loss %.4f" % (i, losses[-1]))
    with torch.no_grad():
        whole = learner(p, obs, reset, cu, positions, tables)
        steps = actor(p, obs, dones, tables)
    apart = max(float((a - b).abs().max()) for a, b in zip(whole, steps))
    size = max(float(a.abs().max()) for a in whole)
    report("learner and actor apart by %.4f of %.4f" % (apart, size))
    rl.check_scratch()
    rl.check_all_workspaces()
    return losses, apart, size


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--updates", type=int, default=30)
    main(ap.parse_args().updates)
