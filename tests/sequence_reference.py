"""The sequence operators in 64 bits, step by step, for the tests.

Each function takes CPU tensors, works in float64 and follows the operator's
definition. `*_slack` values bound what the kernels' documented roundings can
move a result by: U is the largest relative error of one rounding to bfloat16.
"""
import math

import torch

U = 2.0 ** -8


def gated_scan(x, gate, reset=None, h0=None):
    x, gate = x.double(), gate.double()
    B, T, D = x.shape
    a = torch.sigmoid(gate)
    h = torch.zeros(B, T, D, dtype=torch.float64)
    cur = torch.zeros(B, D, dtype=torch.float64) if h0 is None else h0.double()
    for t in range(T):
        if reset is not None:
            cur = torch.where(reset[:, t, None].bool(), torch.zeros_like(cur), cur)
        cur = a[:, t] * cur + torch.sigmoid(-gate[:, t]) * x[:, t]
        h[:, t] = cur
    return h


def gated_scan_backward(dh, x, gate, reset=None, h0=None, dh_last=None):
    """(dx, dgate, dh0, slack of dgate where the states were rounded to bfloat16)."""
    h = gated_scan(x, gate, reset, h0)
    x, gate, dh = x.double(), gate.double(), dh.double()
    B, T, D = x.shape
    a, om = torch.sigmoid(gate), torch.sigmoid(-gate)
    dx, dg, slack = (torch.zeros(B, T, D, dtype=torch.float64) for _ in range(3))
    cur = torch.zeros(B, D, dtype=torch.float64) if dh_last is None else dh_last.double()
    for t in reversed(range(T)):
        lam = dh[:, t] + cur
        if t:
            before = h[:, t - 1]
        else:
            before = torch.zeros(B, D, dtype=torch.float64) if h0 is None else h0.double()
        keep = torch.ones(B, 1, dtype=torch.float64)
        if reset is not None:
            keep = 1.0 - reset[:, t, None].double()
        before = torch.where(keep > 0, before, torch.zeros_like(before))
        dx[:, t] = om[:, t] * lam
        dg[:, t] = a[:, t] * om[:, t] * lam * (before - x[:, t])
        slack[:, t] = U * (a[:, t] * om[:, t] * lam * before).abs()
        cur = torch.where(keep > 0, a[:, t] * lam, torch.zeros_like(lam))
    return dx, dg, cur, slack


def pairs_of(R, interleaved):
    i = torch.arange(R // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)


def rotate(u, cos, sin, interleaved):
    y = u.clone()
    if cos.shape[-1]:
        p, q = pairs_of(2 * cos.shape[-1], interleaved)
        y[..., p] = u[..., p] * cos - u[..., q] * sin
        y[..., q] = u[..., q] * cos + u[..., p] * sin
    return y


def norm_rope(x, w, cos, sin, positions, eps, interleaved):
    x, w = x.double(), w.double()
    c, s = (t.double()[positions.long()][:, None] for t in (cos, sin))
    r = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    return rotate(x * r * w, c, s, interleaved)


def norm_rope_backward(dy, x, w, cos, sin, positions, eps, interleaved):
    x, w, dy = x.double(), w.double(), dy.double()
    c, s = (t.double()[positions.long()][:, None] for t in (cos, sin))
    r = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    du = rotate(dy, c, -s, interleaved)
    dw = (du * x * r).sum((0, 1))
    g = du * w
    return r * (g - x * r * r * (g * x).mean(-1, keepdim=True)), dw


def attention(q, k, v, lens, scale):
    """(out, lse, slack of out): P is rounded to bfloat16 for its product with v."""
    q, k, v = q.double(), k.double(), v.double()
    n, Hq, D = q.shape
    group = Hq // k.shape[1]
    out, slack = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.zeros(Hq, n, dtype=torch.float64)
    at = 0
    for length in lens:
        r = slice(at, at + length)
        at += length
        if not length:
            continue
        later = torch.ones(length, length, dtype=torch.bool).triu(1)
        for h in range(Hq):
            s = (q[r, h] @ k[r, h // group].T * scale).masked_fill(later, -math.inf)
            lse[h, r] = torch.logsumexp(s, 1)
            p = torch.softmax(s, 1)
            out[r, h] = p @ v[r, h // group]
            slack[r, h] = U * (p @ v[r, h // group].abs())
    return out, lse, slack


def attention_backward(dout, q, k, v, lens, scale):
    """(dq, dk, dv) and their slacks: P and dS are rounded to bfloat16 for
    their products, and delta comes from the rounded output."""
    q, k, v, dout = q.double(), k.double(), v.double(), dout.double()
    group = q.shape[1] // k.shape[1]
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    sq, sk, sv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    at = 0
    for length in lens:
        r = slice(at, at + length)
        at += length
        if not length:
            continue
        later = torch.ones(length, length, dtype=torch.bool).triu(1)
        for h in range(q.shape[1]):
            g = h // group
            p = torch.softmax((q[r, h] @ k[r, g].T * scale).masked_fill(later, -math.inf), 1)
            out = p @ v[r, g]
            do = dout[r, h]
            delta = (do * out).sum(1, keepdim=True)
            ds = p * (do @ v[r, g].T - delta)
            # the rounded output moves delta by at most U sum |do| (|out| + p |v|)
            off = U * (do.abs() * (out.abs() + p @ v[r, g].abs())).sum(1, keepdim=True)
            err = U * ds.abs() + p * off
            dq[r, h] += scale * ds @ k[r, g]
            dk[r, g] += scale * ds.T @ q[r, h]
            dv[r, g] += p.T @ do
            sq[r, h] += scale * err @ k[r, g].abs()
            sk[r, g] += scale * err.T @ q[r, h].abs()
            sv[r, g] += U * p.T @ do.abs()
    return (dq, dk, dv), (sq, sk, sv)


def attention_step(q, kc, vc, lengths, scale):
    q, kc, vc = q.double(), kc.double(), vc.double()
    B, Hq, _ = q.shape
    group = Hq // kc.shape[2]
    out, slack = torch.zeros_like(q), torch.zeros_like(q)
    for b in range(B):
        n = int(lengths[b])
        if n == 0:
            continue
        for h in range(Hq):
            p = torch.softmax(kc[b, :n, h // group] @ q[b, h] * scale, 0)
            out[b, h] = p @ vc[b, :n, h // group]
            slack[b, h] = U * (p @ vc[b, :n, h // group].abs())
    return out, slack
