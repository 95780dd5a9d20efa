"""Linear attention in 64 bits, as one matrix of weights per sequence and head,
and bounds on what the kernels' documented roundings can move a result by.

U is the largest relative error of one rounding to bfloat16. Three quantities
are rounded to it for their products: weights, states, and decayed keys. Each
rounding's error is at most U of the term it belongs to, its sign independent
of the others', so its variance is at most (U term)^2 / 3; a sum's error stays
within six standard deviations, 6 / sqrt(3) U sqrt(sum of term^2), at the few
million elements tested. A decayed key of a returned state is held in two
parts, off by at most U^2 together.
"""
import math

import torch

U = 2.0 ** -8
SIX = 6.0 / math.sqrt(3.0)


def powers(ld, steps):
    """exp(ld) ** steps for integers steps >= 0, 1 at 0 whatever ld is."""
    s = steps.double()
    return torch.where(steps > 0, torch.exp(ld.double() * s.clamp(min=1.0)), torch.ones_like(s))


def weights(ld, n):
    i = torch.arange(n)
    apart = i[:, None] - i[None, :]
    return powers(ld, apart.clamp(min=0)) * (apart >= 0)


def linear(q, k, v, ld, lens, state=None, scale=None):
    """(out, last) in 64 bits; differentiable."""
    n, Hq, D = q.shape
    Hk = k.shape[1]
    scale = D ** -0.5 if scale is None else scale
    q, k, v = q.double(), k.double(), v.double()
    outs, lasts, at = [], [], 0
    for s, m in enumerate(lens):
        r = slice(at, at + m)
        at += m
        i = torch.arange(m)
        heads, states = [], []
        for h in range(Hk):
            first = None if state is None else state[s, h].double()
            W = weights(ld[h], m)
            tail = powers(ld[h], m - 1 - i)
            last = (k[r, h] * tail[:, None]).T @ v[r, h]
            if first is not None:
                last = last + powers(ld[h], torch.tensor(m)) * first
            states.append(last)
            for g in range(Hq // Hk):
                x = q[r, h * (Hq // Hk) + g] * scale
                o = ((x @ k[r, h].T) * W) @ v[r, h]
                if first is not None:
                    o = o + powers(ld[h], i + 1)[:, None] * (x @ first)
                heads.append(o)
        outs.append(torch.stack(heads, 1))
        lasts.append(torch.stack(states))
    rest = torch.zeros(n - at, Hq, D, dtype=torch.float64)
    return torch.cat(outs + [rest]), torch.stack(lasts)


def _walk_slack(x, y, z, ld, first, inclusive_first):
    """Slack of out_t = sum_{j<=t} a^(t-j) (x_t . y_j) z_j + ... for one
    sequence and one reader x [m, D]; y, z [m, sources, D] enter the state."""
    m = x.shape[0]
    i = torch.arange(m)
    W = weights(ld, m)
    from_first = powers(ld, i + (0 if inclusive_first else 1))
    var = torch.zeros(m, z.shape[2], dtype=torch.float64)
    S = torch.zeros(m, y.shape[2], z.shape[2], dtype=torch.float64)
    for j in range(y.shape[1]):
        P = (x @ y[:, j].T) * W
        var += P.square() @ z[:, j].square()
        # decayed keys, term by term
        var += torch.einsum("td,tj,jd,je->te", x.square(), W.square(), y[:, j].square(),
                            z[:, j].square())
        S += torch.einsum("tj,jd,je->tde", W, y[:, j], z[:, j])
    if first is not None:
        S += from_first[:, None, None] * first
    var += torch.einsum("td,tde->te", x.square(), S.square())
    return SIX * U * var.sqrt()


def slack(q, k, v, ld, lens, state=None, scale=None):
    """Of out. [tokens, Hq, D]"""
    n, Hq, D = q.shape
    Hk = k.shape[1]
    G = Hq // Hk
    scale = D ** -0.5 if scale is None else scale
    res, at = torch.zeros(n, Hq, D, dtype=torch.float64), 0
    for s, m in enumerate(lens):
        r = slice(at, at + m)
        at += m
        if m == 0:
            continue
        for h in range(Hq):
            g = h // G
            first = None if state is None else state[s, g].double()
            res[r, h] = _walk_slack(q[r, h].double() * scale, k[r, g:g + 1].double(),
                                    v[r, g:g + 1].double(), ld[g], first, False)
    return res


def backward_slack(dout, q, k, v, ld, lens, state=None, dlast=None, scale=None):
    """Of (dq, dk, dv): the same walk on other arrays."""
    n, Hq, D = q.shape
    Hk = k.shape[1]
    G = Hq // Hk
    scale = D ** -0.5 if scale is None else scale
    dq = slack(dout, v, k, ld, lens, None if state is None else state.transpose(-1, -2), scale)
    dk, dv = (torch.zeros(n, Hk, D, dtype=torch.float64) for _ in range(2))
    at = 0
    for s, m in enumerate(lens):
        r = slice(at, at + m)
        at += m
        if m == 0:
            continue
        for h in range(Hk):
            qs, ds = (t[r, h * G:(h + 1) * G].double().flip(0) for t in (q * scale, dout))
            ks, vs = (t[r, h].double().flip(0) for t in (k, v))
            R = None if dlast is None else dlast[s, h].double()
            dv[r, h] = _walk_slack(ks, qs, ds, ld[h], R, True).flip(0)
            dk[r, h] = _walk_slack(vs, ds, qs, ld[h], None if R is None else R.T, True).flip(0)
    return dq, dk, dv


def state_slack(y, z, ld, lens, extra=0):
    """Of a state that y [tokens, Hk, sources, D] and z enter: two-part keys."""
    Hk, D = y.shape[1], y.shape[3]
    res, at = torch.zeros(len(lens), Hk, D, D, dtype=torch.float64), 0
    for s, m in enumerate(lens):
        r = slice(at, at + m)
        at += m
        if m == 0:
            continue
        tail = powers(2 * ld[:, None].double(), (m - 1 - torch.arange(m) + extra)[None])
        res[s] = torch.einsum("hj,jhsd,jhse->hde", tail, y[r].double().square(),
                              z[r].double().square()).sqrt()
    return SIX * U * U * res


def step(q, k, v, ld, state, reset=None, scale=None):
    B, Hq, D = q.shape
    Hk = k.shape[1]
    scale = D ** -0.5 if scale is None else scale
    old = state.double()
    if reset is not None:
        old = torch.where(reset.bool()[:, None, None, None], torch.zeros_like(old), old)
    a = ld.double().exp()[:, None, None]
    old = torch.where(a > 0, a * old, torch.zeros_like(old))
    new = old + k.double()[..., :, None] * v.double()[..., None, :]
    x = q.double().view(B, Hk, Hq // Hk, D) * scale
    return (x @ new).view(B, Hq, D), new
