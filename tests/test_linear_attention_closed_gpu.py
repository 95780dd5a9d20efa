"""Linear attention in heads that keep nothing (log_decay -infinity): a result depends
on its own token alone, whatever others hold, and so do the last state and the
gradients. With one token to a sum the definition is

  out = scale (q k) v,  dq = scale (dout v) k,  last = k v^T of the last token,
  G = scale sum_heads q dout^T (and dlast at a last token),  dk = G v,  dv = G^T k

and the bounds of tests/linear_reference.py, six standard deviations of the roundings
of weights, keys and states, are SIX U of the root of (x y)^2 z^2 + (x^2 y^2) z^2 +
x^2 S^2; 1.87 of it beside an element that is not finite.
"""
import math

import pytest
import torch

from tests.linear_reference import SIX
from tests.test_linear_attention_gpu import F, U, bounds, cuda, gen, rand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rl():
    assert torch.cuda.is_available(), "the -m gpu tests need a CUDA device"
    import linear_recurrence_scan_affine_gb300 as m
    return m


def reader(x, y, z, R=None):
    """x S and its bound's root, S = sum_heads y z^T + R: x [n, D], y and z [n, G, D]."""
    P = torch.einsum("nd,ngd->ng", x, y)
    out, S = torch.einsum("ng,nge->ne", P, z), torch.einsum("ngd,nge->nde", y, z)
    if R is not None:
        out, S = out + torch.einsum("nd,nde->ne", x, R), S + R
    var = torch.einsum("ng,nge->ne", P ** 2, z ** 2) \
        + torch.einsum("nd,ngd,nge->ne", x ** 2, y ** 2, z ** 2) \
        + torch.einsum("nd,nde->ne", x ** 2, S ** 2)
    return out, SIX * U * var.sqrt()


@pytest.mark.parametrize("lens,D,G", [([200], 64, 1), ([300, 50], 128, 2), ([128, 1, 129], 72, 1),
                                      ([2600], 64, 1), ([2600], 128, 1)], ids=str)
@pytest.mark.parametrize("which", ["k", "v", "q", "d", None])
def test_a_token_alone(rl, lens, D, G, which):
    n, g, scale = sum(lens), gen(D + len(lens)), D ** -0.5
    q, k, v, do = (rand(g, n, h, D) for h in (G, 1, 1, G))
    S, dl = (rand(g, len(lens), 1, D, D, dtype=torch.float32) for _ in range(2))
    ld = torch.tensor([-math.inf])
    ends = bounds(lens).tolist()
    bad = [t for t in (0, 31, 40, 127, 128, 150, 199, 290, 1024, 2300, n - 1)
           if t < n and t + 1 not in ends]  # (not a sequence's last)
    arrays = {"q": q, "k": k, "v": v, "d": do}
    clean = {a: t.clone().double() for a, t in arrays.items()}
    if which:
        for i, t in enumerate(bad):
            arrays[which][t, 0, (5 * i) % D] = (math.nan, math.inf)[i % 2]
    cq, ck, cv, cl, cS, cdo, cdl, cu = cuda(q, k, v, ld, S, do, dl, bounds(lens))
    out, last = rl.rlcs_linear_attention(cq, ck, cv, cl, cu, state=cS, return_state=True)
    dq, dk, dv, dstate = rl.rlcs_linear_attention_backward(cdo, cq, ck, cv, cl, cu, state=cS,
                                                           dlast=cdl)
    rl.check_scratch()
    q, k, v, do = (clean[a] for a in "qkvd")
    ends = torch.tensor([e - 1 for e in ends[1:]])
    R = torch.zeros(n, D, D, dtype=torch.float64)
    R[ends] = dl[:, 0].double()
    wants = {"dk": reader(v[:, 0], do, scale * q, R.transpose(1, 2)),
             "dv": reader(k[:, 0], scale * q, do, R)}
    for h in range(G):
        wants["out", h] = reader(scale * q[:, h], k, v)
        wants["dq", h] = reader(scale * do[:, h], v, k)
    other = torch.ones(n, dtype=torch.bool)
    if which:
        other[bad] = False
    for key, (want, slack) in wants.items():
        name, h = (key, 0) if isinstance(key, str) else key
        got = {"out": out, "dq": dq, "dk": dk, "dv": dv}[name][:, h].double().cpu()[other]
        want, slack = want[other], slack[other]
        tol = F * torch.maximum(want.abs(), want.square().mean().sqrt()) + 1.87 * slack \
            + U * want.abs()
        off = (got - want).abs()
        assert bool((off <= tol).all()), (key, float((off / tol).max()))
    want = torch.einsum("nd,ne->nde", k[ends, 0], v[ends, 0])
    assert bool(((last[:, 0].double().cpu() - want).abs() <= F * want.abs()).all())
    assert not dstate.any()
