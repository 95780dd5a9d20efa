"""Linear attention with elements that are not finite: a result is not finite where it
depends on one by the definition, and nowhere else, however tokens share a tile.

Bounds are those of tests/linear_reference.py. In a tile with such an element what
the state gives is rounded to bfloat16 once more: by U / 2 of it, at most six of the
standard deviations that SIX U sqrt(var) is made of, 3 U sqrt(var). So 1.87 of the
slack there.
"""
import math

import pytest
import torch

from tests import linear_reference as ref
from tests.test_linear_attention_gpu import F, U, bounds, case, cuda

pytestmark = pytest.mark.gpu

PARTS = ("out", "dq", "dk", "dv")


@pytest.fixture(scope="module")
def rl():
    assert torch.cuda.is_available(), "the -m gpu tests need a CUDA device"
    import linear_recurrence_scan_affine_gb300 as m
    return m


def reached(which, t, h, d, G, shapes, at, end):
    """For each result, the elements that the element (t, h, d) of `which` reaches;
    its sequence is [at, end)."""
    res = {n: torch.zeros(s, dtype=torch.bool) for n, s in shapes.items()}
    own = slice(h * G, (h + 1) * G) if which in "kv" else slice(h, h + 1)
    kv = h if which in "kv" else h // G
    if which == "q":
        res["out"][t, h] = True
        res["dk"][at:t + 1, kv, d] = True
        res["dv"][at:t + 1, kv] = True
    elif which == "k":
        res["out"][t:end, own] = True
        res["dq"][t:end, own, d] = True
        res["dv"][t, kv] = True
    elif which == "v":
        res["out"][t:end, own, d] = True
        res["dq"][t:end, own] = True
        res["dk"][t, kv] = True
    else:
        res["dq"][t, h] = True
        res["dk"][at:t + 1, kv] = True
        res["dv"][at:t + 1, kv, d] = True
    return res


def run(rl, lens, args):
    q, k, v, ld, S, do, dl = cuda(*args)
    cu = bounds(lens).cuda()
    out = rl.rlcs_linear_attention(q, k, v, ld, cu, state=S)
    grads = rl.rlcs_linear_attention_backward(do, q, k, v, ld, cu, state=S, dlast=dl)
    rl.check_scratch()
    return dict(zip(PARTS, (out, *grads[:3])))


def wants(lens, args):
    """Results without what is not finite, and their bounds."""
    q, k, v, ld, S, do, dl = [t if t is None else torch.nan_to_num(t, 0.0, 0.0, 0.0) for t in args]
    leaves = [t.double().requires_grad_() for t in (q, k, v)]
    want, last = ref.linear(*leaves, ld, lens, S)
    loss = (want * do.double()).sum()
    if dl is not None:
        loss = loss + (last * dl.double()).sum()
    grads = torch.autograd.grad(loss, leaves)
    slacks = (ref.slack(q, k, v, ld, lens, S), *ref.backward_slack(do, q, k, v, ld, lens, S, dl))
    return {n: (w.detach(), s) for n, w, s in zip(PARTS, (want, *grads), slacks)}


def check(rl, lens, args, bad):
    q, k, v, ld, S, do, dl = args
    Hq, Hk = q.shape[1], k.shape[1]
    arrays = {"q": q, "k": k, "v": v, "d": do}
    shapes = dict(out=q.shape, dq=q.shape, dk=k.shape, dv=k.shape)
    hit = {n: torch.zeros(s, dtype=torch.bool) for n, s in shapes.items()}
    ends = bounds(lens).tolist()
    for which, t, h, d, value in bad:
        arrays[which][t, h, d] = value
        seq = max(i for i in range(len(lens)) if ends[i] <= t)
        for n, m in reached(which, t, h, d, Hq // Hk, shapes, ends[seq], ends[seq + 1]).items():
            hit[n] |= m
    got = run(rl, lens, args)
    for n, (want, slack) in wants(lens, args).items():
        g = got[n].double().cpu()
        assert torch.equal(~torch.isfinite(g), hit[n]), (n, bad)
        tol = F * torch.maximum(want.abs(), want.square().mean().sqrt()) + 1.87 * slack \
            + U * want.abs()
        off = (g - want).abs()
        assert bool((off <= tol)[~hit[n]].all()), (n, bad, float((off / tol)[~hit[n]].max()))


@pytest.mark.parametrize("lens,Hq,Hk,D,states", [
    ([200], 2, 2, 64, False), ([128], 2, 1, 128, True), ([60, 300], 2, 1, 64, True),
    ([1, 257, 31], 3, 1, 72, False), ([140, 129], 2, 2, 128, True), ([260], 4, 2, 40, True),
    ([2600], 1, 1, 64, True)], ids=str)
@pytest.mark.parametrize("which", ["q", "k", "v", "d"])
def test_one_element(rl, lens, Hq, Hk, D, states, which):
    n = sum(lens)
    heads = Hq if which in "qd" else Hk
    for i, t in enumerate(sorted({0, 31, 32, 100, 128, 133, n - 1})):
        if t < n:
            value = (math.nan, math.inf, -math.inf)[i % 3]
            check(rl, lens, case(n + i, lens, Hq, Hk, D, states, [-0.02, -0.1][:Hk]),
                  [(which, t, i % heads, (7 * i) % D, value)])


def test_several_elements(rl):
    lens = [130, 256, 77]
    check(rl, lens, case(1, lens, 4, 2, 128, True, [-0.02, -0.1]),
          [("v", 120, 0, 3, math.nan), ("k", 129, 1, 9, math.inf), ("v", 200, 0, 127, -math.inf),
           ("v", 330, 1, 64, math.nan), ("d", 400, 3, 0, math.inf), ("q", 460, 0, 33, math.nan)])


def test_nothing_finite(rl):
    lens = [300, 40]
    args = case(2, lens, 2, 1, 64, False)
    for t in (args[0], args[1], args[2], args[5]):
        t.fill_(math.nan)
    for g in run(rl, lens, args).values():
        assert bool(torch.isnan(g).all())


def test_views_and_tokens_of_no_sequence(rl):
    # the element's neighbours are read where they lie: strided heads, an offset
    n, D, first = 400, 64, 30
    args = case(3, [n], 2, 2, D, False, [-0.02, -0.1])
    fused = torch.cat(args[:3], 1)
    fused[first + 90, 4, 7] = math.nan  # a value
    q, k, v = fused.cuda().split([2, 2, 2], 1)
    cu = torch.tensor([first, first + 100, n], dtype=torch.int32)
    ld = args[3]
    out = rl.rlcs_linear_attention(q, k, v, ld.cuda(), cu.cuda()).double().cpu()
    hit = torch.zeros(n, 2, D, dtype=torch.bool)
    hit[first + 90:first + 100, 0, 7] = True
    assert torch.equal(~torch.isfinite(out), hit)
    lens = [100, n - first - 100]
    q, k, v = (torch.nan_to_num(t[first:].cpu(), 0.0) for t in (q, k, v))
    want, slack = ref.linear(q, k, v, ld, lens)[0], ref.slack(q, k, v, ld, lens)
    off = (out[first:] - want).abs()
    tol = F * torch.maximum(want.abs(), want.square().mean().sqrt()) + 1.87 * slack + U * want.abs()
    assert bool((off <= tol)[~hit[first:]].all()) and not out[:first].any()
