"""Every element of a result is written, whatever part of its tokens the
sequences hold. New tensors start as NaN here."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rl():
    assert torch.cuda.is_available(), "the -m gpu tests need a CUDA device"
    import linear_recurrence_scan_affine_gb300 as m
    return m


@pytest.fixture
def poisoned(monkeypatch):
    """torch.empty fills what it makes with NaN (or ones, where there is none)."""
    empty = torch.empty

    def filled(*args, **kw):
        t = empty(*args, **kw)
        return t.fill_(math.nan if t.is_floating_point() else 255)
    monkeypatch.setattr(torch, "empty", filled)


# bounds that begin late, end early, or hold nothing; tokens
BOUNDS = [([40, 150], 200), ([0, 129], 130), ([0, 128, 128, 256], 256), ([1, 2], 3), ([7, 7, 7], 9),
          ([0, 0], 500), ([900, 1000, 1100], 2500), ([0], 70), ([5, 300], 300), ([64, 192], 192),
          ([0, 20, 70], 71)]


@pytest.mark.parametrize("Hq,Hk,D", [(2, 2, 64), (8, 1, 128), (4, 2, 80), (6, 2, 8)])
@pytest.mark.parametrize("cu,n", BOUNDS, ids=lambda v: str(v).replace(", ", "-"))
def test_attention_rows_no_sequence_holds(rl, poisoned, cu, n, Hq, Hk, D):
    g = torch.Generator().manual_seed(n + D)
    q, k, v, dout = (torch.randn(n, h, D, generator=g).bfloat16().cuda() for h in (Hq, Hk, Hk, Hq))
    bounds = torch.tensor(cu, dtype=torch.int32).cuda()
    held = torch.zeros(n, dtype=torch.bool).cuda()
    held[cu[0]:cu[-1]] = True
    out, lse = rl.rlcs_attention(q, k, v, bounds, return_lse=True)
    grads = rl.rlcs_attention_backward(dout, q, k, v, out, lse, bounds)
    for t in (out, *grads):
        assert float(t[~held].float().abs().sum()) == 0.0  # NaN would not be
        assert torch.isfinite(t).all()
    assert bool((lse[:, ~held] == -math.inf).all()) and torch.isfinite(lse[:, held]).all()
    # the rows that are held do not depend on the others
    part = [t[cu[0]:cu[-1]].contiguous() for t in (q, k, v, dout)]
    inner = bounds - cu[0]
    o2, l2 = rl.rlcs_attention(*part[:3], inner, return_lse=True)
    assert torch.equal(out[held], o2) and torch.equal(lse[:, held], l2)
    for a, b in zip(grads, rl.rlcs_attention_backward(part[3], *part[:3], o2, l2, inner)):
        # (a group's query heads may be shared by more blocks: another order of sums)
        assert torch.allclose(a[held].float(), b.float(), rtol=2.0 ** -7, atol=2.0 ** -12)


@pytest.mark.parametrize("D", [64, 7])
@pytest.mark.parametrize("n", [0, 5])
def test_norm_gradient_without_key_heads(rl, poisoned, n, D):
    g = torch.Generator().manual_seed(1)
    q, dq = (torch.randn(n, 3, D, generator=g).cuda() for _ in range(2))
    k, w = torch.zeros(n, 0, D).cuda(), torch.ones(D).cuda()
    cos = sin = torch.ones(4, 0).cuda()
    pos = torch.zeros(n, dtype=torch.int32).cuda()
    got = rl.rlcs_qk_norm_rope_backward(dq, k, q, k, w, w, cos, sin, pos)
    assert float(got[3].abs().sum()) == 0.0
    assert torch.isfinite(got[0]).all() and torch.isfinite(got[2]).all()
