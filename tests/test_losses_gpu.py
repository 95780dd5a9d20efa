"""The losses of a policy's logits against their definitions in 64 bits
(tests/loss_reference.py).

Bounds. A float32 result may be off by F = 2e-5 of the larger of its size and
the array's root mean square: an element e_i = 2^y_i carries the rounding of
y_i, |y_i| 2^-24 and a few more, up to 1e-5 where y_i is -100 and e_i far below
anything that counts; a sum of a row some dozens of 2^-24. A bfloat16 gradient
adds one rounding, U = 2^-8 of its size. A log probability is a difference of
numbers up to the row's spread: 4 roundings of that size.
"""
import math

import pytest
import torch

from tests import loss_reference as ref

pytestmark = pytest.mark.gpu

F, U = 2e-5, 2.0 ** -8
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def rl():
    assert torch.cuda.is_available(), "the -m gpu tests need a CUDA device"
    import linear_recurrence_scan_affine_gb300 as m
    return m


def gen(seed):
    return torch.Generator().manual_seed(seed)


def close(name, got, want, slack=0.0):
    want = want.detach().double()
    assert tuple(got.shape) == tuple(want.shape), (name, got.shape, want.shape)
    if want.numel() == 0:
        return
    got64 = got.double().cpu()
    same = torch.isnan(got64) == torch.isnan(want)
    assert bool(same.all()), "%s: NaN elsewhere" % name
    fine = torch.isfinite(want)
    assert torch.equal(got64[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)]), name
    if isinstance(slack, torch.Tensor):
        slack = slack.expand(want.shape)[fine]
    got64, want = got64[fine], want[fine]
    if want.numel() == 0:
        return
    rms = want.square().mean().sqrt()
    tol = F * torch.maximum(want.abs(), rms) + slack
    if got.dtype == torch.bfloat16:
        tol = tol + U * want.abs()
    off = (got64 - want).abs()
    worst = (off / tol.clamp(min=1e-300)).max()
    assert bool((off <= tol).all()), "%s: %.3g times the bound" % (name, worst)


def cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def rows(seed, n, V, dtype, illegal=0.0, spread=2.0):
    """Logits, actions, old and reference log probabilities, advantages; no ratio
    within 1e-3 of a bound, where a rounding would decide which side counts."""
    g = gen(seed)
    x = torch.randn(n, V, generator=g) * spread
    a = torch.randint(0, V, (n,), generator=g, dtype=torch.int32)
    if illegal:
        bad = torch.rand(n, V, generator=g) < illegal
        bad[torch.arange(n), a.long()] = False
        x[bad] = -math.inf
    x = x.to(DT[dtype])
    logp = ref.logs(x).gather(1, a.long()[:, None])[:, 0]
    off = 0.25 * torch.randn(n, generator=g, dtype=torch.float64)
    for edge in (math.log(0.8), math.log(1.2), math.log(0.9), math.log(1.3)):
        off = torch.where((off - edge).abs() < 1e-3, torch.full_like(off, edge + 2e-3), off)
    old = (logp - off).float()
    against = (logp + 0.3 * torch.randn(n, generator=g, dtype=torch.float64)).float()
    adv = torch.randn(n, generator=g)
    mask = torch.rand(n, generator=g) < 0.7
    return x, a, old, adv, against, mask, torch.randn(n, generator=g)


def logp_slack(x):
    finite = torch.where(torch.isfinite(x.double()), x.double(), torch.zeros(()).double())
    return 4 * 2.0 ** -24 * (finite.amax() - finite.amin() + math.log(x.shape[1]) + 1)


SIZES = [1, 2, 3, 6, 7, 8, 31, 32, 33, 64, 65, 100, 255, 256, 257, 511, 1000, 1023, 1024, 1025,
         2049, 4100, 8191, 16384, 32001, 50001, 70000, 131075, 262147]


def check_policy(rl, data, kl_coef=0.0, ent=0.0, low=0.2, high=0.2, use_ref=True, use_mask=True):
    x, a, old, adv, against, mask, w = data
    against = against if use_ref else None
    mask = mask if use_mask else None
    cx, ca, co, cadv, cr, cm, cw = cuda(x, a, old, adv, against, mask, w)
    kw = dict(ref_logp=cr, mask=cm, clip_low=low, clip_high=high, kl_coef=kl_coef,
              entropy_coef=ent)
    got = rl.rlcs_policy_loss(cx, ca, co, cadv, **kw)
    dx, both = rl.rlcs_policy_loss_backward(cw, cx, ca, co, cadv, return_loss=True, **kw)
    alone = rl.rlcs_policy_loss_backward(cw, cx, ca, co, cadv, **kw)
    x64 = x.double().requires_grad_()
    want = ref.policy(x64, a, old, adv, against, mask, low, high, kl_coef, ent)
    ls = logp_slack(x)
    for name, g, w_ in zip(("loss", "logp", "entropy", "kl"), got, want):
        if w_ is None:
            assert g is None and both.kl is None
        else:
            # a loss and a KL term move with logp: by the ratio's and exp(d)'s slopes
            close(name, g, w_, ls * (4.0 if name in ("loss", "kl") else 1.0))
            assert torch.equal(g, getattr(both, name)), name
    wdx, = torch.autograd.grad((want[0] * w.double()).sum(), x64)
    # a row's slope moves with logp too
    slope = 4.0 * ls * (w.abs() * (adv.abs() + kl_coef + abs(ent))).double()[:, None]
    p = torch.softmax(x.double(), 1)
    p.scatter_add_(1, a.long()[:, None], torch.ones(len(a), 1, dtype=torch.float64))
    close("dlogits", dx, wdx, slope * p)
    assert torch.equal(dx, alone)

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,V,below", [(1, 26, 60.0), (3, 130, 20.0), (2, 1000, 60.0),
                                       (4, 20000, 30.0), (300, 5, 60.0), (1, 131075, 80.0)])
def test_policy_close_to_its_reference(rl, dtype, n, V, below):
    """kl where ref_logp is within a hundredth of a log probability far below 0:
    off by (e^d - 1) times the error of l, which is that of log z alone, not a
    rounding of l's own size (2^-24 below). z: 2^-22 from each power of two, a few
    2^-24 from the rounded exponents near the top and some from adding: 2^-20.
    kl itself comes from d by a few roundings, 2^-21 of it."""
    g = gen(V + n)
    x = (2.0 * torch.randn(n, V, generator=g)).to(DT[dtype])
    a = torch.randint(0, V, (n,), generator=g, dtype=torch.int32)
    x[torch.arange(n), a.long()] = -below - 3.0 * torch.rand(n, generator=g).to(DT[dtype])
    l = ref.logs(x).gather(1, a.long()[:, None])[:, 0]
    against = (l + 0.01 * torch.randn(n, generator=g, dtype=torch.float64)).float()
    old, adv = l.float(), torch.randn(n, generator=g)
    want = ref.policy(x, a, old, adv, against)
    got = rl.rlcs_policy_loss(*cuda(x, a, old, adv), ref_logp=against.cuda())
    d = against.double() - l
    tol = torch.expm1(d).abs() * 2.0 ** -20 + want[3] * 2.0 ** -21 + 2.0 ** -40
    off = (got.kl.double().cpu() - want[3]).abs()
    assert bool((off <= tol).all()), float((off / tol).max())
    off = (got.logp.double().cpu() - l).abs()  # one rounding, to the type it has
    assert bool((off <= 2.0 ** -20 + l.abs() * 2.0 ** -24).all())



@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", SIZES)
def test_policy_sizes(rl, V, dtype):
    n = max(3, min(300, 400000 // V))
    check_policy(rl, rows(V, n, V, dtype), kl_coef=0.1, ent=0.02)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,V", [(1, 6), (5000, 6), (4099, 33), (700, 640), (257, 5000)])
def test_policy_terms(rl, n, V, dtype):
    data = rows(n + V, n, V, dtype, illegal=0.3)
    check_policy(rl, data)
    check_policy(rl, data, use_ref=False, use_mask=False)
    check_policy(rl, data, kl_coef=0.2, use_mask=False)
    check_policy(rl, data, ent=0.1, use_ref=False)
    check_policy(rl, data, kl_coef=0.05, ent=-0.1, low=0.1, high=0.3)


@pytest.mark.parametrize("V", [700001, 1100003])
def test_policy_very_long_rows(rl, V):
    check_policy(rl, rows(V, 3, V, "f32"), kl_coef=0.1, ent=0.02)
    check_policy(rl, rows(V, 3, V, "bf16"), kl_coef=0.1)


def test_clipping(rl):
    # ratios on both sides of both bounds, both signs of the advantage, zero advantage
    logit = torch.zeros(12, 4)
    ratio = torch.tensor([0.5, 0.5, 0.5, 1.0, 1.0, 1.0, 2.0, 2.0, 2.0, 0.79, 1.21, 1.19])
    adv = torch.tensor([1.0, -1, 0, 1, -1, 0, 1, -1, 0, -1, 1, 1])
    old = math.log(0.25) - ratio.log()
    a = torch.zeros(12, dtype=torch.int32)
    cx, ca, co, cadv = cuda(logit, a, old, adv)
    dx, got = rl.rlcs_policy_loss_backward(torch.ones(12).cuda(), cx, ca, co, cadv,
                                           return_loss=True)
    want = torch.tensor([-0.5, 0.8, 0, -1, 1, 0, -1.2, 2, 0, 0.8, -1.2, -1.19])
    close("loss", got.loss, want)
    slope = torch.tensor([-0.5, 0, 0, -1, 1, 0, 0, 2, 0, 0, 0, -1.19])
    close("dlogits", dx, slope[:, None] * (torch.eye(4)[0] - 0.25))


def test_small_kl_keeps_its_digits(rl):
    # d from 1e-5 to 3: kl is d^2 / 2 and more, no difference of rounded numbers.
    # One action of two has probability 1/2 exactly, so that d is the input.
    d = torch.cat([torch.logspace(-5, 0.5, 200), -torch.logspace(-5, 0.5, 200)])
    n = len(d)
    half = torch.full((n,), math.log(0.5), dtype=torch.float64)
    x = torch.zeros(n, 2)
    against = (half + d.double()).float()
    z = torch.zeros(n)
    a = torch.zeros(n, dtype=torch.int32)
    kl = rl.rlcs_policy_loss(*cuda(x, a, z, z), ref_logp=against.cuda()).kl.double().cpu()
    # log 0.5 is off by up to 2^-25, and so is d; the rest is a few roundings
    true = against.double() - half
    want = torch.expm1(true) - true
    off = (kl - want).abs()
    assert bool((off <= 2.0 ** -23 * true.expm1().abs() + 1e-6 * want + 1e-14).all())
    assert bool((kl >= 0).all())


def check_distill(rl, seed, n, V, K, dtype, temperature=1.0, whole=False, absent=0.0, mask=True,
                  repeat=False):
    x = rows(seed, n, V, dtype)[0]
    g = gen(seed + 1)
    ids = torch.stack([torch.randperm(V, generator=g)[:K] if V < 5000
                       else torch.randint(0, V, (K,), generator=g) for _ in range(n)])
    if repeat:
        ids = ids[:, torch.randint(0, K, (K,), generator=g)]
    ids = ids.to(torch.int32)
    top = torch.randn(n, K, generator=g) * 2.0
    if absent:
        r = torch.rand(n, K, generator=g)
        ids[r < absent] = -1
        ids[(r >= absent) & (r < 1.5 * absent)] = V
        top[r > 1 - absent] = -math.inf
        ids[0] = -5  # a row without an entry
    lse = (torch.logsumexp(top / temperature, 1) + 0.4).clamp(min=-50.0) if whole else None
    m = torch.rand(n, generator=g) < 0.7 if mask else None
    w = torch.randn(n, generator=g)
    cx, ci, ct, cl, cm, cw = cuda(x, ids, top, lse, m, w)
    kw = dict(teacher_lse=cl, mask=cm, temperature=temperature)
    loss = rl.rlcs_distill_loss(cx, ci, ct, **kw)
    dx, both = rl.rlcs_distill_loss_backward(cw, cx, ci, ct, return_loss=True, **kw)
    assert torch.equal(loss, both)
    assert torch.equal(dx, rl.rlcs_distill_loss_backward(cw, cx, ci, ct, **kw))
    x64 = x.double().requires_grad_()
    want = ref.distill(x64, ids, top, lse, m, temperature)
    # sums of terms that cancel: their sizes' logs, at most the rows' spread
    close("loss", loss, want, logp_slack(x) / temperature + 2.0 ** -20)
    wdx, = torch.autograd.grad((want * w.double()).sum(), x64)
    # p and its target cancel: what is left of their roundings to float32, some
    # 2^-24 of each, is there before a rounding to bfloat16 too
    close("dlogits", dx, wdx, 2.0 ** -19 * (w.abs().double() / temperature)[:, None]
          * torch.softmax(x.double() / temperature, 1).clamp(min=1e-30))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", SIZES)
def test_distill_sizes(rl, V, dtype):
    n = max(3, min(200, 400000 // V))
    check_distill(rl, V, n, V, min(V, 20), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,V,K", [(1, 1, 1), (300, 7, 7), (50, 600, 33), (20, 3000, 257),
                                   (4, 9000, 1024)])
def test_distill_terms(rl, n, V, K, dtype):
    for t, whole, absent, mask in ((1.0, False, 0.2, False), (2.0, True, 0.0, True),
                                   (0.5, True, 0.3, True), (3.0, False, 0.0, False)):
        check_distill(rl, n + V, n, V, K, dtype, t, whole, absent, mask)
    check_distill(rl, n + V, n, V, K, dtype, repeat=True)


@pytest.mark.parametrize("V", [700001, 1100003])
def test_distill_very_long_rows(rl, V):
    check_distill(rl, V, 3, V, 40, "f32", repeat=True)
    check_distill(rl, V, 3, V, 40, "bf16", 2.0)


def both(rl, x, seed=0, K=3):
    """Every output of both losses on these logits, in place of nothing."""
    n, V = x.shape
    g = gen(seed)
    a = torch.randint(0, V, (n,), generator=g, dtype=torch.int32).cuda()
    one = torch.ones(n).cuda()
    ids = torch.randint(0, V, (n, K), generator=g, dtype=torch.int32).cuda()
    top = torch.randn(n, K, generator=g).cuda()
    dx, p = rl.rlcs_policy_loss_backward(one, x, a, -one, one, ref_logp=-one, kl_coef=0.1,
                                         entropy_coef=0.1, return_loss=True)
    dy, d = rl.rlcs_distill_loss_backward(one, x, ids, top, return_loss=True)
    return [dx, *p, dy, d]


def near(a, b):
    """Two results that each keep their bound: a row may be summed in another order
    where it starts elsewhere in a 16-byte word, or comes with other rows."""
    a, b = a.double(), b.double()
    off, rms = (a - b).abs(), b.square().mean().sqrt()
    return bool((off <= 2 * F * torch.maximum(b.abs(), rms) + 2 * U * b.abs()).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [5, 40, 900, 5001, 40000])
def test_rows_apart(rl, V, dtype):
    # rows inside wider ones, starting at every place of a 16-byte word
    n = 6
    wide = (torch.randn(n, V + 24, generator=gen(V)) * 2).to(DT[dtype]).cuda()
    for shift in (0, 1, 2, 5, 7, 8):
        x = wide[:, shift:shift + V]
        want = both(rl, x.contiguous())
        for a, b in zip(both(rl, x), want):
            assert near(a, b)
    flat = (torch.randn(n * V + 9, generator=gen(V)) * 2).to(DT[dtype]).cuda()
    for shift in (1, 3, 8):
        x = flat[shift:shift + n * V].view(n, V)
        for a, b in zip(both(rl, x), both(rl, x.clone())):
            assert near(a, b)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [6, 70, 1001, 9000, 33333, 150000])
def test_in_place(rl, V, dtype):
    n = 7
    x, a, old, adv, against, mask, w = cuda(*rows(3, n, V, dtype))
    kw = dict(ref_logp=against, mask=mask, kl_coef=0.1, entropy_coef=0.01)
    want = rl.rlcs_policy_loss_backward(w, x, a, old, adv, **kw)
    y = x.clone()
    got = rl.rlcs_policy_loss_backward(w, y, a, old, adv, out=y, **kw)
    assert got.data_ptr() == y.data_ptr() and torch.equal(got, want)
    ids = torch.randint(0, V, (n, 5), generator=gen(1), dtype=torch.int32).cuda()
    top = torch.randn(n, 5, generator=gen(2)).cuda()
    want = rl.rlcs_distill_loss_backward(w, x, ids, top, mask=mask)
    got = rl.rlcs_distill_loss_backward(w, x, ids, top, mask=mask, out=x)
    assert got.data_ptr() == x.data_ptr() and torch.equal(got, want)


@pytest.mark.parametrize("V,dtype", [(120000, "f32"), (250000, "bf16")])
def test_in_place_with_many_entries(rl, V, dtype):
    # rows that blocks of a cluster share: none may write over a logit that
    # another has still to read for its entries
    n, K = 400, 1000
    x = (torch.randn(n, V, device="cuda") * 2).to(DT[dtype])
    ids = torch.randint(0, V, (n, K), device="cuda", dtype=torch.int32)
    top, w = torch.randn(n, K, device="cuda"), torch.rand(n, device="cuda") + 0.5
    want, loss = rl.rlcs_distill_loss_backward(w, x, ids, top, return_loss=True)
    for _ in range(3):
        y = x.clone()
        got, same = rl.rlcs_distill_loss_backward(w, y, ids, top, out=y, return_loss=True)
        assert torch.equal(same, loss) and torch.equal(got, want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [6, 33, 1000, 5000, 40001, 140000])
def test_rows_that_are_not_finite(rl, V, dtype):
    n = 9
    x, a, old, adv, against, mask, w = rows(4, n, V, dtype)
    clean = rl.rlcs_policy_loss(*cuda(x, a, old, adv))
    x[1, V // 2] = math.nan
    x[2, V - 1] = math.inf
    x[3] = -math.inf
    x[4] = torch.finfo(x.dtype).min          # all at the lowest value: all alike
    x[5, 1:] = torch.finfo(x.dtype).min      # one left
    x[6, :V - 1] = -math.inf                 # the last one left
    a[5], a[6] = 0, V - 1
    dx, got = rl.rlcs_policy_loss_backward(*cuda(w, x, a, old, adv), entropy_coef=0.1,
                                           return_loss=True)
    for t in got[:3]:
        assert bool(torch.isnan(t[1:4]).all()) and bool(torch.isfinite(t[4:]).all())
        assert bool(torch.isfinite(t[0]))
    assert bool(torch.isnan(dx[1:4].float()).all())
    assert bool(torch.isfinite(dx[4:].float()).all()) and bool(torch.isfinite(dx[0].float()).all())
    for i in (0, 7, 8):
        assert got.logp[i] == clean.logp[i]
    assert abs(float(got.logp[4]) + math.log(V)) < 1e-5 * math.log(V)
    assert abs(float(got.entropy[4]) - math.log(V)) < 1e-5 * math.log(V)
    for i in (5, 6):
        # certain: to a few roundings of c x's size, and on the right side
        size = 4 * 2.0 ** -24 * (1 + 2 * abs(float(x[i, a[i]])))
        assert -size <= float(got.logp[i]) <= 0.0 and 0.0 <= float(got.entropy[i]) <= size
        scale = abs(float(w[i])) * (1 + abs(float(adv[i])) * math.exp(-float(old[i])))
        assert float(dx[i].abs().max()) <= size * scale
    # masked tokens: nothing of them counts
    off = torch.ones(n, dtype=torch.bool)
    off[1:4] = False
    for t in (old, adv, w):
        t[1:4] = math.nan
    a[1:4] = -1
    dx, got = rl.rlcs_policy_loss_backward(*cuda(w, x, a, old, adv), mask=off.cuda(),
                                           entropy_coef=0.1, return_loss=True)
    for t in (dx, *got[:3]):
        assert not t[1:4].any() and bool(torch.isfinite(t.float()).all())
    ids = torch.zeros(n, 2, dtype=torch.int32)
    top = torch.zeros(n, 2)
    ids[1:4] = -1                            # rows without an entry: the same
    w[1:4] = 1.0
    dx, loss = rl.rlcs_distill_loss_backward(*cuda(w, x, ids, top), return_loss=True)
    assert not loss[1:4].any() and not dx[1:4].any()
    ids[1:4] = 0
    dx, loss = rl.rlcs_distill_loss_backward(*cuda(w, x, ids, top), return_loss=True)
    assert bool(torch.isnan(loss[1:4]).all()) and bool(torch.isnan(dx[1:4].float()).all())
    assert bool(torch.isfinite(dx[4:6].float()).all())


@pytest.mark.parametrize("V", [6, 500, 40000])
def test_actions_outside(rl, V):
    x, a, old, adv, against, mask, w = rows(5, 5, V, "f32")
    a[1], a[3] = -1, V
    dx, got = rl.rlcs_policy_loss_backward(*cuda(w, x, a, old, adv), ref_logp=against.cuda(),
                                           return_loss=True)
    for t in (got.loss, got.logp, got.kl):
        assert torch.isnan(t).tolist() == [False, True, False, True, False]
    assert bool(torch.isfinite(got.entropy).all())
    assert bool(torch.isnan(dx[[1, 3]]).all()) and bool(torch.isfinite(dx[[0, 2, 4]]).all())


def test_large_logits(rl):
    # a common offset costs no digits: exponents c x - m are rounded once, at
    # their own size, and what m was rounded by is in all of them and in the sum
    # alike. So results move by roundings of the row's spread, as logp_slack has
    # them, not of the offset (4096 * 2^-24 would be 40 times more).
    x, a, old, adv, against, mask, w = rows(6, 50, 300, "f32")
    x = (x * 8).round() / 8  # multiples of 1/8: 4096 + x is exact
    tol = logp_slack(x)
    for off in (4096.0, -4096.0):
        got = rl.rlcs_policy_loss(*cuda(x + off, a, old, adv))
        want = rl.rlcs_policy_loss(*cuda(x, a, old, adv))
        assert float((got.logp - want.logp).abs().max()) <= 2 * tol
        assert float((got.entropy - want.entropy).abs().max()) <= 2 * tol
        assert bool(((got.loss - want.loss).abs() <= 8 * tol * (1 + adv.abs().cuda())).all())


def test_gradient_against_differences(rl):
    # along a direction u: the central difference's truncation is eps^2 / 6 times
    # a third derivative of order |u|^3 per row, its rounding F / eps per loss
    n, V = 40, 30
    x, a, old, adv, against, _, w = rows(7, n, V, "f32")
    u = torch.randn(n, V, generator=gen(8))
    eps = 2.0 ** -6
    kw = dict(ref_logp=against.cuda(), kl_coef=0.3, entropy_coef=0.2, clip_low=1.0, clip_high=1e6)
    dx = rl.rlcs_policy_loss_backward(*cuda(w, x, a, old, adv), **kw).double().cpu()
    up, down = (rl.rlcs_policy_loss(*cuda(x + e * u, a, old, adv), **kw).loss.double().cpu()
                for e in (eps, -eps))
    off = (up - down) / (2 * eps) * w.double() - (dx * u.double()).sum(1)
    size = w.abs().double() * (adv.abs().double() + 1.0) * 4.0  # ratios stay below 4
    assert bool((off.abs() <= size * (eps ** 2 * u.abs().amax(1).double() ** 3 + F / eps)).all())
    ids = torch.stack([torch.randperm(V, generator=gen(i))[:6] for i in range(n)]).int()
    top = torch.randn(n, 6, generator=gen(9))
    for t in (1.0, 2.0):
        kw = dict(temperature=t)
        dx = rl.rlcs_distill_loss_backward(*cuda(w, x, ids, top), **kw).double().cpu()
        up, down = (rl.rlcs_distill_loss(*cuda(x + e * u, ids, top), **kw).double().cpu()
                    for e in (eps, -eps))
        off = (up - down) / (2 * eps) * w.double() - (dx * u.double()).sum(1)
        size = w.abs().double() * 4.0
        assert bool((off.abs() <= size * (eps ** 2 * u.abs().amax(1).double() ** 3
                                          + F / eps)).all())


def test_empty_calls(rl):
    x = torch.zeros(0, 5).cuda()
    e, i = torch.zeros(0).cuda(), torch.zeros(0, dtype=torch.int32).cuda()
    dx, got = rl.rlcs_policy_loss_backward(e, x, i, e, e, return_loss=True)
    assert dx.shape == (0, 5) and got.loss.shape == (0,) and got.kl is None
    dx, loss = rl.rlcs_distill_loss_backward(e, x, i[:, None], e[:, None], return_loss=True)
    assert dx.shape == (0, 5) and loss.shape == (0,)


def test_every_element_is_written(rl):
    for V in (6, 100, 3001, 50000, 300000):
        x = torch.randn(5, V, generator=gen(V)).cuda()
        torch.full((8 << 20,), math.nan, device="cuda")  # memory the results may come from
        for t in both(rl, x):
            assert bool(torch.isfinite(t).all()), V


def test_repeats_streams_and_graphs(rl):
    for V, dtype in ((6, "f32"), (700, "bf16"), (30001, "bf16"), (140000, "f32")):
        x = rows(V, 40, V, dtype)[0].cuda()
        want = both(rl, x)
        assert all(torch.equal(a, b) for a, b in zip(want, both(rl, x)))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            other = both(rl, x)
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(want, other))
        n = x.shape[0]
        a = torch.zeros(n, dtype=torch.int32).cuda()
        one = torch.ones(n).cuda()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            dx, got = rl.rlcs_policy_loss_backward(one, x, a, -one, one, return_loss=True)
        x.mul_(0.5)
        want, wl = rl.rlcs_policy_loss_backward(one, x, a, -one, one, return_loss=True)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(dx, want) and torch.equal(got.loss, wl.loss)


def test_offsets_past_32_bits(rl):
    n, V = 70001, 32000  # 2.24e9 elements
    x = torch.randn(n, V, device="cuda", dtype=torch.bfloat16)
    a = torch.randint(0, V, (n,), device="cuda", dtype=torch.int32)
    one = torch.ones(n, device="cuda")
    got = rl.rlcs_policy_loss_backward(one, x, a, -one, one, out=x.clone(), entropy_coef=0.1)
    want = rl.rlcs_policy_loss_backward(one[-9:], x[-9:], a[-9:], -one[-9:], one[-9:],
                                        entropy_coef=0.1)
    assert near(got[-9:], want)


def test_refusals(rl):
    x = torch.zeros(4, 5).cuda()
    a, one = torch.zeros(4, dtype=torch.int32).cuda(), torch.ones(4).cuda()
    ids, top = torch.zeros(4, 2, dtype=torch.int32).cuda(), torch.zeros(4, 2).cuda()
    pol, back = rl.rlcs_policy_loss, rl.rlcs_policy_loss_backward
    dis, dback = rl.rlcs_distill_loss, rl.rlcs_distill_loss_backward
    for bad in (lambda: pol(x.half(), a, one, one), lambda: pol(x[0], a, one, one),
                lambda: pol(x, a.long(), one, one), lambda: pol(x, a[:3], one, one),
                lambda: pol(x, a, one.double(), one), lambda: pol(x, a, one, one.cpu()),
                lambda: pol(x, a, one, one, mask=one), lambda: pol(x, a, one, one, ref_logp=one[:2]),
                lambda: back(one[:2], x, a, one, one),
                lambda: back(one, x, a, one, one, out=x[:, :4]),
                lambda: back(one, x, a, one, one, out=x.bfloat16()),
                lambda: dis(x, ids.long(), top), lambda: dis(x, ids, top[:, :1]),
                lambda: dis(x, ids[:3], top), lambda: dis(x, ids, top.bfloat16()),
                lambda: dis(x, ids, top, teacher_lse=one[:1]),
                lambda: dback(one, x, ids, top, out=x.t())):
        with pytest.raises((ValueError, TypeError)):
            bad()
    for bad in (lambda: pol(x, a, one, one, clip_low=-0.1), lambda: pol(x, a, one, one, clip_low=1.1),
                lambda: pol(x, a, one, one, clip_high=math.nan),
                lambda: pol(x, a, one, one, kl_coef=0.1),
                lambda: pol(x, a, one, one, entropy_coef=math.inf),
                lambda: pol(x[:, :0], a, one, one),
                lambda: dis(x, ids, top, temperature=0.0), lambda: dis(x, ids[:, :0], top[:, :0]),
                lambda: dis(x, ids.repeat(1, 513), top.repeat(1, 513))):
        with pytest.raises(rl.RlcsError):
            bad()
    # an output that lies partly on the logits
    flat = torch.zeros(25).cuda()
    with pytest.raises(rl.RlcsError):
        back(one, flat[:20].view(4, 5), a, one, one, out=flat[5:].view(4, 5))
