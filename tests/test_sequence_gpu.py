"""The sequence operators against their definitions in 64 bits.

Bounds. A float32 result may be off by F = 2e-5 of the larger of its size and
the array's root mean square: a few hundred roundings of 2^-24, with room for
the gates' fast exponential (2 ulp). A bfloat16 result adds one rounding,
U = 2^-8 of its size; the attention results and the gate's gradient add the
slack of their documented inner roundings (tests/sequence_reference.py).
"""
import math

import pytest
import torch

from tests import sequence_reference as ref

pytestmark = pytest.mark.gpu

F, U = 2e-5, ref.U
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def rl():
    assert torch.cuda.is_available(), "the -m gpu tests need a CUDA device"
    import linear_recurrence_scan_affine_gb300 as m
    return m


def rand(gen, *shape, scale=1.0, shift=0.0, dtype=torch.float32):
    return (torch.randn(shape, generator=gen) * scale + shift).to(dtype)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def close(name, got, want, slack=0.0):
    want = want.double()
    assert tuple(got.shape) == tuple(want.shape), (name, got.shape, want.shape)
    if want.numel() == 0:
        return
    rms = want.square().mean().sqrt()
    tol = F * torch.maximum(want.abs(), rms) + slack
    if got.dtype == torch.bfloat16:
        tol = tol + U * want.abs()
    off = (got.double().cpu() - want).abs()
    worst = (off / tol.clamp(min=1e-300)).max()
    assert bool((off <= tol).all()), "%s: %.3g times the bound" % (name, worst)


def cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


# ---------------------------------------------------------------------------
# Gated linear recurrence
# ---------------------------------------------------------------------------
SCAN_SHAPES = [(1, 1, 1), (2, 1, 64), (1, 15, 3), (3, 16, 33), (2, 17, 64), (1, 127, 130),
               (2, 128, 66), (2, 129, 31), (1, 1000, 256), (5, 300, 70), (1, 5000, 40),
               (40, 33, 96), (1, 20000, 64), (2, 4099, 520)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,D", SCAN_SHAPES)
@pytest.mark.parametrize("extras", [False, True])
def test_gated_scan_and_gradient(rl, B, T, D, dtype, extras):
    g, dt = gen(B * 7919 + T * 31 + D), DT[dtype]
    x, dh = rand(g, B, T, D, dtype=dt), rand(g, B, T, D, dtype=dt)
    gate = rand(g, B, T, D, scale=2.0, shift=2.0, dtype=dt)
    reset = h0 = dh_last = None
    if extras:
        reset = torch.rand(B, T, generator=g) < 0.05
        h0, dh_last = rand(g, B, D), rand(g, B, D)
    cx, cg, cr, c0, cd, cl = cuda(x, gate, reset, h0, dh, dh_last)
    h, last = rl.rlcs_gated_scan(cx, cg, reset=cr, h0=c0)
    want = ref.gated_scan(x, gate, reset, h0)
    close("h", h, want)
    close("h_last", last, want[:, -1])
    dx, dg, dh0 = rl.rlcs_gated_scan_backward(cd, cx, cg, h, reset=cr, h0=c0, dh_last=cl)
    wx, wg, w0, slack = ref.gated_scan_backward(dh, x, gate, reset, h0, dh_last)
    close("dx", dx, wx)
    close("dgate", dg, wg, slack if dtype == "bf16" else 0.0)
    close("dh0", dh0, w0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,D", [(1, 6000, 33), (2, 4500, 130), (20, 700, 72), (1000, 130, 40),
                                   (30, 150, 65), (800, 140, 3)])
def test_gated_scan_shares(rl, B, T, D, dtype):
    # walks shared by clusters of 16, 8 and 1 blocks and by single warps, over
    # channels that fill a warp's columns and ones that do not
    g, dt = gen(B + T + D), DT[dtype]
    x, dh = rand(g, B, T, D, dtype=dt), rand(g, B, T, D, dtype=dt)
    gate = rand(g, B, T, D, scale=2.0, shift=3.0, dtype=dt)
    reset = torch.rand(B, T, generator=g) < 0.01
    cx, cg, cr, cd = cuda(x, gate, reset, dh)
    h, last = rl.rlcs_gated_scan(cx, cg, reset=cr)
    want = ref.gated_scan(x, gate, reset)
    close("h", h, want)
    close("h_last", last, want[:, -1])
    got = rl.rlcs_gated_scan_backward(cd, cx, cg, h, reset=cr)
    again = rl.rlcs_gated_scan_backward(cd, cx, cg, h, reset=cr)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    wx, wg, w0, slack = ref.gated_scan_backward(dh, x, gate, reset)
    close("dx", got[0], wx)
    close("dgate", got[1], wg, slack if dtype == "bf16" else 0.0)
    close("dh0", got[2], w0)


def test_gated_scan_gradient_against_differences(rl):
    # the directional derivative of sum(h * dh), in float32: the quotient's own
    # rounding is about 2^-24 / eps of the terms' root sum of squares
    g = gen(5)
    B, T, D = 2, 200, 48
    x, gate, dh = rand(g, B, T, D), rand(g, B, T, D, scale=1.5, shift=1.0), rand(g, B, T, D)
    reset = torch.rand(B, T, generator=g) < 0.03
    h0, u, w, z = rand(g, B, D), rand(g, B, T, D), rand(g, B, T, D), rand(g, B, D)
    cx, cg, cd, cr, c0 = cuda(x, gate, dh, reset, h0)
    h, _ = rl.rlcs_gated_scan(cx, cg, reset=cr, h0=c0)
    dx, dg, dh0 = rl.rlcs_gated_scan_backward(cd, cx, cg, h, reset=cr, h0=c0)
    grad = float((dx.cpu().double() * u).sum() + (dg.cpu().double() * w).sum()
                 + (dh0.cpu().double() * z).sum())
    eps = 2.0 ** -7
    side = []
    for e in (eps, -eps):
        he, _ = rl.rlcs_gated_scan((x + e * u).cuda(), (gate + e * w).cuda(), reset=cr,
                                   h0=(h0 + e * z).cuda())
        side.append(float((he.cpu().double() * dh).sum()))
    size = math.sqrt(B * T * D)
    assert abs((side[0] - side[1]) / (2 * eps) - grad) < 40 * eps * eps * size + 1e-4 * size


def test_gated_scan_saturated_gates(rl):
    # gates far out on both sides: carried unchanged, or dropped, without overflow
    T = 300
    x = torch.linspace(-2, 2, T).view(1, T, 1).repeat(1, 1, 4)
    gate = torch.tensor([200.0, -200.0, 80.0, -80.0]).view(1, 1, 4).repeat(1, T, 1)
    h0 = torch.full((1, 4), 3.0)
    h, last = rl.rlcs_gated_scan(x.cuda(), gate.cuda(), h0=h0.cuda())
    close("h", h, ref.gated_scan(x, gate, None, h0))
    assert torch.equal(h[0, :, 0].cpu(), torch.full((T,), 3.0))
    assert torch.equal(h[0, :, 1].cpu(), x[0, :, 1])


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_gated_scan_cuts_stop_non_finite_states(rl, bad):
    g = gen(11)
    B, T, D = 1, 700, 34
    x, gate, dh = rand(g, B, T, D), rand(g, B, T, D), rand(g, B, T, D)
    reset = torch.zeros(B, T, dtype=torch.bool)
    reset[0, 130] = reset[0, 401] = True
    clean = x.clone()
    x[0, 200:380] = bad
    cx, cg, cr, cd = cuda(x, gate, reset, dh)
    h, _ = rl.rlcs_gated_scan(cx, cg, reset=cr)
    want = ref.gated_scan(clean, gate, reset)
    close("before", h[:, :200], want[:, :200])
    close("after", h[:, 401:], want[:, 401:])
    cd[0, 200:380] = bad
    dx, dg, _ = rl.rlcs_gated_scan_backward(cd, cx, cg, h, reset=cr)
    wx, wg, _, _ = ref.gated_scan_backward(dh, clean, gate, reset)
    close("dx", dx[:, 401:], wx[:, 401:])
    close("dx", dx[:, :130], wx[:, :130])
    close("dgate", dg[:, 401:], wg[:, 401:])
    close("dgate", dg[:, :130], wg[:, :130])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,D", [(1, 1), (7, 33), (64, 512), (3, 1030)])
def test_gated_step_continues_the_scan(rl, B, D, dtype):
    g, dt = gen(B + D), DT[dtype]
    x, gate = rand(g, B, 6, D, dtype=dt), rand(g, B, 6, D, shift=1.0, dtype=dt)
    reset = torch.rand(B, 6, generator=g) < 0.2
    want = ref.gated_scan(x, gate, reset)
    cx, cg, cr = cuda(x, gate, reset)
    _, state = rl.rlcs_gated_scan(cx[:, :3], cg[:, :3], reset=cr[:, :3])
    for t in range(3, 6):
        old = state.clone()
        h, new = rl.rlcs_gated_step(cx[:, t], cg[:, t], state, reset=cr[:, t])
        assert torch.equal(state, old)  # not updated unless asked to
        close("h", h, want[:, t])
        close("state", new, want[:, t])
        h2, same = rl.rlcs_gated_step(cx[:, t], cg[:, t], state, reset=cr[:, t], new_state=state)
        assert same is state and torch.equal(state, new) and torch.equal(h, h2)


# ---------------------------------------------------------------------------
# Head norm and rotary positions
# ---------------------------------------------------------------------------
def tables(max_pos, R):
    inv = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / max(R, 1))
    ang = torch.arange(max_pos, dtype=torch.float64)[:, None] * inv
    return ang.cos().float(), ang.sin().float()


NORM_SHAPES = [(1, 1, 1, 8, 8), (1, 4, 2, 64, 64), (5, 3, 1, 128, 64), (33, 6, 3, 80, 20),
               (64, 16, 4, 128, 128), (100, 2, 2, 32, 8), (17, 5, 5, 96, 24), (9, 2, 1, 7, 2),
               (13, 3, 1, 130, 34), (300, 8, 1, 256, 128), (1000, 4, 4, 64, 0), (4, 1, 1, 1000, 10)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,Hq,Hk,D,R", NORM_SHAPES)
def test_qk_norm_rope_and_gradient(rl, n, Hq, Hk, D, R, interleaved, dtype):
    g, dt = gen(n + 3 * D + R), DT[dtype]
    cos, sin = tables(700, R)
    pos = torch.randint(0, 700, (n,), generator=g, dtype=torch.int32)
    fused = rand(g, n, (Hq + Hk) * D, dtype=dt).cuda()  # strided views of one projection
    q, k = fused[:, :Hq * D].view(n, Hq, D), fused[:, Hq * D:].view(n, Hk, D)
    qw, kw = rand(g, D, scale=0.2, shift=1.0), rand(g, D, scale=0.2, shift=1.0)
    dq, dk = rand(g, n, Hq, D, dtype=dt), rand(g, n, Hk, D, dtype=dt)
    args = (q, k, qw.cuda(), kw.cuda(), cos.cuda(), sin.cuda(), pos.cuda())
    eps = 1e-5
    qo, ko = rl.rlcs_qk_norm_rope(*args, eps=eps, interleaved=interleaved)
    got = rl.rlcs_qk_norm_rope_backward(dq.cuda(), dk.cuda(), *args, eps=eps,
                                        interleaved=interleaved)
    for name, x, w, d, o, dx, dw in (("q", q, qw, dq, qo, got[0], got[2]),
                                     ("k", k, kw, dk, ko, got[1], got[3])):
        x = x.cpu()
        close(name, o, ref.norm_rope(x, w, cos, sin, pos, eps, interleaved))
        wx, ww = ref.norm_rope_backward(d, x, w, cos, sin, pos, eps, interleaved)
        close("d" + name, dx, wx)
        close("dw" + name, dw, ww)


def test_qk_norm_rope_gradient_against_differences(rl):
    g = gen(3)
    n, Hq, Hk, D, R = 20, 3, 1, 48, 32
    cos, sin = tables(50, R)
    pos = torch.randint(0, 50, (n,), generator=g, dtype=torch.int32)
    q, k = rand(g, n, Hq, D), rand(g, n, Hk, D)
    qw, kw = rand(g, D, shift=1.0), rand(g, D, shift=1.0)
    dq, dk = rand(g, n, Hq, D), rand(g, n, Hk, D)
    dirs = [rand(g, *t.shape) for t in (q, k, qw, kw)]
    tail = cuda(cos, sin, pos)
    grads = rl.rlcs_qk_norm_rope_backward(*cuda(dq, dk, q, k, qw, kw), *tail)
    grad = sum(float((a.cpu().double() * u).sum()) for a, u in zip(grads, dirs))
    eps, side = 2.0 ** -7, []
    for e in (eps, -eps):
        moved = [(t + e * u).cuda() for t, u in zip((q, k, qw, kw), dirs)]
        qo, ko = rl.rlcs_qk_norm_rope(*moved, *tail)
        side.append(float((qo.cpu().double() * dq).sum() + (ko.cpu().double() * dk).sum()))
    size = math.sqrt(n * (Hq + Hk) * D)
    assert abs((side[0] - side[1]) / (2 * eps) - grad) < 40 * eps * eps * size + 1e-4 * size


def test_qk_norm_rope_positions_outside_the_table(rl):
    g = gen(2)
    n, D, R = 6, 64, 32
    cos, sin = cuda(*tables(10, R))
    q, k, w = rand(g, n, 2, D).cuda(), rand(g, n, 1, D).cuda(), torch.ones(D).cuda()
    pos = torch.tensor([0, 9, 10, -1, 2 ** 31 - 1, 3], dtype=torch.int32).cuda()
    qo, ko = rl.rlcs_qk_norm_rope(q, k, w, w, cos, sin, pos)
    for o in (qo, ko):
        bad = torch.isnan(o[..., :R]).all(-1).all(-1).cpu()
        assert bad.tolist() == [False, False, True, True, True, False]
        assert not torch.isnan(o[..., R:]).any() and not torch.isnan(o[[0, 1, 5]]).any()


def test_qk_norm_rope_zero_heads_and_tokens(rl):
    D = 64
    cos, sin = cuda(*tables(4, D))
    w = torch.ones(D).cuda()
    q = torch.zeros(0, 3, D).cuda()
    pos = torch.zeros(0, dtype=torch.int32).cuda()
    qo, ko = rl.rlcs_qk_norm_rope(q, q[:, :1], w, w, cos, sin, pos)
    assert qo.shape == (0, 3, D) and ko.shape == (0, 1, D)
    dq, dk, dqw, dkw = rl.rlcs_qk_norm_rope_backward(q, q[:, :1], q, q[:, :1], w, w, cos, sin, pos)
    assert float(dqw.abs().sum()) == 0.0 and float(dkw.abs().sum()) == 0.0
    # a head of zeros: eps alone under the root
    z = torch.zeros(1, 1, D).cuda()
    qo, _ = rl.rlcs_qk_norm_rope(z, z, w, w, cos, sin, torch.zeros(1, dtype=torch.int32).cuda())
    assert float(qo.abs().sum()) == 0.0


@pytest.mark.parametrize("scaling,kw", [("plain", {}), ("linear", dict(factor=4.0)),
                                        ("base", dict(factor=4.0)),
                                        ("parts", dict(factor=8.0, trained_len=2048.0, scale=1.2))])
def test_rope_table(rl, scaling, kw):
    n, R, base = 40000, 64, 10000.0
    cos, sin = rl.rlcs_rope_table(n, R, base, scaling=scaling, **kw)
    i = torch.arange(R // 2, dtype=torch.float64)
    factor = kw.get("factor", 1.0)
    f = base ** (-2 * i / R)
    if scaling == "linear":
        f = f / factor
    if scaling == "base":
        f = (base * factor ** (R / (R - 2))) ** (-2 * i / R)
    if scaling == "parts":
        keep = ((2048.0 * f / (2 * math.pi) - 1.0) / 31.0).clamp(0.0, 1.0)
        f = f * keep + f / factor * (1 - keep)
    ang = torch.arange(n, dtype=torch.float64)[:, None] * f
    scale = kw.get("scale", 1.0)
    # the angle in double, up to 4e4 rad off by 1e-11, then one rounding to float32
    assert float((cos.cpu().double() - scale * ang.cos()).abs().max()) < 1.3e-7
    assert float((sin.cpu().double() - scale * ang.sin()).abs().max()) < 1.3e-7


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------
def bounds(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32)


LENS = [[1], [2, 0, 1], [63, 65], [127], [128], [129, 1], [5, 200, 0, 0, 333, 1], [257, 64, 256],
        [700]]
HEADS = [(1, 1, 64), (4, 2, 128), (6, 2, 64), (8, 1, 128), (3, 3, 8), (4, 1, 80)]


@pytest.mark.parametrize("lens", LENS, ids=lambda v: "-".join(map(str, v)))
@pytest.mark.parametrize("Hq,Hk,D", HEADS)
def test_attention_and_gradient(rl, lens, Hq, Hk, D):
    n = sum(lens)
    g = gen(n * 13 + Hq + D)
    bf = torch.bfloat16
    fused = rand(g, n, (Hq + 2 * Hk) * D, dtype=bf).cuda()
    q = fused[:, :Hq * D].view(n, Hq, D)
    k = fused[:, Hq * D:(Hq + Hk) * D].view(n, Hk, D)
    v = fused[:, (Hq + Hk) * D:].view(n, Hk, D)
    dout = rand(g, n, Hq, D, dtype=bf)
    cu, scale = bounds(lens).cuda(), 1.3 * D ** -0.5
    out, lse = rl.rlcs_attention(q, k, v, cu, scale=scale, return_lse=True)
    assert torch.equal(out, rl.rlcs_attention(q, k, v, cu, scale=scale))
    qc, kc, vc = q.cpu(), k.cpu(), v.cpu()
    want, wlse, slack = ref.attention(qc, kc, vc, lens, scale)
    close("out", out, want, slack)
    close("lse", lse, wlse)
    got = rl.rlcs_attention_backward(dout.cuda(), q, k, v, out, lse, cu, scale=scale)
    again = rl.rlcs_attention_backward(dout.cuda(), q, k, v, out, lse, cu, scale=scale)
    grads, slacks = ref.attention_backward(dout, qc, kc, vc, lens, scale)
    for name, a, b, w, s in zip(("dq", "dk", "dv"), got, again, grads, slacks):
        assert torch.equal(a, b), name  # the same bits every time
        close(name, a, w, s)
    rl.check_scratch()


def test_attention_gradient_against_differences(rl):
    # the kernel's gradient against a difference quotient of the definition in
    # 64 bits; the gradient's own bound, summed as independent errors
    g = gen(17)
    lens, Hq, Hk, D = [70, 140], 4, 2, 64
    n, scale, bf = sum(lens), D ** -0.5, torch.bfloat16
    q, k, v = rand(g, n, Hq, D, dtype=bf), rand(g, n, Hk, D, dtype=bf), rand(g, n, Hk, D, dtype=bf)
    dout = rand(g, n, Hq, D, dtype=bf)
    cu = bounds(lens).cuda()
    out, lse = rl.rlcs_attention(*cuda(q, k, v), cu, return_lse=True)
    grads = rl.rlcs_attention_backward(dout.cuda(), *cuda(q, k, v), out, lse, cu)
    _, slacks = ref.attention_backward(dout, q, k, v, lens, scale)
    eps = 1e-5
    for i, (a, s) in enumerate(zip(grads, slacks)):
        u = rand(g, *a.shape).double()
        side = []
        for e in (eps, -eps):
            moved = [t.double() for t in (q, k, v)]
            moved[i] = moved[i] + e * u
            side.append(float((ref.attention(*moved, lens, scale)[0] * dout.double()).sum()))
        want = (side[0] - side[1]) / (2 * eps)
        a = a.cpu().double()
        tol = float(((s + U * a.abs()) * u).square().sum().sqrt()) * 4 + 1e-6 * abs(want)
        assert abs(float((a * u).sum()) - want) < tol, "qkv"[i]


def test_attention_sequences_do_not_touch(rl):
    # not-a-number and infinite neighbours on both sides of a sequence, at
    # every place inside a tile that its ends can fall on
    g = gen(23)
    Hq, Hk, D, bf = 4, 2, 64, torch.bfloat16
    for lens in ([3, 90, 40], [130, 61, 100], [128, 128, 128], [64, 200, 7]):
        n, lo, hi = sum(lens), lens[0], lens[0] + lens[1]
        q, k, v = (rand(g, n, h, D, dtype=bf).cuda() for h in (Hq, Hk, Hk))
        dout = rand(g, n, Hq, D, dtype=bf).cuda()
        cu = bounds(lens).cuda()
        clean = rl.rlcs_attention(q, k, v, cu, return_lse=True)
        grads = rl.rlcs_attention_backward(dout, q, k, v, *clean, cu)
        for t, bad in zip((q, k, v, dout), (math.nan, math.inf, math.nan, math.inf)):
            t[:lo], t[hi:] = bad, -bad
        out, lse = rl.rlcs_attention(q, k, v, cu, return_lse=True)
        assert torch.equal(out[lo:hi], clean[0][lo:hi])
        assert torch.equal(lse[:, lo:hi], clean[1][:, lo:hi])
        for a, b in zip(rl.rlcs_attention_backward(dout, q, k, v, out, lse, cu), grads):
            assert torch.equal(a[lo:hi], b[lo:hi])


def test_attention_large_scores(rl):
    # one key far ahead of the rest, first, last and in the middle: the running
    # maximum moves by hundreds and every row's weight stays on that key
    Hq, D, n = 2, 64, 300
    for hot in (0, 150, 299):
        q = torch.full((n, Hq, D), 4.0, dtype=torch.bfloat16)
        k = torch.full((n, 1, D), -4.0, dtype=torch.bfloat16)
        k[hot] = 4.0
        v = rand(gen(1), n, 1, D, dtype=torch.bfloat16)
        lens = [n]
        out, lse = rl.rlcs_attention(*cuda(q, k, v), bounds(lens).cuda(), return_lse=True)
        want, wlse, slack = ref.attention(q, k, v, lens, D ** -0.5)
        close("out", out, want, slack)
        close("lse", lse, wlse)


def test_attention_tokens_outside_every_sequence(rl):
    # bounds that end early leave the rest unwritten; clamped ones stay in the arrays
    g = gen(4)
    n, D = 200, 64
    q, k, v = (rand(g, n, 2, D, dtype=torch.bfloat16).cuda() for _ in range(3))
    want = rl.rlcs_attention(q[:150].contiguous(), k[:150].contiguous(), v[:150].contiguous(),
                             bounds([150]).cuda())
    out = rl.rlcs_attention(q, k, v, torch.tensor([0, 150], dtype=torch.int32).cuda())
    assert torch.equal(out[:150], want)
    far = rl.rlcs_attention(q, k, v, torch.tensor([-5, 10 ** 9], dtype=torch.int32).cuda())
    full = rl.rlcs_attention(q, k, v, bounds([n]).cuda())
    assert torch.equal(far, full)


def test_attention_without_tokens(rl):
    q = torch.zeros(0, 4, 64, dtype=torch.bfloat16).cuda()
    k = q[:, :2]
    for cu in (bounds([0, 0]).cuda(), bounds([]).cuda()):
        out, lse = rl.rlcs_attention(q, k, k, cu, return_lse=True)
        assert out.shape == q.shape and lse.shape == (4, 0)
        dq, dk, dv = rl.rlcs_attention_backward(q, q, k, k, out, lse, cu)
        assert dq.shape == q.shape and dk.shape == dv.shape == k.shape


STEP_SHAPES = [(1, 1, 1, 1, 64), (3, 17, 4, 2, 64), (2, 300, 16, 4, 128), (5, 64, 8, 1, 128),
               (1, 5000, 6, 3, 64), (7, 129, 3, 3, 8), (2, 1000, 40, 2, 80), (130, 33, 4, 4, 128)]


@pytest.mark.parametrize("B,S,Hq,Hk,D", STEP_SHAPES)
def test_attention_step(rl, B, S, Hq, Hk, D):
    g = gen(B + S + Hq)
    bf = torch.bfloat16
    q, kc, vc = rand(g, B, Hq, D, dtype=bf), rand(g, B, S, Hk, D, dtype=bf), \
        rand(g, B, S, Hk, D, dtype=bf)
    lengths = torch.randint(0, S + 1, (B,), generator=g, dtype=torch.int32)
    lengths[0], lengths[-1] = S, min(S, 1) if B > 1 else S
    if B > 2:
        lengths[1] = 0
    want, slack = ref.attention_step(q, kc, vc, lengths, D ** -0.5)
    for b in range(B):  # what the unused entries hold does not matter
        kc[b, int(lengths[b]):], vc[b, int(lengths[b]):] = math.inf, math.nan
    args = cuda(q, kc, vc, lengths)
    out = rl.rlcs_attention_step(*args)
    close("out", out, want, slack)
    assert torch.equal(out, rl.rlcs_attention_step(*args))
    # heads before positions in memory, and lengths past the cache
    alt = [t.cuda().transpose(1, 2).contiguous().transpose(1, 2) for t in (kc, vc)]
    assert torch.equal(out, rl.rlcs_attention_step(args[0], *alt, args[3]))
    over = torch.where(args[3] == S, args[3] + 1000, args[3])
    assert torch.equal(out, rl.rlcs_attention_step(*args[:3], over))


def test_attention_step_continues_attention(rl):
    # the last row of a causal pass is one step over the cache before it
    g = gen(8)
    n, Hq, Hk, D = 321, 8, 2, 128
    q, k, v = (rand(g, n, h, D, dtype=torch.bfloat16) for h in (Hq, Hk, Hk))
    want, _, slack = ref.attention(q, k, v, [n], D ** -0.5)
    out = rl.rlcs_attention_step(q[-1:].cuda(), k[None].cuda(), v[None].cuda(),
                                 torch.tensor([n], dtype=torch.int32).cuda())
    close("out", out, want[-1:], slack[-1:])


def test_attention_step_offsets_past_32_bits(rl):
    # a cache of 2^31 + elements whose last sequence lies past the 32-bit range
    B, S, Hk, D = 3, 900000, 8, 128
    need = B * S * Hk * D * 2 * 2
    if torch.cuda.mem_get_info()[0] < need * 1.2:
        pytest.skip("needs %.0f GB" % (need / 1e9))
    g = gen(9)
    kc = torch.zeros(B, S, Hk, D, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    n = 777
    k, v = rand(g, n, Hk, D, dtype=torch.bfloat16), rand(g, n, Hk, D, dtype=torch.bfloat16)
    kc[2, :n], vc[2, :n] = k.cuda(), v.cuda()
    q = rand(g, B, Hk, D, dtype=torch.bfloat16)
    lengths = torch.tensor([0, 0, n], dtype=torch.int32)
    out = rl.rlcs_attention_step(q.cuda(), kc, vc, lengths.cuda())
    want, slack = ref.attention_step(q[2:], k[None], v[None], [n], D ** -0.5)
    close("out", out[2:], want, slack)
    assert float(out[:2].abs().sum()) == 0.0


# ---------------------------------------------------------------------------
# Streams and graphs
# ---------------------------------------------------------------------------
def test_calls_on_another_stream_and_in_a_graph(rl):
    g = gen(31)
    bf = torch.bfloat16
    x, gate = rand(g, 2, 600, 96, dtype=bf).cuda(), rand(g, 2, 600, 96, dtype=bf).cuda()
    q, k = rand(g, 300, 4, 64, dtype=bf).cuda(), rand(g, 300, 2, 64, dtype=bf).cuda()
    cu, w = bounds([100, 200]).cuda(), torch.ones(64).cuda()
    cos, sin = rl.rlcs_rope_table(300, 64)
    pos = torch.arange(300, dtype=torch.int32).cuda()

    def everything(stream=None):
        h, last = rl.rlcs_gated_scan(x, gate, stream=stream)
        dx = rl.rlcs_gated_scan_backward(x, x, gate, h, stream=stream)
        qr, kr = rl.rlcs_qk_norm_rope(q, k, w, w, cos, sin, pos, stream=stream)
        dn = rl.rlcs_qk_norm_rope_backward(qr, kr, q, k, w, w, cos, sin, pos, stream=stream)
        out, lse = rl.rlcs_attention(qr, kr, k, cu, return_lse=True, stream=stream)
        da = rl.rlcs_attention_backward(q, qr, kr, k, out, lse, cu, stream=stream)
        st = rl.rlcs_attention_step(qr[:1], kr[None], k[None], pos[200:201], stream=stream)
        return [h, last, *dx, qr, kr, *dn, out, lse, *da, st]

    want = everything()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = everything(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with torch.cuda.stream(side):
        everything()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            kept = everything()
    x.copy_(x.flip(1))
    q.copy_(q.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(kept, everything()))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("at", [0, 1, 63, 64, 100, 127, 128, 250, 299])
def test_attention_later_tokens_stay_masked(rl, D, at):
    # keys and values of a later token, whatever they hold, change no bit of
    # an earlier row; one infinite element reaches its own column alone, in
    # the rows that see it
    g = gen(31 + at)
    n, Hq, Hk, bf = 300, 4, 2, torch.bfloat16
    q, k, v = (rand(g, n, h, D, dtype=bf).cuda() for h in (Hq, Hk, Hk))
    cu = bounds([n]).cuda()
    out, lse = rl.rlcs_attention(q, k, v, cu, return_lse=True)
    for bad in (math.nan, math.inf):
        k2, v2 = k.clone(), v.clone()
        k2[at:], v2[at:] = bad, -bad
        got, glse = rl.rlcs_attention(q, k2, v2, cu, return_lse=True)
        assert torch.equal(got[:at], out[:at]) and torch.equal(glse[:, :at], lse[:, :at])
        assert torch.isnan(got[at:]).all()
    v2 = v.clone()
    v2[at, 0, 3], v2[at, 1, D - 1] = math.inf, -math.inf
    want = out.clone()
    want[at:, :2, 3], want[at:, 2:, D - 1] = math.inf, -math.inf
    assert torch.equal(rl.rlcs_attention(q, k, v2, cu), want)
    v2[n - 1, 0, 3] = -math.inf
    got = rl.rlcs_attention(q, k, v2, cu)
    assert torch.equal(got[:n - 1], want[:n - 1])
    assert torch.isnan(got[n - 1, :2, 3]).all() or at == n - 1


@pytest.mark.parametrize("count,longest,D", [(128, 3, 64), (129, 200, 64), (700, 5, 128),
                                             (1500, 2, 64)])
def test_attention_many_sequences(rl, count, longest, D):
    # more sequences than a warp, and than a block, has lanes; many are empty
    g = gen(count)
    lens = [int(x) for x in torch.randint(0, longest + 1, (count,), generator=g)]
    n, Hq, Hk, bf = sum(lens), 2, 1, torch.bfloat16
    q, k, v, dout = (rand(g, n, h, D, dtype=bf) for h in (Hq, Hk, Hk, Hq))
    cu, scale = bounds(lens).cuda(), D ** -0.5
    out, lse = rl.rlcs_attention(*cuda(q, k, v), cu, return_lse=True)
    want, wlse, slack = ref.attention(q, k, v, lens, scale)
    close("out", out, want, slack)
    close("lse", lse, wlse)
    got = rl.rlcs_attention_backward(dout.cuda(), *cuda(q, k, v), out, lse, cu)
    grads, slacks = ref.attention_backward(dout, q, k, v, lens, scale)
    for name, a, b, s in zip(("dq", "dk", "dv"), got, grads, slacks):
        close(name, a, b, s)


@pytest.mark.parametrize("B,S,Hq,Hk,D", [(1, 20000, 16, 1, 128), (3, 9000, 24, 1, 72),
                                         (300, 260, 4, 2, 64), (40, 700, 8, 8, 128),
                                         (600, 3, 2, 1, 64)])
def test_attention_step_runs(rl, B, S, Hq, Hk, D):
    # heads cut into a few runs and into many, several heads to a run, and
    # more sequences than threads, some without entries
    g = gen(B + S)
    bf = torch.bfloat16
    q, kc, vc = (rand(g, *shape, dtype=bf) for shape in ((B, Hq, D), (B, S, Hk, D), (B, S, Hk, D)))
    lengths = torch.randint(0, S + 1, (B,), generator=g, dtype=torch.int32)
    lengths[0] = S
    lengths[B // 2 + 1:B // 2 + 4] = 0
    want, slack = ref.attention_step(q, kc, vc, lengths, D ** -0.5)
    out = rl.rlcs_attention_step(*cuda(q, kc, vc, lengths))
    close("out", out, want, slack)
    assert torch.equal(out, rl.rlcs_attention_step(*cuda(q, kc, vc, lengths)))


def test_attention_step_large_scores(rl):
    # one entry far ahead of the rest, anywhere in the cache: the running
    # maximum moves by hundreds within a run and between runs
    B, S, Hq, D = 1, 3000, 4, 64
    for hot in (0, 17, 1500, 2999):
        q = torch.full((B, Hq, D), 4.0, dtype=torch.bfloat16)
        kc = torch.full((B, S, 1, D), -4.0, dtype=torch.bfloat16)
        kc[:, hot] = 4.0
        vc = rand(gen(hot), B, S, 1, D, dtype=torch.bfloat16)
        lengths = torch.tensor([S], dtype=torch.int32)
        want, slack = ref.attention_step(q, kc, vc, lengths, D ** -0.5)
        close("out", rl.rlcs_attention_step(*cuda(q, kc, vc, lengths)), want, slack)


@pytest.mark.parametrize("longest,D", [(2, 64), (3, 128), (17, 64), (60, 128), (64, 64), (128, 128)])
def test_attention_gradient_of_short_rows(rl, longest, D):
    # rows with all their keys in one tile take delta from P and dP, not from
    # the rounded output, and dS as two bfloat16 terms: dq and dk carry the
    # rounding of the result alone (2^-9 of each element at most) and that of
    # float32 sums
    g = gen(longest + D)
    lens = [int(x) for x in torch.randint(1, longest + 1, (40,), generator=g)] + [longest]
    n, Hq, Hk, bf = sum(lens), 6, 3, torch.bfloat16
    q, k, v, dout = (rand(g, n, h, D, dtype=bf) for h in (Hq, Hk, Hk, Hq))
    cu, scale = bounds(lens).cuda(), D ** -0.5
    out, lse = rl.rlcs_attention(*cuda(q, k, v), cu, return_lse=True)
    dq, dk, _ = rl.rlcs_attention_backward(dout.cuda(), *cuda(q, k, v), out, lse, cu)
    (wq, wk, _), _ = ref.attention_backward(dout, q, k, v, lens, scale)
    for name, a, w in (("dq", dq, wq), ("dk", dk, wk)):
        off = float((a.cpu().double() - w).norm() / w.norm())
        assert off < 2.0 ** -9 + 1e-4, (name, off)


# channel groups (of 64) by steps that take clusters of each size: 16, 10, 9,
# 6, 4, 3 and 2 blocks where the device has the room that was measured
@pytest.mark.parametrize("B,T,D", [(1, 4200, 384), (1, 2700, 832), (1, 2500, 960), (2, 1700, 704),
                                   (5, 1100, 448), (10, 900, 256), (37, 600, 100)])
def test_gated_scan_over_clusters(rl, B, T, D):
    for dtype in ("bf16", "f32"):
        test_gated_scan_and_gradient(rl, B, T, D, dtype, True)
