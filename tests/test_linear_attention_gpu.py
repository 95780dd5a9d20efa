"""Linear attention against its definition in 64 bits (tests/linear_reference.py,
where the bounds on bfloat16 results are derived).

A bfloat16 result adds one rounding, U of its size. A float32 state may be off
by F of the larger of its size and the array's root mean square, a few hundred
roundings of 2^-24, besides its keys' two-part rounding.
"""
import math

import pytest
import torch

from tests import linear_reference as ref

pytestmark = pytest.mark.gpu

F, U = 2e-5, ref.U


@pytest.fixture(scope="module")
def rl():
    assert torch.cuda.is_available(), "the -m gpu tests need a CUDA device"
    import linear_recurrence_scan_affine_gb300 as m
    return m


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rand(g, *shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def close(name, got, want, slack=0.0):
    want = want.detach().double()
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


def bounds(lens, first=0):
    at = [first]
    for n in lens:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32)


def case(seed, lens, Hq, Hk, D, states, decays=None):
    g = gen(seed)
    n = sum(lens)
    q, k, v, do = (rand(g, n, h, D) for h in (Hq, Hk, Hk, Hq))
    ld = -0.36 * (1.0 / 360.0) ** torch.rand(Hk, generator=g) if decays is None \
        else torch.tensor(decays)
    S = rand(g, len(lens), Hk, D, D, scale=2.0, dtype=torch.float32) if states else None
    dl = rand(g, len(lens), Hk, D, D, dtype=torch.float32) if states else None
    return q, k, v, ld.float(), S, do, dl


def check_all(rl, lens, args, scale=None):
    q, k, v, ld, S, do, dl = args
    cq, ck, cv, cl, cS, cdo, cdl, cu = cuda(q, k, v, ld, S, do, dl, bounds(lens))
    out, last = rl.rlcs_linear_attention(cq, ck, cv, cl, cu, state=cS, scale=scale,
                                         return_state=True)
    alone = rl.rlcs_linear_attention(cq, ck, cv, cl, cu, state=cS, scale=scale)
    leaves = [t.double().requires_grad_() for t in (q, k, v)]
    first = None if S is None else S.double().requires_grad_()
    want, wlast = ref.linear(*leaves, ld, lens, first, scale)
    sl = ref.slack(q, k, v, ld, lens, S, scale)
    close("out", out, want, sl)
    close("out without a state", alone, want, sl)
    close("last", last, wlast, ref.state_slack(k[:, :, None], v[:, :, None], ld, lens))
    grads = rl.rlcs_linear_attention_backward(cdo, cq, ck, cv, cl, cu, state=cS, dlast=cdl,
                                              scale=scale)
    loss = (want * do.double()).sum()
    if dl is not None:
        loss = loss + (wlast * dl.double()).sum()
    wants = torch.autograd.grad(loss, leaves + ([] if S is None else [first]))
    slacks = ref.backward_slack(do, q, k, v, ld, lens, S, dl, scale)
    for name, got, w, s in zip(("dq", "dk", "dv"), grads, wants, slacks):
        close(name, got, w, s)
    if S is None:
        assert grads[3] is None
    else:
        G = q.shape[1] // k.shape[1]
        n, _, D = q.shape
        y = (q.double() * (D ** -0.5 if scale is None else scale)).view(n, -1, G, D).flip(0)
        z = do.double().view(n, -1, G, D).flip(0)
        back = ref.state_slack(y, z, ld, lens[::-1], extra=1).flip(0)
        close("dstate", grads[3], wants[3], back)
    return out, last, grads


LENS = [[1], [2], [0, 1, 0], [63], [64], [65], [127, 1], [128], [129], [128, 128], [0, 5, 0, 130, 1],
        [256], [257], [300, 41], [7] * 9]


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("Hq,Hk,D", [(2, 2, 64), (3, 1, 128)])
@pytest.mark.parametrize("states", [False, True])
def test_lengths(rl, lens, Hq, Hk, D, states):
    check_all(rl, lens, case(sum(lens) * 131 + D, lens, Hq, Hk, D, states))


@pytest.mark.parametrize("Hq,Hk,D", [(1, 1, 8), (2, 1, 16), (4, 2, 40), (6, 3, 72), (5, 1, 96),
                                     (4, 4, 120), (8, 2, 32)])
def test_heads(rl, Hq, Hk, D):
    lens = [140, 3, 200]
    check_all(rl, lens, case(Hq + D, lens, Hq, Hk, D, True))


@pytest.mark.parametrize("lens,D", [([1500], 64), ([1100, 90, 1300], 128), ([2600], 16)], ids=str)
def test_long(rl, lens, D):
    check_all(rl, lens, case(D, lens, 1, 1, D, True))


@pytest.mark.parametrize("D", [64, 128])
def test_decays(rl, D):
    # nothing kept, almost nothing, fast, slow, all kept, and a little growth
    decays = [-math.inf, -100.0, -2.0, -1e-3, 0.0, 1e-3]
    lens = [150, 1, 260]
    check_all(rl, lens, case(3, lens, 6, 6, D, True, decays))


def test_scale(rl):
    lens = [150, 20]
    for scale in (1.0, 0.01, 3.0):
        check_all(rl, lens, case(5, lens, 4, 2, 64, True), scale)


def test_tokens_of_no_sequence(rl):
    g = gen(2)
    n, lens, first = 300, [70, 0, 130], 20
    q, k, v, do = (rand(g, n, h, 64) for h in (4, 2, 2, 4))
    ld = torch.tensor([-0.1, -0.01])
    inside = slice(first, first + sum(lens))
    for t in (q, k, v, do):  # what no sequence holds may hold anything
        t[:first], t[inside.stop:] = math.nan, math.inf
    args = cuda(q, k, v, ld, bounds(lens, first))
    torch.full((1 << 22,), math.nan, device="cuda")  # memory the results may come from
    out, last = rl.rlcs_linear_attention(*args, return_state=True)
    dq, dk, dv, _ = rl.rlcs_linear_attention_backward(do.cuda(), *args)
    want, wlast = ref.linear(q[inside], k[inside], v[inside], ld, lens)
    for name, t in (("out", out), ("dq", dq), ("dk", dk), ("dv", dv)):
        assert not t[:first].any() and not t[inside.stop:].any(), name
        assert bool(torch.isfinite(t).all()), name
    close("out", out[inside], want, ref.slack(q[inside], k[inside], v[inside], ld, lens))
    close("last", last, wlast, ref.state_slack(k[inside][:, :, None], v[inside][:, :, None], ld,
                                               lens))


def test_many_units_and_tokens_of_no_sequence(rl):
    # more units of work than run at once, and most tokens in none of them
    H, D, n, first = 16, 64, 9000, 700
    g = gen(31)
    lens = torch.randint(0, 60, (40,), generator=g).tolist()
    q, k, v, do = (rand(g, n, H, D).cuda() for _ in range(4))
    ld = -torch.rand(H, generator=g).cuda()
    cu = bounds(lens, first).cuda()
    inside = slice(first, first + sum(lens))
    for t in (q, k, v, do):
        t[:first], t[inside.stop:] = math.nan, math.nan
    junk = torch.full((1 << 26,), math.nan, device="cuda")  # memory the results may come from
    del junk
    out = rl.rlcs_linear_attention(q, k, v, ld, cu)
    grads = rl.rlcs_linear_attention_backward(do, q, k, v, ld, cu)[:3]
    part = [t[inside].contiguous() for t in (do, q, k, v)]
    small = [rl.rlcs_linear_attention(*part[1:], ld, bounds(lens).cuda()),
             *rl.rlcs_linear_attention_backward(*part, ld, bounds(lens).cuda())[:3]]
    for t, w in zip((out, *grads), small):
        assert not t[:first].any() and not t[inside.stop:].any()
        assert torch.equal(t[inside], w)
    rl.check_scratch()


def test_no_tokens_and_no_sequences(rl):
    S = torch.randn(3, 2, 64, 64, device="cuda")
    e = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    ld = torch.zeros(2, device="cuda")
    out, last = rl.rlcs_linear_attention(e, e, e, ld, bounds([0, 0, 0]).cuda(), state=S,
                                         return_state=True)
    assert out.shape == e.shape and torch.equal(last, S)
    _, last = rl.rlcs_linear_attention(e, e, e, ld, bounds([0, 0, 0]).cuda(), return_state=True)
    assert not last.any()
    grads = rl.rlcs_linear_attention_backward(e, e, e, e, ld, bounds([0, 0, 0]).cuda(), state=S,
                                              dlast=S)
    assert torch.equal(grads[3], S)
    x = torch.ones(5, 2, 64, dtype=torch.bfloat16, device="cuda")
    out, last = rl.rlcs_linear_attention(x, x, x, ld, bounds([]).cuda(), return_state=True)
    assert not out.any() and last.shape == (0, 2, 64, 64)
    assert not any(t.any() for t in
                   rl.rlcs_linear_attention_backward(x, x, x, x, ld, bounds([]).cuda())[:3])


def test_many_short_sequences(rl):
    g = gen(9)
    lens = torch.randint(0, 12, (700,), generator=g).tolist()
    check_all(rl, lens, case(4, lens, 2, 1, 16, True))


def test_views(rl):
    # a fused projection's views, read in place or copied, give the same bits
    lens, Hq, Hk, D = [200, 130], 4, 2, 64
    n = sum(lens)
    fused = rand(gen(3), n, (Hq + 2 * Hk) * D + 8).cuda()
    ld, cu = torch.tensor([-0.05, -0.3]).cuda(), bounds(lens).cuda()
    do = rand(gen(4), n, Hq, D).cuda()
    for shift in (0, 3, 8):
        part = fused[:, shift:shift + (Hq + 2 * Hk) * D] if shift < 8 else fused[:, 8:]
        q, k, v = part.view(n, Hq + 2 * Hk, D).split([Hq, Hk, Hk], 1)
        a = rl.rlcs_linear_attention(q, k, v, ld, cu, return_state=True)
        b = rl.rlcs_linear_attention(q.contiguous(), k.contiguous(), v.contiguous(), ld, cu,
                                     return_state=True)
        assert all(torch.equal(x, y) for x, y in zip(a, b))
        a = rl.rlcs_linear_attention_backward(do, q, k, v, ld, cu)
        b = rl.rlcs_linear_attention_backward(do, *(t.contiguous() for t in (q, k, v)), ld, cu)
        assert all(torch.equal(x, y) for x, y in zip(a[:3], b[:3]))


def test_values_that_are_not_finite_stay_in_their_sequence_and_head(rl):
    lens, H, D = [150, 140, 160], 3, 64
    args = case(6, lens, H, H, D, True)
    q, k, v, ld, S, do, dl = args
    cu = bounds(lens).cuda()
    call = lambda: (rl.rlcs_linear_attention(*cuda(q, k, v, ld), cu, state=S.cuda(),  # noqa: E731
                                             return_state=True)
                    + rl.rlcs_linear_attention_backward(*cuda(do, q, k, v, ld), cu,
                                                        state=S.cuda(), dlast=dl.cuda()))
    clean = call()
    for t, bad in ((q, math.nan), (k, math.inf), (v, math.nan), (do, -math.inf)):
        t[150 + 70, 1, 5] = bad
    S[1, 1, 0, 0], dl[1, 1, 3, 3] = math.nan, math.inf
    for name, a, b in zip(("out", "last", "dq", "dk", "dv", "dstate"), clean, call()):
        if a.dim() == 3:
            same = torch.equal(a[:150], b[:150]) and torch.equal(a[290:], b[290:])
            same = same and torch.equal(a[:, [0, 2]], b[:, [0, 2]])
        else:
            same = torch.equal(a[[0, 2]], b[[0, 2]]) and torch.equal(a[:, [0, 2]], b[:, [0, 2]])
        assert same, name
    out = call()[0]
    assert not torch.isfinite(out[150 + 70:290, 1].float()).all()


def test_a_nan_state_passes_no_closed_head(rl):
    # a decay of zero keeps nothing, whatever the state holds
    args = case(8, [40, 200], 2, 2, 64, True, [-math.inf, -0.1])
    q, k, v, ld, S, _, _ = args
    clean = rl.rlcs_linear_attention(*cuda(q, k, v, ld), bounds([40, 200]).cuda(), state=S.cuda(),
                                     return_state=True)
    S[:, 0] = math.nan
    got = rl.rlcs_linear_attention(*cuda(q, k, v, ld), bounds([40, 200]).cuda(), state=S.cuda(),
                                   return_state=True)
    assert all(torch.equal(a, b) for a, b in zip(clean, got))


@pytest.mark.parametrize("Hq,Hk,D", [(6, 2, 64), (4, 4, 128), (12, 3, 32)])
def test_empty_sequences_between_many(rl, Hq, Hk, D):
    # blocks take up unit after unit, some without a token, of one chunk and of several
    g = gen(41)
    lens = [0 if torch.rand(1, generator=g) < 0.4 else
            int(torch.randint(1, 400, (1,), generator=g)) for _ in range(300)]
    for some in (lens, lens[:120]):  # more sequences than are put in order, and fewer
        q, k, v, ld, S, do, dl = cuda(*case(43, some, Hq, Hk, D, True))
        cu = bounds(some).cuda()
        out, last = rl.rlcs_linear_attention(q, k, v, ld, cu, state=S, return_state=True)
        grads = rl.rlcs_linear_attention_backward(do, q, k, v, ld, cu, state=S, dlast=dl)
        rl.check_scratch()
        at = cu.tolist()
        for s in range(0, len(some), 17):  # each sequence as if alone
            r = slice(at[s], at[s + 1])
            one = bounds([some[s]]).cuda()
            args = (q[r], k[r], v[r], ld, one)
            o, l = rl.rlcs_linear_attention(*args, state=S[s:s + 1], return_state=True)
            b = rl.rlcs_linear_attention_backward(do[r], *args, state=S[s:s + 1],
                                                  dlast=dl[s:s + 1])
            assert torch.equal(out[r], o) and torch.equal(last[s:s + 1], l), s
            assert all(torch.equal(x[r], y) for x, y in zip(grads[:3], b)), s
            assert torch.equal(grads[3][s:s + 1], b[3]), s


def test_gradient_against_differences(rl):
    # The loss is linear in each of q, k and v, so a central difference along a
    # direction has no truncation error in one array at a time; its rounding is
    # that of 2 n results to bfloat16, U / sqrt(3) of each, over 2 eps.
    lens, Hq, Hk, D = [130, 40], 4, 2, 64
    q, k, v, ld, S, do, dl = case(12, lens, Hq, Hk, D, True)
    cu = bounds(lens).cuda()
    grads = rl.rlcs_linear_attention_backward(*cuda(do, q, k, v, ld), cu, state=S.cuda(),
                                              dlast=dl.cuda())
    g = gen(13)
    arrays = [q, k, v, S]
    for i, name in enumerate(("dq", "dk", "dv", "dstate")):
        # directions of +-1 on arrays rounded to multiples of 1/8 within 16: exact in bfloat16
        u = torch.randint(0, 2, arrays[i].shape, generator=g) * 2.0 - 1.0
        base = [t if j != i else (t.float() * 8).round().clamp(-120, 120).div(8).to(t.dtype)
                for j, t in enumerate(arrays)]
        side, size = [], 0.0
        for e in (1.0, -1.0):
            moved = [t if j != i else (t.float() + e * u).to(t.dtype) for j, t in enumerate(base)]
            o, last = rl.rlcs_linear_attention(*cuda(*moved[:3], ld), cu, state=moved[3].cuda(),
                                               return_state=True)
            o, last = o.double().cpu(), last.double().cpu()
            side.append(float((o * do.double()).sum() + (last * dl.double()).sum()))
            size += float((o * do.double()).square().sum())
        # inner roundings: two more of U for each result, as the out's own bound has them
        sl = ref.slack(*base[:3], ld, lens, base[3]) / ref.SIX
        size += 2.0 * float((sl * do.double() / U).square().sum())
        grad = float((grads[i].double().cpu() * u.double()).sum())
        gsize = float((grads[i].double().cpu() * u).square().sum()) ** 0.5
        off = abs((side[0] - side[1]) / 2 - grad)
        # base differs from the arrays the gradient was taken at only in the array it is linear in
        assert off <= 6.0 * U * (size ** 0.5 / 2 + 2.0 * gsize), (name, off)


def test_steps_reach_the_whole(rl):
    lens, Hq, Hk, D = [150], 4, 2, 128
    q, k, v, ld, S, _, _ = case(15, lens, Hq, Hk, D, True)
    cq, ck, cv, cl, state = cuda(q, k, v, ld, S)
    whole, last = rl.rlcs_linear_attention(cq, ck, cv, cl, bounds(lens).cuda(), state=state,
                                           return_state=True)
    outs = []
    state = state.clone()
    for t in range(lens[0]):
        o, state = rl.rlcs_linear_attention_step(cq[t:t + 1], ck[t:t + 1], cv[t:t + 1], cl, state,
                                                 new_state=state)
        outs.append(o)
    want, wlast = ref.linear(q, k, v, ld, lens, S)
    sl = ref.slack(q, k, v, ld, lens, S)
    close("steps", torch.cat(outs), want)
    close("state of steps", state, wlast)
    close("whole", whole, want, sl)
    close("state of the whole", last, wlast,
          ref.state_slack(k[:, :, None], v[:, :, None], ld, lens))


@pytest.mark.parametrize("B,Hq,Hk,D", [(1, 1, 1, 8), (3, 4, 2, 64), (70, 6, 2, 40), (5, 16, 16, 128),
                                       (300, 3, 1, 128), (2, 9, 1, 96), (1, 40, 2, 128)])
def test_step(rl, B, Hq, Hk, D):
    g = gen(B + D)
    fused = rand(g, B, (Hq + 2 * Hk) * D + 3)
    q, k, v = fused[:, 3:].view(B, Hq + 2 * Hk, D).split([Hq, Hk, Hk], 1)
    ld = torch.rand(Hk, generator=g) * -0.5
    ld[0] = 0.0
    S = rand(g, B, Hk, D, D, dtype=torch.float32)
    reset = torch.rand(B, generator=g) < 0.3
    S[reset] = math.nan
    cf = fused.cuda()
    cq, ck, cv = cf[:, 3:].view(B, Hq + 2 * Hk, D).split([Hq, Hk, Hk], 1)
    cl, cS, cr = cuda(ld, S, reset)
    out, new = rl.rlcs_linear_attention_step(cq, ck, cv, cl, cS, reset=cr)
    want, wnew = ref.step(q, k, v, ld, S, reset)
    close("out", out, want)
    close("state", new, wnew)
    again, same = rl.rlcs_linear_attention_step(cq, ck, cv, cl, cS, reset=cr.to(torch.uint8),
                                                new_state=cS, scale=D ** -0.5)
    assert same.data_ptr() == cS.data_ptr()
    assert torch.equal(again, out) and torch.equal(same, new)
    empty = rl.rlcs_linear_attention_step(cq[:0], ck[:0], cv[:0], cl, cS[:0])
    assert empty[0].shape == (0, Hq, D) and empty[1].shape == (0, Hk, D, D)


def test_step_keeps_nothing_of_a_closed_head(rl):
    q, k, v = (rand(gen(i), 2, 1, 16).cuda() for i in range(3))
    S = torch.full((2, 1, 16, 16), math.inf, device="cuda")
    out, new = rl.rlcs_linear_attention_step(q, k, v, torch.tensor([-math.inf]).cuda(), S)
    want, wnew = ref.step(q.cpu(), k.cpu(), v.cpu(), torch.tensor([-math.inf]),
                          torch.zeros(2, 1, 16, 16))
    close("out", out, want)
    close("state", new, wnew)


def test_repeats_streams_and_graphs(rl):
    lens, Hq, Hk, D = [400, 0, 333], 4, 2, 128
    args = case(21, lens, Hq, Hk, D, True)
    q, k, v, ld, S, do, dl = cuda(*args)
    cu = bounds(lens).cuda()

    def call(stream=None):
        f = rl.rlcs_linear_attention(q, k, v, ld, cu, state=S, return_state=True, stream=stream)
        b = rl.rlcs_linear_attention_backward(do, q, k, v, ld, cu, state=S, dlast=dl,
                                              stream=stream)
        s = rl.rlcs_linear_attention_step(q[:3], k[:3], v[:3], ld, S, stream=stream)
        return f + b + s

    want = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = call(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, other))
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            graphs.append((graph, call()))
    fresh = [t.clone() for t in want]
    q.neg_()  # replays see new inputs
    want = call()
    for graph, _ in graphs:
        graph.replay()
    torch.cuda.synchronize()
    for _, got in graphs:
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert not torch.equal(want[0], fresh[0])
    rl.check_scratch()


@pytest.mark.parametrize("D", [64, 128])
def test_calls_one_behind_another(rl, D):
    """Last states come from a launch that runs beside the one before it: calls
    that follow each other without a pause, each on what the last has just written
    and with its inputs written over at once, give the bits of calls that wait."""
    lens = [1000, 3, 0, 517] + [40] * 30
    H = 6
    args = case(33, lens, H, H, D, True)
    cu = bounds(lens).cuda()

    def chain(pause):
        q, k, v, ld, S, do, dl = cuda(*args)
        stop = torch.cuda.synchronize if pause else (lambda: None)
        got = []
        # (keys grow by the product of states and values: 1, 10, 30, 5000, 10^8, 10^19
        # and then, at the sixth call, gradients past float32's range)
        for _ in range(4):
            stop()
            out, last = rl.rlcs_linear_attention(q, k, v, ld, cu, state=S, return_state=True)
            stop()
            grads = rl.rlcs_linear_attention_backward(out, q, k, v, ld, cu, state=S, dlast=last)
            stop()
            got += [t.clone() for t in (out, last, *grads)]
            stop()
            for t in (k, v, S):
                t.fill_(float("nan"))
            k, v, S = grads[1].mul_(0.01), out.mul_(0.1), last
        return got

    want = chain(True)
    for _ in range(3):
        for a, b in zip(want, chain(False)):
            assert bool(torch.isfinite(a).all()) and torch.equal(a, b)


def test_offsets_past_32_bits(rl):
    # 2^31 elements and more to an array: its last sequence equals a small call's
    H, D = 128, 128
    n = (1 << 31) // (H * D) + 300
    x = torch.randn(n, H, D, device="cuda", dtype=torch.bfloat16)
    ld = torch.full((H,), -0.02, device="cuda")
    lens = [n - 200, 200]
    out, last = rl.rlcs_linear_attention(x, x, x, ld, bounds(lens).cuda(), return_state=True)
    y = x[-200:].contiguous()
    o, s = rl.rlcs_linear_attention(y, y, y, ld, bounds([200]).cuda(), return_state=True)
    assert torch.equal(out[-200:], o) and torch.equal(last[1:], s)
    grads = rl.rlcs_linear_attention_backward(x, x, x, x, ld, bounds(lens).cuda())
    small = rl.rlcs_linear_attention_backward(y, y, y, y, ld, bounds([200]).cuda())
    for a, b in zip(grads[:3], small[:3]):
        assert torch.equal(a[-200:], b)


def test_refusals(rl):
    q, k = torch.zeros(6, 4, 64).bfloat16().cuda(), torch.zeros(6, 2, 64).bfloat16().cuda()
    ld, cu = torch.zeros(2).cuda(), bounds([6]).cuda()
    S = torch.zeros(1, 2, 64, 64).cuda()
    call, back, step = (rl.rlcs_linear_attention, rl.rlcs_linear_attention_backward,
                        rl.rlcs_linear_attention_step)
    for bad in (lambda: call(q.float(), k.float(), k.float(), ld, cu),
                lambda: call(q[:, :3], k, k, ld, cu),
                lambda: call(q, k[:5], k, ld, cu),
                lambda: call(q, k, k, ld[:1], cu),
                lambda: call(q, k, k, ld.double(), cu),
                lambda: call(q, k, k, ld, cu.long()),
                lambda: call(q, k, k, ld, cu[:0]),
                lambda: call(q, k, k, ld, cu, state=S[0]),
                lambda: call(q, k, k, ld, cu, state=S.double()),
                lambda: call(q, k, k, ld.cpu(), cu),
                lambda: back(k, q, k, k, ld, cu),
                lambda: back(q, q, k, k, ld, cu, dlast=S[:, :1]),
                lambda: step(q, k, k, ld, S),
                lambda: step(q[:1], k[:1], k[:1], ld, S, new_state=S[:, :, :, ::2]),
                lambda: step(q[:1], k[:1], k[:1], ld, S, reset=torch.zeros(2).bool().cuda())):
        with pytest.raises((ValueError, TypeError)):
            bad()
    wide = torch.zeros(6, 2, 136).bfloat16().cuda()
    for bad in (lambda: call(wide, wide, wide, ld, cu),
                lambda: call(q, k, k, ld, cu, scale=0.0),
                lambda: call(q, k, k, ld, cu, scale=math.nan),
                lambda: call(q[..., :12], k[..., :12], k[..., :12], ld, cu)):
        with pytest.raises(rl.RlcsError):
            bad()
