"""The gated linear recurrence where its gates are closed: h, dx, dgate and
dh0 element by element against 64 bits.

Bounds, relative to each element's own terms. With e = exp(g), g < 0, formed
as 2^(g log2 e): the product's rounding and the constant's move the exponent
by at most 1.5 |g| 2^-24 log2 e, the instruction adds 2^-22, the reciprocal
in 1 - a 2^-23, and each product or sum 2^-24: E(g) = (2 |g| + 32) 2^-24 has
room for all of them. A bfloat16 result adds one rounding, U = 2^-8, and
below the smallest normal number, 2^-126, half a step of 2^-133; dgate reads
states that were rounded to bfloat16.
"""
import pytest
import torch

from tests import sequence_reference as ref

pytestmark = pytest.mark.gpu
U = ref.U
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def rl():
    assert torch.cuda.is_available(), "the -m gpu tests need a CUDA device"
    import linear_recurrence_scan_affine_gb300 as m
    return m


def within(name, got, want, tol):
    off = (got.double().cpu() - want).abs()
    if got.dtype == torch.bfloat16:
        tol = tol + U * want.abs() + 2.0 ** -134
    worst = (off / tol.clamp(min=1e-300)).max()
    assert bool((off <= tol).all()), "%s: %.3g times the bound" % (name, worst)


def inputs(seed, B, T, D, dt, lo, hi):
    g = torch.Generator().manual_seed(seed)
    x, dh = (torch.randn(B, T, D, generator=g).to(dt) for _ in range(2))
    gate = (torch.rand(B, T, D, generator=g) * (hi - lo) + lo).to(dt)
    # a large first state, so that what is carried shows in h
    h0 = torch.randn(B, D, generator=g) * 1e6
    return x, dh, gate, h0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lo,hi", [(-20.0, -8.0), (-80.0, -16.0), (-12.0, 0.0)])
@pytest.mark.parametrize("B,T,D", [(2, 20, 64), (1, 700, 34), (1, 700, 33), (1, 5000, 40),
                                   (800, 140, 3)])
def test_closed_gates(rl, B, T, D, lo, hi, dtype):
    # walks by warps alone, by one block and by a cluster
    x, dh, gate, h0 = inputs(B + T + D, B, T, D, DT[dtype], lo, hi)
    cx, cd, cg, c0 = (t.cuda() for t in (x, dh, gate, h0))
    h, last = rl.rlcs_gated_scan(cx, cg, h0=c0)
    dx, dg, dh0 = rl.rlcs_gated_scan_backward(cd, cx, cg, h, h0=c0)

    wh = ref.gated_scan(x, gate, None, h0)
    wx, wg, w0, slack = ref.gated_scan_backward(dh, x, gate, None, h0)
    g64, x64, d64 = gate.double(), x.double(), dh.double()
    a, om = torch.sigmoid(g64), torch.sigmoid(-g64)
    E = (2 * g64.abs() + 32) * 2.0 ** -24
    # sums of the terms' sizes, carried as the recurrence carries its values,
    # with the steps' own relative errors added up on the way
    size, err = torch.empty_like(wh), torch.empty_like(wh)
    prev, perr = h0.double().abs(), torch.zeros(B, D, dtype=torch.float64)
    first = prev
    for t in range(T):
        perr = a[:, t] * (perr + E[:, t] * prev) + E[:, t] * om[:, t] * x64[:, t].abs()
        prev = a[:, t] * prev + om[:, t] * x64[:, t].abs()
        size[:, t], err[:, t] = prev, perr
    lsize, lerr = torch.empty_like(wh), torch.empty_like(wh)
    mu, merr = (torch.zeros(B, D, dtype=torch.float64) for _ in range(2))
    for t in range(T - 1, -1, -1):
        lsize[:, t] = d64[:, t].abs() + mu
        lerr[:, t] = merr + 2.0 ** -23 * lsize[:, t]
        merr = a[:, t] * (lerr[:, t] + E[:, t] * lsize[:, t])
        mu = a[:, t] * lsize[:, t]
    before = torch.cat([first[:, None], size[:, :-1]], 1)
    berr = torch.cat([torch.zeros_like(first)[:, None], err[:, :-1]], 1)
    within("h", h, wh, err)
    within("h_last", last, wh[:, -1], err[:, -1])
    within("dx", dx, wx, om * (lerr + E * lsize))
    diff = before + x64.abs()
    tol = a * om * ((lerr + 2 * E * lsize) * diff + lsize * (berr + 2.0 ** -23 * diff))
    within("dgate", dg, wg, tol + (slack * (1 + tol) if dtype == "bf16" else 0.0))
    within("dh0", dh0, w0, merr)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_step_and_scan_agree_on_closed_gates(rl, dtype):
    B, D = 64, 96
    x, _, gate, h0 = inputs(3, B, 1, D, DT[dtype], -30.0, 0.0)
    cx, cg, c0 = (t.cuda() for t in (x, gate, h0))
    _, last = rl.rlcs_gated_scan(cx, cg, h0=c0)
    _, new = rl.rlcs_gated_step(cx[:, 0], cg[:, 0], c0)
    g = gate[:, 0].double()
    tol = 2 * (2 * g.abs() + 32) * 2.0 ** -24 * (torch.sigmoid(g) * h0.double().abs()
                                                + torch.sigmoid(-g) * x[:, 0].double().abs())
    within("state", last, new.double().cpu(), tol)
