"""Float32 states of linear attention over long sequences, against 64 bits.

A first state's gradient is a times the last state of the same sums walked the other
way: that of (q, dout) in the place of (k, v), the first token last. So it may be off
by no more than that last state, but for chance: two thirds more.

And the last state: a decayed key is held in two bfloat16 parts, off by at most 2^-17
of it (half a step of each: 2^-9 of 2^-8). The sum is cut off to float32 each time a
part of 16 tokens is added, by 2^-24 of it on the average, and was a^(16 i) of its
size i additions before the end: 2 / (1 - a^16) cuts in all.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,D", [(131072, 128), (131072, 64), (1000, 128)])
def test_states_of_long_sequences(n, D):
    import linear_recurrence_scan_affine_gb300 as rl
    g = torch.Generator(device="cuda").manual_seed(n + D)
    decays = [-0.001, -0.003, -0.01, -0.1]
    H = len(decays)
    x, y = (torch.randn(n, H, D, device="cuda", generator=g).bfloat16() for _ in range(2))
    ld = torch.tensor(decays, device="cuda")
    cu = torch.tensor([0, n], device="cuda", dtype=torch.int32)
    _, last = rl.rlcs_linear_attention(x, x, y, ld, cu, return_state=True)
    zero = torch.zeros(1, H, D, D, device="cuda")
    rx, ry = x.flip(0).contiguous(), y.flip(0).contiguous()
    first = rl.rlcs_linear_attention_backward(ry, rx, rx, ry, ld, cu, state=zero, scale=1.0)[3]
    rl.check_scratch()
    steps = (n - 1 - torch.arange(n, device="cuda")).double()
    for h in range(H):
        a = float(ld[h].double().exp())
        want = (x[:, h].double() * (a ** steps)[:, None]).T @ y[:, h].double()
        off = float((last[0, h].double() - want).norm() / want.norm())
        back = float((first[0, h].double() - a * want).norm() / (a * want.norm()))
        assert off <= 2.0 ** -17 + 2.0 ** -23 / (1.0 - a ** 16), (h, off)
        assert back <= off / 0.6, (h, back, off)
