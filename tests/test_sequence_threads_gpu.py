"""The sequence operators as the first CUDA calls of a new thread."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rl():
    assert torch.cuda.is_available(), "the -m gpu tests need a CUDA device"
    import linear_recurrence_scan_affine_gb300 as m
    return m


def test_first_calls_of_a_thread(rl):
    g = torch.Generator().manual_seed(0)
    n, bf = 200, torch.bfloat16
    q, k, v = (torch.randn(n, h, 64, generator=g).to(bf).cuda() for h in (4, 2, 2))
    x, gate = (torch.randn(2, 300, 96, generator=g).to(bf).cuda() for _ in range(2))
    state = torch.zeros(2, 96).cuda()
    cu = torch.tensor([0, 50, n], dtype=torch.int32).cuda()
    w, length = torch.ones(64).cuda(), torch.tensor([150], dtype=torch.int32).cuda()
    cos, sin = rl.rlcs_rope_table(n, 64)
    pos = torch.arange(n, dtype=torch.int32).cuda()
    h, _ = rl.rlcs_gated_scan(x, gate)
    out, lse = rl.rlcs_attention(q, k, v, cu, return_lse=True)
    calls = [lambda: rl.rlcs_gated_scan(x, gate),
             lambda: rl.rlcs_gated_scan_backward(x, x, gate, h),
             lambda: rl.rlcs_gated_step(x[:, 0], gate[:, 0], state),
             lambda: rl.rlcs_rope_table(n, 64),
             lambda: rl.rlcs_qk_norm_rope(q, k, w, w, cos, sin, pos),
             lambda: rl.rlcs_qk_norm_rope_backward(q, k, q, k, w, w, cos, sin, pos),
             lambda: rl.rlcs_attention(q, k, v, cu, return_lse=True),
             lambda: rl.rlcs_attention_backward(q, q, k, v, out, lse, cu),
             lambda: rl.rlcs_attention_step(q[:1], k[None], v[None], length)]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    got = [None] * len(calls)

    def run(i):
        try:
            got[i] = calls[i]()
        except BaseException as e:
            got[i] = e

    for i in range(len(calls)):
        t = threading.Thread(target=run, args=(i,))
        t.start()
        t.join()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert not isinstance(a, BaseException), a
        a, b = ([t] if isinstance(t, torch.Tensor) else t for t in (a, b))
        assert all(torch.equal(s, t) for s, t in zip(a, b))
