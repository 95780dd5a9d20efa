"""Linear attention over as many tokens as a call takes, 2^31 - 128 in one sequence:
windows of the result against 64 bits (tests/linear_reference.py). A head of 8, so
that queries, keys and values (one array) and the result take 69 GB."""
import pytest
import torch

from tests import linear_reference as ref
from tests.test_linear_attention_gpu import bounds, close

pytestmark = pytest.mark.gpu


def test_most_tokens():
    import linear_recurrence_scan_affine_gb300 as rl
    n, D, piece = 2 ** 31 - 128, 8, 1 << 25
    free = torch.cuda.mem_get_info()[0]
    if free < 90e9:
        pytest.skip("takes 69 GB of device memory")
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(n, 1, D, dtype=torch.bfloat16, device="cuda")
    for i in range(0, n, piece):
        x[i:i + piece].normal_(generator=g)
    ld = torch.tensor([-0.1])
    out = rl.rlcs_linear_attention(x, x, x, ld.cuda(), bounds([n]).cuda())
    # the first, the last, and places where one of 304 shares of the tokens ends,
    # within 128 tokens for each share before it: what lies 1000 tokens back
    # counts by e^-100
    starts = [0, n - 3000] + [j * n // 304 - 1500 for j in (1, 2, 3, 8, 100, 303)]
    for at in starts:
        w = x[at:at + 3000].cpu()
        want, _ = ref.linear(w, w, w, ld, [len(w)])
        warm = 1000 if at else 0
        close("tokens from %d" % at, out[at:at + 3000][warm:], want[warm:],
              ref.slack(w, w, w, ld, [len(w)])[warm:])
    del x, out
    torch.cuda.empty_cache()
    rl.check_scratch()
