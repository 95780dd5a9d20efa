"""The smoke run computes its references on the CPU: what it launches is the
package's kernels and copies."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

import __graft_entry__ as entry

pytestmark = pytest.mark.gpu

# what making inputs and reading results takes
MOVES = {"_to_copy", "copy_", "empty", "empty_like", "empty_strided", "ones", "ones_like", "cat",
         "fill_", "clone", "_pin_memory"}
VIEWS = {"view", "slice", "select", "unsqueeze", "detach", "alias", "expand", "t", "permute",
         "_unsafe_view", "transpose", "numpy_T"}


def test_smoke_computes_nothing_else_on_the_gpu():
    assert torch.cuda.is_available(), "the -m gpu tests need a CUDA device"
    import numpy as np

    import linear_recurrence_scan_affine_gb300 as rl
    other = []

    class Watch(TorchDispatchMode):
        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            out = func(*args, **(kwargs or {}))
            name = func.overloadpacket.__name__
            if isinstance(out, torch.Tensor) and out.is_cuda and name not in MOVES | VIEWS:
                other.append(name)
            return out

    def check(name, got, want, tol=1e-4):
        got = got.cpu().double().numpy()
        assert np.all(np.abs(got - want) <= tol * np.maximum(1.0, np.abs(want))), name

    with Watch():
        entry.sequence_smoke(rl, check)
    assert len(other) <= 10, other
