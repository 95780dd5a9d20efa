"""The binding's cached workspaces as calls outgrow them, on the CPU."""
import contextlib
import gc
import types
import weakref

import pytest
import torch

from linear_recurrence_scan_affine_gb300 import binding


@pytest.fixture
def cache(monkeypatch):
    """Workspaces of a stream 7, in host memory."""
    monkeypatch.setattr(binding, "_ws_cache", {})
    monkeypatch.setattr(binding, "_ws_outgrown", [], raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda device=None: types.SimpleNamespace(cuda_stream=7))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    return lambda need: binding.workspace_for(0, 0, torch.device("cpu"), need=need)


def test_an_outgrown_workspace_stays(cache):
    # a graph captured with it writes to it at every replay
    sizes, refs, places = (1000, 100000, 5000000), [], set()
    for need in sizes:
        ws, size = cache(need)
        assert size >= need
        refs.append(weakref.ref(ws))
        places.add(ws.data_ptr())
        del ws
    gc.collect()
    assert all(r() is not None for r in refs) and len(places) == len(sizes)


def test_what_is_kept_is_bounded(cache):
    need = 1 << 16
    for _ in range(2000):  # a little more each time
        need += 64
        size = cache(need)[1]
    kept = sum(ws.numel() for ws in binding._ws_outgrown)
    assert kept < size <= 4 * need


def test_the_same_workspace_while_it_is_large_enough(cache):
    a, size = cache(1 << 20)
    assert cache(1000)[0] is a and cache(1 << 20)[0] is a and cache(size)[0] is a
