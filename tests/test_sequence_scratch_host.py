"""Whose scratch a sequence operator's call gets, on the CPU: the library's
functions and the allocator are stand-ins that keep book."""
import threading

import pytest
import torch

from linear_recurrence_scan_affine_gb300 import binding, sequence


class Memory:
    """Hands out address ranges and knows which are in use."""

    def __init__(self):
        self.next, self.live, self.lock = 1 << 20, {}, threading.Lock()

    def alloc(self, size, stream):
        with self.lock:
            at = self.next
            self.next += size + 512
            self.live[at] = (size, stream)
            return at

    def free(self, at):
        with self.lock:
            del self.live[at]


@pytest.fixture
def memory(monkeypatch):
    """The binding on CPU tensors: stream 7 of a device called -1."""
    m = Memory()
    monkeypatch.setattr(sequence, "_alloc", m.alloc, raising=False)
    monkeypatch.setattr(sequence, "_free", m.free, raising=False)
    monkeypatch.setattr(sequence, "_need", lambda t, *a: t)
    monkeypatch.setattr(sequence, "_main", lambda t, *a: (t, -1))
    monkeypatch.setattr(sequence, "_raw_stream", lambda dev: 7)
    monkeypatch.setattr(sequence, "_attended", set(), raising=False)
    return m


def calls(size):
    """Each call that has scratch, with arguments of about this many tokens."""
    bf = torch.bfloat16
    q, k = torch.zeros(size, 4, 64, dtype=bf), torch.zeros(size, 2, 64, dtype=bf)
    cu = torch.tensor([0, size], dtype=torch.int32)
    w, table = torch.ones(64), torch.ones(8, 32)
    pos = torch.zeros(size, dtype=torch.int32)
    lse = torch.zeros(4, size)
    cache = torch.zeros(size, 16, 2, 64, dtype=bf)
    return {
        "rlcs_attention": lambda: sequence.rlcs_attention(q, k, k, cu),
        "rlcs_attention_backward":
            lambda: sequence.rlcs_attention_backward(q, q, k, k, q, lse, cu),
        "rlcs_attention_step": lambda: sequence.rlcs_attention_step(q, cache, cache, pos),
        "rlcs_qk_norm_rope_backward":
            lambda: sequence.rlcs_qk_norm_rope_backward(q, k, q, k, w, w, table, table, pos),
    }


NAMES = sorted(calls(1))


@pytest.mark.parametrize("first", NAMES)
@pytest.mark.parametrize("second", NAMES)
def test_calls_of_two_threads_have_their_own(memory, monkeypatch, first, second):
    # both inside the library at once, as the foreign call releases the
    # interpreter lock, on one stream
    meet, seen = threading.Barrier(2, timeout=20), []

    def library(*args):
        at, size, stream = args[-3:]
        meet.wait()
        with memory.lock:
            seen.append((at, size))
            assert memory.live[at] == (size, 7) and stream == 7
        meet.wait()
        return 0

    for name in {first, second}:
        monkeypatch.setitem(sequence._fn, name, library)
    failed = []

    def run(name, size):
        try:
            calls(size)[name]()
        except BaseException as e:
            failed.append(e)
            meet.abort()

    threads = [threading.Thread(target=run, args=a) for a in ((first, 5), (second, 300))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    (a, n), (b, m) = sorted(seen)
    assert a + n <= b and m > 0
    assert not memory.live  # both given back


@pytest.mark.parametrize("name", NAMES)
def test_a_larger_call_leaves_no_one_without(memory, monkeypatch, name):
    # a scratch is in use for its call alone, whatever came before
    seen = []

    def library(*args):
        at, size, _ = args[-3:]
        assert memory.live == {at: (size, 7)}
        seen.append(size)
        return 0

    monkeypatch.setitem(sequence._fn, name, library)
    for size in (3, 400, 3):
        calls(size)[name]()
    assert seen[0] == seen[2] and not memory.live


@pytest.mark.parametrize("name", NAMES)
def test_a_refused_call_gives_it_back(memory, monkeypatch, name):
    monkeypatch.setitem(sequence._fn, name, lambda *args: 1)
    with pytest.raises(binding.RlcsError):
        calls(4)[name]()
    assert not memory.live
