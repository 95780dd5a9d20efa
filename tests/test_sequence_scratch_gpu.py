"""Sequence operators called from several threads, and in graphs that outlive
calls of other sizes."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rl():
    assert torch.cuda.is_available(), "the -m gpu tests need a CUDA device"
    import linear_recurrence_scan_affine_gb300 as m
    return m


class Work:
    """Calls with scratch at one set of sizes: attention with its gradient, the
    norm's gradient, and a new token over caches whose heads are cut."""

    def __init__(self, rl, seed, lens, B, S, Hq=8, Hk=2, D=64):
        g = torch.Generator().manual_seed(seed)
        bf = torch.bfloat16

        def normal(*shape, dtype=bf):
            return torch.randn(shape, generator=g).to(dtype).cuda()
        n = sum(lens)
        self.rl = rl
        self.q, self.k, self.v = normal(n, Hq, D), normal(n, Hk, D), normal(n, Hk, D)
        ends = [0]
        for x in lens:
            ends.append(ends[-1] + x)
        self.cu = torch.tensor(ends, dtype=torch.int32).cuda()
        self.w = normal(D, dtype=torch.float32)
        self.cos, self.sin = rl.rlcs_rope_table(n, D)
        self.pos = torch.arange(n, dtype=torch.int32).cuda()
        self.token = normal(B, Hq, D)
        self.caches = normal(2, B, S, Hk, D)
        self.lengths = torch.randint(1, S + 1, (B,), generator=g, dtype=torch.int32).cuda()

    def __call__(self):
        rl = self.rl
        out, lse = rl.rlcs_attention(self.q, self.k, self.v, self.cu, return_lse=True)
        grads = rl.rlcs_attention_backward(self.q, self.q, self.k, self.v, out, lse, self.cu)
        norms = rl.rlcs_qk_norm_rope_backward(self.q, self.k, self.q, self.k, self.w, self.w,
                                              self.cos, self.sin, self.pos)
        step = rl.rlcs_attention_step(self.token, *self.caches, self.lengths)
        return [out, lse, *grads, *norms, step]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_threads_on_one_stream(rl):
    works = [Work(rl, 1, [100, 300, 7], 3, 5000), Work(rl, 2, [900, 60], 40, 700),
             Work(rl, 3, [5], 1, 20000)]
    want = [w() for w in works]
    torch.cuda.synchronize()
    got = [[] for _ in works]
    failed = []

    def run(i):
        try:
            for _ in range(60):
                got[i].append(works[i]())
        except BaseException as e:
            failed.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(works))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    for i, results in enumerate(got):
        assert all(same(r, want[i]) for r in results)


def captured(work, stream):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        results = work()
    return graph, results


def test_graph_after_larger_calls_on_its_stream(rl):
    small, large = Work(rl, 4, [120, 80], 2, 3000), Work(rl, 5, [3000, 1000], 64, 6000)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        small()  # loads the kernels
        side.synchronize()
        graph, kept = captured(small, side)
        for _ in range(3):
            large()
        side.synchronize()
        # what the allocator can now give away
        others = [torch.full((1 << k,), 7, dtype=torch.uint8, device="cuda")
                  for k in range(9, 25) for _ in range(4)]
        want = small()
        for t in kept:
            t.zero_()
        for _ in range(3):
            graph.replay()
        side.synchronize()
        assert same(kept, want)
        assert all(bool((t == 7).all()) for t in others)
    rl.check_scratch()


def test_graphs_of_one_stream_on_two(rl):
    works = [Work(rl, 6, [700, 300], 8, 4000), Work(rl, 7, [90, 1500], 5, 9000)]
    want = [w() for w in works]
    side = torch.cuda.Stream()
    pairs = [captured(w, side) for w in works]
    streams = [torch.cuda.Stream() for _ in works]
    torch.cuda.synchronize()
    for _ in range(20):
        for (graph, _), s in zip(pairs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for (_, kept), w in zip(pairs, want):
        assert same(kept, w)
    rl.check_scratch()


def test_first_calls_of_a_stream_in_a_capture(rl):
    work = Work(rl, 8, [64, 200], 2, 900)
    want = work()  # on another stream
    torch.cuda.synchronize()
    graph, kept = captured(work, torch.cuda.Stream())
    rl.check_scratch()  # nothing has run yet
    graph.replay()
    torch.cuda.synchronize()
    assert same(kept, want)
    rl.check_scratch()
