"""Calls captured without a workspace of the caller's: a replay finds memory that is its
graph's, whatever was called, captured or allocated since."""
from __future__ import annotations

import pytest
import torch

from linear_02_amd import inputs

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
D = 128


@pytest.fixture(scope="module")
def wl():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    from linear_02_amd import wl as mod
    return mod


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


class Work:
    """A projection of single tokens and attention of its rows over divided keys, as one
    function of x."""

    def __init__(self, wl, seed, n_seq, keys):
        g = torch.Generator().manual_seed(seed)
        self.g, self.wl, self.n_seq, self.keys = g, wl, n_seq, keys
        self.theta = wl.theta_to(inputs.theta(g, 4 * D, 4 * D, 32), DEV)
        pages = keys // 64
        self.cache = wl.new_cache(n_seq * pages, 1, 64, D, torch.arange(n_seq * pages, dtype=torch.int32, device=DEV).view(n_seq, -1))
        k, v = (torch.randn(n_seq * keys, D, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
        at = torch.arange(n_seq * keys, dtype=torch.int32, device=DEV)
        wl.wl_cache_write(self.cache, k, v, at // keys, at % keys)
        self.start, self.lens = ints(list(range(n_seq + 1))), ints([keys - 64 * s for s in range(n_seq)])
        self.x = torch.empty(n_seq, 4 * D, dtype=torch.bfloat16, device=DEV)
        self.renew()

    def renew(self):
        self.x.copy_(torch.randn(self.x.shape, generator=self.g))

    def run(self):
        y = self.wl.wl_linear(self.theta, self.x)
        return y, self.wl.wl_attention(y, self.cache, self.start, self.lens, 1, self.keys, D ** -0.5)

    def captured(self):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = self.run()
        return graph, out


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_replays_after_larger_calls_and_other_captures(wl):
    small, large = Work(wl, 1, 2, 1024), Work(wl, 2, 4, 8192)
    graph, out = small.captured()
    graph2, out2 = large.captured()
    kept = []
    for it in range(4):
        small.renew(), large.renew()
        kept.append(large.run())                                     # the shared workspace grows
        kept.append([torch.full((1 << 22,), 7.0, device=DEV) for _ in range(8)])   # whatever was freed is taken
        torch.cuda.synchronize()
        if it % 2 == 0:                                              # the later capture first
            graph2.replay(), graph.replay()
        else:
            graph.replay(), graph2.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (*out, *out2)]
        assert same(got[:2], small.run()) and same(got[2:], large.run())
        assert all((t == 7).all() for k in kept[1::2] for t in k)
    # a third graph on the same capture stream, replayed before anything else has run on it
    small.renew()
    graph3, out3 = small.captured()
    graph3.replay()
    torch.cuda.synchronize()
    assert same(out3, small.run())


def test_two_graphs_side_by_side(wl):
    work = [Work(wl, 3, 3, 4096), Work(wl, 4, 2, 4096)]
    graphs = [w.captured() for w in work]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        want = []
        for w in work:
            w.renew()
            want.append([t.clone() for t in w.run()])
        torch.cuda.synchronize()
        for _ in range(5):
            for (graph, _), s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    graph.replay()
        torch.cuda.synchronize()
        for (_, out), w in zip(graphs, want):
            assert same(out, w)


def test_a_call_captured_twice_and_launched_between(wl):
    """One OpCall in two graphs, with eager launches and growth between."""
    w, large = Work(wl, 5, 2, 2048), Work(wl, 6, 4, 8192)
    y = w.run()[0]
    call = wl.attention_call(y, w.cache, w.start, w.lens, 1, w.keys, D ** -0.5)
    want = call.launch().clone()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call.launch()
        graphs.append(g)
        with torch.cuda.stream(torch.cuda.Stream()):
            large.run()
        large.run(), call.launch()
    hold = [torch.full((1 << 22,), 7.0, device=DEV) for _ in range(8)]
    for g in graphs * 3:
        call.out.fill_(3)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(call.out, want)
    assert all((t == 7).all() for t in hold)
