"""The operations around a serving batch together, as a decode loop uses them: plan,
projections, latent write, attention, head, verification, and the next plan on what was
kept; eagerly, as one recorded step, on other streams, and captured by torch."""
from __future__ import annotations

import random

import pytest
import torch

from tests import serve_ref
from tests.layer_ref import f64

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
H, N, R, V, L, D, VOCAB, PAGE = 8, 128, 64, 128, 512, 256, 512, 16


@pytest.fixture(scope="module")
def wl():
    from linear_02_amd import wl as mod
    return mod


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


class Loop:
    """One layer of latent attention between an input x and logits, over n_seq streams."""

    def __init__(self, wl, n_seq, T, fmt, tree, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.wl, self.n_seq, self.T, self.tree = wl, n_seq, T, tree
        self.pages = wl.new_pages(n_seq, 12, 60, PAGE, DEV)
        self.cache = wl.new_latent_cache(60, PAGE, L, R, self.pages.table, fmt)
        dt = self.cache.dtype
        mat = lambda o, i: {"W0": (torch.randn(o, i, generator=g) * i ** -0.5).to(dt).to(DEV), "s": None, "U": None, "V": None,  # noqa: E731
                            "d_in": i, "d_out": o, "r": 0}
        self.down, self.up, self.head = mat(L + R, D), mat(H * (N + R), D), mat(VOCAB, H * V)
        self.w = (torch.randn(H, N + V, L, generator=g) * L ** -0.5).to(dt).to(DEV)
        self.x, self.u = torch.zeros(T, D, dtype=dt, device=DEV), torch.zeros(T, 2, device=DEV)
        self.past, self.n_new = torch.zeros(n_seq, dtype=torch.int32, device=DEV), torch.zeros(n_seq, dtype=torch.int32, device=DEV)
        self.token = torch.zeros(T, dtype=torch.int32, device=DEV)
        self.parent = torch.zeros(T, dtype=torch.int32, device=DEV) if tree else None
        self.mask = torch.zeros(T, 1, dtype=torch.int32, device=DEV) if tree else None
        freq, _ = wl.rope_frequencies(R, device=DEV)
        self.rope = wl.Rope(freq)
        self.buf = {k: torch.zeros(T, n, dtype=dt, device=DEV) for k, n in
                    (("c", L + R), ("q", H * (N + R)), ("o", H * V), ("logits", VOCAB))}

    def calls(self, **kw):
        wl, b = self.wl, self.buf
        plan = wl.batch_plan_call(self.pages, self.past, self.n_new, self.T, **kw)
        q_start, kv_len, seq, slot = plan.out
        write = wl.latent_write_call(self.cache, b["c"], seq, slot, q=b["q"], n_q=H, rope=self.rope, q_out=b["q"])
        attend = wl.latent_attention_call(b["q"], self.cache, self.w, q_start, kv_len, 8, 12 * PAGE, (N + R) ** -0.5,
                                          tree=self.mask, o=b["o"], **kw)
        verify = wl.verify_drafts_call(b["logits"], self.token, q_start, self.u, parent=self.parent, length=self.past, max_q=8, **kw)
        return [plan, (wl.OP_LINEAR, [self.down], self.x, b["c"]), (wl.OP_LINEAR, [self.up], self.x, b["q"]), write, attend,
                (wl.OP_LINEAR, [self.head], b["o"], b["logits"]), verify]

    def eager(self):
        calls = self.calls()
        for c in calls:
            if isinstance(c, self.wl.OpCall):
                c.launch()
            else:
                self.wl.wl_linear(c[1][0], c[2], c[3])
        return calls

    def state(self):
        return [t.clone() for t in (self.past, self.pages.table, self.pages.held, self.pages.free, self.pages.n_free, self.cache.rows)]

    def feed(self, rng, g, drop=()):
        """New inputs: rows of every stream, drafted tokens, random numbers."""
        new = [0 if s in drop else rng.randrange(1, 6) for s in range(self.n_seq)]
        for s in drop:
            self.past[s] = 0
        self.n_new.copy_(i32(new))
        self.x.copy_(torch.randn(self.T, D, generator=g))
        self.u.copy_(torch.rand(self.T, 2, generator=g))
        self.token.copy_(torch.randint(4, (self.T,), generator=g).to(torch.int32))
        if self.tree:
            parent, mask = [], []
            for n in new:
                seen = []
                for i in range(n):
                    p = rng.randrange(max(i - 2, 0), i) if i else -1
                    parent.append(p)
                    seen.append((seen[p] if i else 0) | 1 << i)
                mask += seen
            pad = [0] * (self.T - len(parent))
            self.parent.copy_(i32(parent + pad)), self.mask.copy_(i32(mask + pad)[:, None])


def outputs(calls, wl):
    return [t for c in calls if isinstance(c, wl.OpCall) for t in (c.out if isinstance(c.out, tuple) else (c.out,))]


@pytest.mark.parametrize("fmt", [BF, E4M3, F32])
@pytest.mark.parametrize("tree", [False, True])
def test_recorded_step_is_the_eager_loop(wl, fmt, tree):
    a, b = (Loop(wl, 5, 30, fmt, tree) for _ in range(2))
    calls = b.calls()
    step = wl.LayerStep(calls)
    for k in range(8):
        for loop in (a, b):
            loop.feed(random.Random(k), torch.Generator().manual_seed(k), drop=(1,) if k == 4 else ())
        done = a.eager()
        step.launch()
        torch.cuda.synchronize()
        rows = int(a.n_new.sum())
        for x, y in zip(outputs(done, wl), outputs(calls, wl)):
            n = rows if x.dim() and x.shape[0] == a.T else x.shape[0]
            assert torch.equal(x[:n], y[:n]), k
        for x, y in zip(a.state(), b.state()):
            if x.dim() < 3:
                assert torch.equal(x, y), k
    assert int(b.past.max()) >= 8
    step.close()


@pytest.mark.parametrize("fmt", [BF, F32])
def test_loop_against_definitions(wl, fmt):
    """Every operation's answer from the others' on the way, in 64 bits."""
    loop = Loop(wl, 4, 24, fmt, False, seed=3)
    past = [0] * 4
    for k in range(5):
        loop.feed(random.Random(100 + k), torch.Generator().manual_seed(100 + k))
        table, held = loop.pages.table.tolist(), loop.pages.held.tolist()
        free = loop.pages.free.tolist()[:int(loop.pages.n_free)]
        new, T = loop.n_new.tolist(), loop.T
        ref = serve_ref.plan(table, held, free, len(free), past, new, T, PAGE)
        plan, *_, verify = loop.eager()
        torch.cuda.synchronize()
        assert [t.tolist() for t in plan.out] == [list(r) for r in ref] and loop.pages.table.tolist() == table
        q_start, kv_len = plan.out[:2]
        o, slack = serve_ref.latent_attention(loop.buf["q"], loop.cache, loop.w, q_start, kv_len, (N + R) ** -0.5)
        n = ref[0][-1]
        got = f64(loop.buf["o"])[:n]
        assert ((got - o[:n]).abs() <= slack[:n] + o[:n].abs() * torch.finfo(fmt).eps / 2 * 1.01).all()
        out, n_out, path, near = serve_ref.verify(loop.buf["logits"].cpu(), loop.token.tolist(), ref[0], loop.u.tolist(), max_q=8)
        assert near > 1e-9
        assert [t.tolist()[:n] if t.shape[0] == T else t.tolist() for t in verify.out] == [out[:n], n_out, path[:n]]
        past = [p + m for p, m in zip(past, n_out)]
        assert loop.past.tolist() == past


def test_two_streams_at_once(wl):
    """Two loops on two streams, each against itself alone."""
    ref = [Loop(wl, 4, 24, BF, False, seed=s) for s in (1, 2)]
    both = [Loop(wl, 4, 24, BF, False, seed=s) for s in (1, 2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for k in range(6):
        for loops in (ref, both):
            for i, loop in enumerate(loops):
                loop.feed(random.Random(10 * k + i), torch.Generator().manual_seed(10 * k + i))
        torch.cuda.synchronize()
        want = [loop.eager() for loop in ref]
        torch.cuda.synchronize()
        got = []
        for loop, s in zip(both, streams):
            with torch.cuda.stream(s):
                got.append(loop.eager())
        torch.cuda.synchronize()
        for i in range(2):
            rows = int(ref[i].n_new.sum())
            for x, y in zip(outputs(want[i], wl), outputs(got[i], wl)):
                n = rows if x.shape[0] == 24 else x.shape[0]
                assert torch.equal(x[:n], y[:n])


def test_two_captured_graphs(wl):
    """Two captures on one stream, replayed in turn with eager calls between: each has scratch of its own."""
    a, b = Loop(wl, 4, 24, BF, False, seed=5), Loop(wl, 4, 24, BF, False, seed=6)
    ra, rb = Loop(wl, 4, 24, BF, False, seed=5), Loop(wl, 4, 24, BF, False, seed=6)
    s = torch.cuda.Stream()
    graphs = []
    for loop in (a, b):
        loop.eager()      # nothing new: no rows, but every path warm
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
            calls = loop.eager()
        torch.cuda.current_stream().wait_stream(s)
        graphs.append((g, calls))
    for k in range(5):
        for loop, ref, (g, calls), salt in ((a, ra, graphs[0], 0), (b, rb, graphs[1], 50)):
            for x in (loop, ref):
                x.feed(random.Random(k + salt), torch.Generator().manual_seed(k + salt))
            g.replay()
            done = ref.eager()
            torch.cuda.synchronize()
            rows = int(ref.n_new.sum())
            for x, y in zip(outputs(done, wl), outputs(calls, wl)):
                n = rows if x.shape[0] == 24 else x.shape[0]
                assert torch.equal(x[:n], y[:n])
            assert torch.equal(loop.past, ref.past)
