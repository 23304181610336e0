"""A whole decoder layer, projections and the operations between them, as one
recorded step: prompts written and attended eagerly, then tokens decoded by
launches of one graph that follow the growing sequences.

Every launch is compared bit for bit with the same calls made one by one, and
stage by stage with the 64-bit definitions on that stage's own inputs.
"""
from __future__ import annotations

import pytest
import torch

import layer_ref as ref
from linear_02_amd import inputs
from parity import check

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
D, PAGE = 256, 32


@pytest.fixture(scope="module")
def wl():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    from linear_02_amd import wl as mod
    return mod


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


class Layer:
    """The buffers and calls of one layer for T tokens of n_seq sequences."""

    def __init__(self, wl, dims, dev, norms, cache, x, seq, slot, q_start, kv_len, max_q, max_kv):
        T, w = x.shape[0], dims["q"] + 2 * dims["kv"]
        bf = dict(dtype=torch.bfloat16, device=DEV)
        self.x, self.qkv = x, torch.empty(T, w, **bf)
        freq, _ = wl.rope_frequencies(D, device=DEV)
        self.rope = wl.Rope(freq)
        q, k, v = self.qkv.split([dims["q"], dims["kv"], dims["kv"]], 1)
        self.o, self.y = torch.empty(T, dims["d_model"], **bf), torch.empty(T, dims["d_model"], **bf)
        kw = dict(eps=1e-6, offset=1.0)
        n1 = wl.norm_call(x, pre=norms["in"], want_x=False, **kw)
        write = wl.cache_write_call(cache, k, v, seq, slot, q=q, rope=self.rope, q_norm=norms["q"], k_norm=norms["k"],
                                    q_out=q, **kw)
        att = wl.attention_call(q, cache, q_start, kv_len, max_q, max_kv, D ** -0.5)
        n2 = wl.norm_call(x, y=self.o, post=norms["post"], pre=norms["mlp"], **kw)
        n3 = wl.norm_call(n2.out[0], y=self.y, post=norms["out"], want_n=False, **kw)
        self.n1, self.write, self.att, self.n2, self.n3 = n1, write, att, n2, n3
        self.calls = [n1, (wl.OP_QKV, [dev[f] for f in "qkv"], n1.out[1], self.qkv), write, att,
                      (wl.OP_LINEAR, [dev["o"]], att.out, self.o), n2,
                      (wl.OP_MLP, [dev[f] for f in ("gate", "up", "down")], n2.out[1], self.y), n3]

    def outputs(self):
        return dict(n1=self.n1.out[1], qkv=self.qkv, att=self.att.out, o=self.o, x2=self.n2.out[0], n2=self.n2.out[1], y=self.y,
                    x3=self.n3.out[0])

    def eager(self, wl):
        self.n1.launch()
        _, th, x, y = self.calls[1]
        wl.wl_qkv_fused(*th, x, y=y)
        raw = self.qkv.clone()
        self.write.launch(), self.att.launch()
        wl.wl_linear(self.calls[4][1][0], self.att.out, y=self.o)
        self.n2.launch()
        wl.wl_mlp_fused(*self.calls[6][1], self.n2.out[1], y=self.y)
        self.n3.launch()
        return raw


@pytest.mark.parametrize("fmt", [torch.bfloat16, torch.int8, torch.float8_e4m3fn])
def test_layer_step(wl, orc, fmt):
    g = torch.Generator().manual_seed(77)
    dims = inputs.GEMMA3_1B
    host = inputs.layer(g, dims, 4)
    dev = {f: wl.theta_to(host[f], DEV) for f in inputs.FAMILIES}
    dm = dims["d_model"]
    norms = {n: (torch.randn(D if n in "qk" else dm, generator=g) * 0.2).to(torch.bfloat16).to(DEV)
             for n in ("in", "q", "k", "post", "mlp", "out")}
    prompts = [70, 33, 1]
    n_seq, table = 3, ints([[4, 1, 7, 10], [2, 0, 9, 3], [5, 6, 8, 11]])
    cache = wl.new_cache(12, 1, PAGE, D, table, fmt)
    seq = ints([s for s, n in enumerate(prompts) for _ in range(n)])
    slot = ints([j for n in prompts for j in range(n)])
    start = ints([0, 70, 103, 104])
    rows = lambda n: torch.randn(n, dm, generator=g).to(torch.bfloat16).to(DEV)  # noqa: E731
    # the prompts, eagerly
    pre = Layer(wl, dims, dev, norms, cache, rows(104), seq, slot, start, ints(prompts), 70, 70)
    raw = pre.eager(wl)
    torch.cuda.synchronize()
    stages(orc, host, dims, cache, norms, pre, raw, slot, start, ints(prompts))
    # tokens, by one graph
    slot1, len1 = ints(prompts), ints([n + 1 for n in prompts])
    lay = Layer(wl, dims, dev, norms, cache, rows(3), ints([0, 1, 2]), slot1, ints([0, 1, 2, 3]), len1, 1, PAGE * 4)
    step = wl.LayerStep(lay.calls)
    for it in range(4):
        lay.x.copy_(rows(3))
        step.launch()
        torch.cuda.synchronize()
        got = {k: v.clone() for k, v in lay.outputs().items()}
        kept = [t.clone() for t in (cache.k.view(torch.uint8), cache.v.view(torch.uint8))]
        raw = lay.eager(wl)
        torch.cuda.synchronize()
        for k, v in lay.outputs().items():
            assert torch.equal(v, got[k]), (it, k)
        assert torch.equal(kept[0], cache.k.view(torch.uint8)) and torch.equal(kept[1], cache.v.view(torch.uint8))
        stages(orc, host, dims, cache, norms, lay, raw, slot1, ints([0, 1, 2, 3]), len1)
        slot1 += 1
        len1 += 1
    step.close()


def stages(orc, host, dims, cache, norms, lay, raw, slot, start, lens):
    """Each stage of a layer against its definition on the values the layer gave it."""
    x, o = lay.x, lay.outputs()
    _, n, _, mag = ref.norm(x, None, None, None if norms is None else norms["in"], None, 1e-6, 1.0, 1.0, 1.0)
    ref.assert_near(o["n1"], n, 2 * ref.CHAIN * ref.EPS32 * mag, "n1")
    check(raw, *orc.qkv(host["q"], host["k"], host["v"], o["n1"].cpu()), "qkv")
    want, mag = ref.rotate(raw[:, :dims["q"]], D, slot, lay.rope.freq, 1.0, False, norms["q"], 1e-6, 1.0)
    ref.assert_near(o["qkv"][:, :dims["q"]], want, (ref.CHAIN + 16) * ref.EPS32 * mag, "q")
    want, slack = ref.attention(o["qkv"][:, :dims["q"]], cache, start, lens, D ** -0.5)
    ref.assert_near(o["att"], want, slack, "attention")
    check(o["o"], *orc.linear(host["o"], o["att"].cpu()), "o")
    x2, n2, mx, mn = ref.norm(x, o["o"], norms["post"], norms["mlp"], None, 1e-6, 1.0, 1.0, 1.0)
    ref.assert_near(o["x2"], x2, ref.CHAIN * ref.EPS32 * mx, "x2")
    ref.assert_near(o["n2"], n2, 2 * ref.CHAIN * ref.EPS32 * mn, "n2")
    y, bound, _ = orc.mlp(host["gate"], host["up"], host["down"], o["n2"].cpu())
    check(o["y"], y, bound, "mlp")
    x3, _, mx, _ = ref.norm(o["x2"], o["y"], norms["out"], None, None, 1e-6, 1.0, 1.0, 1.0)
    ref.assert_near(o["x3"], x3, ref.CHAIN * ref.EPS32 * mx, "x3")


def test_step_of_other_operations(wl):
    """Rotation and reading back as ops of a step, and what a step refuses."""
    g = torch.Generator().manual_seed(5)
    cache = wl.new_cache(4, 2, 16, 64, ints([[0, 2], [1, 3]]))
    k = torch.randn(6, 128, generator=g).to(torch.bfloat16).to(DEV)
    freq, _ = wl.rope_frequencies(64, device=DEV)
    pos, seq = ints([0, 5, 9, 2, 31, 7]), ints([0, 0, 0, 1, 1, 1])
    rope = wl.rope_call(k, None, pos, wl.Rope(freq), 64)
    write = wl.cache_write_call(cache, rope.out[0], k, seq, pos)
    read = wl.cache_read_call(cache, seq, pos)
    step = wl.LayerStep([rope, write, read])
    for _ in range(3):
        k.copy_(torch.randn(6, 128, generator=g).to(torch.bfloat16))
        step.launch()
        torch.cuda.synchronize()
        assert torch.equal(read.out[0], wl.wl_rope(k, None, pos, wl.Rope(freq), 64)[0]) and torch.equal(read.out[1], k)
    bad = wl.norm_call(k)
    bad.args.d = 60
    with pytest.raises(wl.WlError) as e:
        wl.LayerStep([rope, bad])
    assert "call 1" in str(e.value)


def attended(wl, g, n_seq, keys):
    """One token each of n_seq sequences over a filled cache: cache, queries, lengths
    and an attention that divides its keys."""
    cache = wl.new_cache(n_seq * keys // 64, 1, 64, D, torch.arange(n_seq * keys // 64, dtype=torch.int32, device=DEV).view(n_seq, -1))
    T = n_seq * keys
    k, v = (torch.randn(T, D, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    at = torch.arange(T, dtype=torch.int32, device=DEV)
    wl.wl_cache_write(cache, k, v, at // keys, at % keys)
    q = torch.randn(n_seq, 4 * D, generator=g).to(torch.bfloat16).to(DEV)
    lens = ints([keys - 100 * s for s in range(n_seq)])
    att = wl.attention_call(q, cache, ints(list(range(n_seq + 1))), lens, 1, keys, D ** -0.5)
    return cache, q, lens, att


def test_step_with_divided_attention_beside_projections(wl):
    """One workspace for a projection and attentions that leave partial outputs in it."""
    g = torch.Generator().manual_seed(11)
    theta = inputs.theta(g, 4 * D, 4 * D, 32)
    dev = wl.theta_to(theta, DEV)
    cache, q, lens, att = attended(wl, g, 3, 2048)
    assert wl.lib.wl_attention_workspace_bytes(att.args) > wl.SYNC_BYTES
    y = torch.empty(3, 4 * D, dtype=torch.bfloat16, device=DEV)
    again = wl.attention_call(y, cache, ints([0, 1, 2, 3]), lens, 1, 2048, D ** -0.5)
    step = wl.LayerStep([att, (wl.OP_LINEAR, [dev], att.out, y), again])
    for it in range(4):
        q.copy_(torch.randn(3, 4 * D, generator=g).to(torch.bfloat16))
        lens -= it
        step.launch()
        torch.cuda.synchronize()
        got = [t.clone() for t in (att.out, y, again.out)]
        att.launch()
        wl.wl_linear(dev, att.out, y=y)
        again.launch()
        torch.cuda.synchronize()
        for a, b, what in zip(got, (att.out, y, again.out), ("first", "projection", "second")):
            assert torch.equal(a, b), (it, what)
        want, slack = ref.attention(q, cache, ints([0, 1, 2, 3]), lens, D ** -0.5)
        ref.assert_near(att.out, want, slack, "first")
        want, slack = ref.attention(y, cache, ints([0, 1, 2, 3]), lens, D ** -0.5)
        ref.assert_near(again.out, want, slack, "second")
    step.close()


def test_two_streams_at_once(wl):
    """Attentions with divided keys, norms and cache reads on two streams, each with
    buffers of its own: the same bits as alone."""
    g = torch.Generator().manual_seed(12)
    work, alone = [], []
    for n_seq in (2, 5):
        cache, q, _, att = attended(wl, g, n_seq, 4096)
        n = wl.norm_call(q)
        slots = torch.arange(n_seq, dtype=torch.int32, device=DEV)
        work.append([n, att, wl.cache_read_call(cache, slots, slots * 700)])
    torch.cuda.synchronize()
    for calls in work:
        for c in calls:
            c.launch()
        torch.cuda.synchronize()
        alone.append([[t.clone() for t in outputs(c)] for c in calls])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for calls in work:
            for c in calls:
                for t in outputs(c):
                    t.fill_(7)
        torch.cuda.synchronize()
        for i in range(3):
            for calls, s in zip(work, streams):
                with torch.cuda.stream(s):
                    calls[i].launch()
        torch.cuda.synchronize()
        for calls, want in zip(work, alone):
            for c, w in zip(calls, want):
                for a, b in zip(outputs(c), w):
                    assert torch.equal(a, b)


def outputs(call):
    out = call.out if isinstance(call.out, (tuple, list)) else [call.out]
    return [t for t in out if t is not None]
