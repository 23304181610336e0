"""wl_attention against its 64-bit definition: masks, lengths, head layouts, cache
types, and what must not reach a query."""
from __future__ import annotations

import pytest
import torch

import layer_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, I8, E4 = torch.bfloat16, torch.float32, torch.int8, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def wl():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    from linear_02_amd import wl as mod
    return mod


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


class Batch:
    """Sequences with the given earlier keys and new tokens over a shuffled cache
    whose unused slots and pages hold NaN."""

    far = False   # whether max_kv is a large limit, as a recorded step has it

    def __init__(self, wl, ctx, rows, hq, hkv, d, page, fmt, seed=0, extra=0, wide=0, dtype=None):
        g = torch.Generator().manual_seed(seed)
        dtype = dtype or (F32 if fmt == F32 else BF)
        self.ctx, self.rows = ctx, rows
        lens = [c + r for c, r in zip(ctx, rows)]
        need = [max(1, -(-n // page)) for n in lens]
        ids = torch.randperm(sum(need) + 2, generator=g).tolist()
        table, at = [], 0
        for n in need:
            table.append(ids[at:at + n] + [-7] * (max(need) - n))
            at += n
        c = wl.new_cache(sum(need) + 2, hkv, page, d, ints(table), fmt)
        if fmt in (BF, F32):
            c.k.fill_(float("nan")), c.v.fill_(float("nan"))
        else:
            c.k.view(torch.uint8).fill_(0x7F), c.v.view(torch.uint8).fill_(0x7F)
            c.k_scale.fill_(float("nan")), c.v_scale.fill_(float("nan"))
        for s, n in enumerate(lens):
            if n < 1:
                continue
            x = [torch.randn(n, hkv * d, generator=g).to(dtype).to(DEV) for _ in range(2)]
            wl.wl_cache_write(c, x[0], x[1], ints([s] * n), torch.arange(n, dtype=torch.int32, device=DEV))
        self.cache, self.T = c, sum(rows) + extra
        self.q_start = ints([sum(rows[:i]) for i in range(len(rows) + 1)])
        self.kv_len = ints([max(n, 0) for n in lens])
        q = torch.randn(self.T, hq * d + wide, generator=g).to(dtype).to(DEV)
        self.q = q[:, wide:]
        self.max_q, self.max_kv, self.scale = max(max(rows), 1), max(max(lens), 1), d ** -0.5
        self.g = g
        if self.far:
            self.max_kv = 1 << 18
            table = torch.nn.functional.pad(c.table, (0, self.max_kv // page - c.table.shape[1]), value=-1)
            self.cache = wl.Cache(c.k, c.v, table, c.k_scale, c.v_scale)

    def tree(self):
        """A random tree per sequence: (words, positions)."""
        n_words = -(-max(self.rows) // 32)
        words, pos = [], []
        for c, n in zip(self.ctx, self.rows):
            seen, depth = [], []
            for i in range(n):
                p = int(torch.randint(-1, i, (1,), generator=self.g)) if i else -1
                seen.append((seen[p] if p >= 0 else 0) | 1 << i)
                depth.append(depth[p] + 1 if p >= 0 else 0)
            words += [[(v >> 32 * w & 0xFFFFFFFF) - ((v >> 32 * w + 31 & 1) << 32) for w in range(n_words)] for v in seen]
            pos += [c + e for e in depth]
        pad = self.T - len(words)
        return ints(words + [[-1] * n_words] * pad), ints(pos + [0] * pad)

    def run(self, wl, **kw):
        return wl.wl_attention(self.q, self.cache, self.q_start, self.kv_len, self.max_q, self.max_kv, self.scale, **kw)

    def check(self, wl, what="", **kw):
        o = torch.full((self.T, self.q.shape[1]), 3.0, dtype=self.q.dtype, device=DEV)
        self.run(wl, o=o, **kw)
        torch.cuda.synchronize()
        want, slack = ref.attention(self.q, self.cache, self.q_start, self.kv_len, self.scale, **kw)
        rows = ~torch.isnan(want).any(1)
        assert int(rows.sum()) == sum(self.rows)
        ref.assert_near(o[rows.to(DEV)], want[rows], slack[rows], what)
        assert (o[~rows.to(DEV)] == 3).all(), "a row outside every sequence was written"
        return o


# earlier keys, new tokens, query heads, key/value heads, d, page, window
CASES = [
    ([0], [1], 4, 1, 256, 16, 0),
    ([999], [1], 4, 1, 256, 16, 512),
    ([30, 31, 32, 0, 63], [1, 1, 1, 1, 1], 8, 2, 64, 32, 0),
    ([127, 500], [1, 1], 7, 1, 128, 64, 100),
    ([5, 0, 77], [3, 17, 8], 8, 8, 96, 16, 0),
    ([200], [40], 12, 4, 128, 16, 33),
    ([0], [130], 4, 1, 256, 64, 0),
    ([100, 0, 10], [60, 1, 129], 6, 2, 64, 128, 0),
    ([1500], [9], 32, 8, 256, 64, 0),
    ([2100], [2], 3, 3, 16, 1024, 1),
    ([300], [33], 40, 2, 48, 16, 64),
    ([17], [257], 2, 1, 256, 32, 100),
    ([700, 3], [2, 70], 9, 1, 208, 16, 0),
]


@pytest.mark.parametrize("fmt", [BF, I8, E4, F32])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_causal(wl, case, fmt):
    ctx, rows, hq, hkv, d, page, window = CASES[case]
    print(f"attention causal {CASES[case]} {fmt}", flush=True)
    Batch(wl, ctx, rows, hq, hkv, d, page, fmt, seed=case, extra=2, wide=8).check(wl, window=window)


TREES = [([100, 40], [8, 5], 4, 1, 256, 16, 0), ([0], [33], 8, 2, 64, 16, 0), ([500, 0, 33], [70, 1, 64], 8, 8, 128, 64, 50),
         ([31], [2], 32, 8, 256, 32, 0), ([1000], [48], 32, 8, 256, 64, 300), ([64], [31], 6, 3, 96, 16, 20)]


@pytest.mark.parametrize("fmt", [BF, I8, E4, F32])
@pytest.mark.parametrize("case", range(len(TREES)))
def test_tree(wl, case, fmt):
    ctx, rows, hq, hkv, d, page, window = TREES[case]
    print(f"attention tree {TREES[case]} {fmt}", flush=True)
    b = Batch(wl, ctx, rows, hq, hkv, d, page, fmt, seed=50 + case, extra=1)
    words, pos = b.tree()
    b.check(wl, tree=words, q_pos=pos, window=window)
    b.check(wl, tree=words, window=window)


@pytest.mark.parametrize("fmt", [BF, I8, F32])
def test_full_mask(wl, fmt):
    Batch(wl, [40, 0, 3], [5, 70, 1], 8, 2, 128, 16, fmt, seed=3).check(wl, mask="full")


@pytest.mark.parametrize("fmt", [BF, E4, F32])
def test_long_contexts_are_joined(wl, fmt):
    """Long keys for few queries, so that the work is split over the keys."""
    for ctx, rows, hq, hkv, d in (([6000], [1], 4, 1, 256), ([4097, 12, 2900], [1, 1, 1], 8, 4, 128), ([5000], [37], 4, 1, 64),
                                  ([3000], [90], 2, 1, 256)):
        print(f"attention long {ctx} {rows} {fmt}", flush=True)
        Batch(wl, ctx, rows, hq, hkv, d, 64, fmt, seed=11).check(wl)


@pytest.mark.parametrize("fmt", [BF, I8, F32])
def test_queries_without_keys(wl, fmt):
    b = Batch(wl, [20, 10, 0], [4, 40, 3], 4, 2, 64, 16, fmt, seed=4)
    words = torch.zeros(b.T, 2, dtype=torch.int32, device=DEV)
    pos = torch.full((b.T,), 1 << 20, dtype=torch.int32, device=DEV)
    o = b.run(wl, tree=words, q_pos=pos, window=3)        # the window is behind every key, the trees are empty
    torch.cuda.synchronize()
    assert (o == 0).all()
    words[5, 0] = 1 << 7
    o = b.run(wl, tree=words, q_pos=pos, window=3)
    torch.cuda.synchronize()
    assert (o[5] != 0).any() and (o[:5] == 0).all() and (o[6:] == 0).all()
    # fewer keys than new tokens: the first queries have no slot
    b.kv_len[0], b.kv_len[2] = 2, 0
    b.check(wl)
    o = b.run(wl)
    torch.cuda.synchronize()
    assert (o[:2] == 0).all() and (o[-3:] == 0).all() and (o[2:4] != 0).any()


@pytest.mark.parametrize("rows", [[1, 1], [3, 2], [150, 40]])
@pytest.mark.parametrize("fmt", [BF, I8, E4, F32])
def test_nan_and_infinity_of_unseen_keys(wl, fmt, rows):
    """Keys that a query does not see hold NaN and infinities; those it sees do not."""
    d, hkv = 128, 2
    ctx = [40, 70]
    b = Batch(wl, ctx, rows, 4, hkv, d, 16, fmt, seed=6)
    want = b.check(wl)
    bad = torch.full((1, hkv * d), float("nan"), dtype=b.q.dtype, device=DEV)
    bad[0, 1::2] = float("inf")
    # the last new token of each sequence: seen by itself alone
    for s in range(2):
        wl.wl_cache_write(b.cache, bad, bad, ints([s]), ints([ctx[s] + rows[s] - 1]))
    o = b.run(wl)
    torch.cuda.synchronize()
    last = torch.zeros(b.T, dtype=torch.bool, device=DEV)
    last[rows[0] - 1] = last[-1] = True
    assert torch.isnan(o[last]).any() and torch.isfinite(o[~last]).all()
    err = (o[~last].double() - want[~last].double()).abs().cpu()
    assert (err <= 4 * ref.half_step(BF) * (want[~last].abs().double().cpu() + 1)).all()
    # keys behind the window
    b = Batch(wl, ctx, rows, 4, hkv, d, 16, fmt, seed=6)
    win = max(rows) + 8
    want = b.run(wl, window=win).clone()
    first = [c - win for c in ctx]
    for s in range(2):
        for j in range(0, max(first[s], 0)):
            wl.wl_cache_write(b.cache, bad, bad, ints([s]), ints([j]))
    o = b.run(wl, window=win)
    torch.cuda.synchronize()
    assert torch.isfinite(o).all()
    assert ((o.double() - want.double()).abs().cpu() <= 4 * ref.half_step(BF) * (want.abs().double().cpu() + 1)).all()


@pytest.mark.parametrize("fmt", [BF, E4, F32])
def test_visible_nan_and_infinity_follow_the_formula(wl, fmt):
    d = 64
    b = Batch(wl, [33], [3], 2, 1, d, 16, fmt, seed=8)
    v = torch.randn(1, d, generator=b.g).to(b.q.dtype).to(DEV)
    w = v.clone()
    w[0, 5] = float("inf")
    wl.wl_cache_write(b.cache, v, w, ints([0]), ints([34]))
    o = b.run(wl).view(3, 2, d)
    torch.cuda.synchronize()
    assert torch.isfinite(o[0]).all()
    if fmt in (BF, F32):
        assert torch.isinf(o[1:, :, 5]).all() and torch.isfinite(o[1:, :, :5]).all() and torch.isfinite(o[1:, :, 6:]).all()
    else:
        assert torch.isnan(o[1:]).all()


@pytest.mark.parametrize("fmt", [BF, I8, F32])
def test_pages_that_are_none(wl, fmt):
    for rows in ([1, 2], [100, 3]):
        b = Batch(wl, [100, 90], rows, 4, 2, 64, 16, fmt, seed=5)
        b.cache.table[0, 2], b.cache.table[1, 0], b.cache.table[0, 5] = -1, b.cache.k.shape[0], 1 << 30
        b.check(wl)


@pytest.mark.parametrize("fmt", [I8, E4])
def test_fp32_queries_over_codes(wl, fmt):
    for ctx, rows, hq, hkv, d, page in (([70, 0], [1, 90], 4, 2, 96, 16), ([1500], [3], 4, 1, 256, 64), ([40], [5], 2, 2, 16, 32)):
        Batch(wl, ctx, rows, hq, hkv, d, page, fmt, seed=12, dtype=F32).check(wl, window=60)


@pytest.mark.parametrize("fmt", [BF, I8, F32])
@pytest.mark.parametrize("rows", [[2, 0, 1, 0], [60, 0, 41, 0]])
def test_idle_sequences(wl, rows, fmt):
    """Sequences of the batch without new tokens, with and without keys."""
    b = Batch(wl, [30, 40, 100, 0], rows, 8, 4, 64, 16, fmt, seed=13, extra=1)
    b.check(wl)
    b.check(wl, mask="full")


@pytest.mark.parametrize("fmt", [BF, E4, F32])
@pytest.mark.parametrize("scale", [0.0, -0.3, 1.5])
def test_scales(wl, scale, fmt):
    """No scale, a negative one, and one whose scores make the running maximum climb."""
    for ctx, rows, d in (([300, 20], [1, 3], 128), ([200], [150], 64), ([90], [40], 256)):
        b = Batch(wl, ctx, rows, 4, 2, d, 16, fmt, seed=14)
        b.scale = scale
        b.check(wl)


def test_pages_shared_by_sequences(wl):
    """A common first page: both sequences read it."""
    b = Batch(wl, [60, 60], [1, 1], 4, 2, 64, 16, BF, seed=15)
    b.cache.table[1, :2] = b.cache.table[0, :2]
    b.check(wl)


def test_limits_of_the_launch(wl):
    """max_q and max_kv below what the arrays say, lengths beyond the table, and
    starts that are no order: bounded, and nothing else is written."""
    b = Batch(wl, [50, 20], [6, 3], 4, 2, 64, 16, BF, seed=2)
    want, _ = ref.attention(b.q, b.cache, b.q_start, b.kv_len, b.scale)
    o = torch.full_like(b.q, 3.0)
    b.max_q = 4
    b.run(wl, o=o)
    torch.cuda.synchronize()
    assert (o[4:6] == 3).all() and (o[:4] != 3).any() and (o[6:] != 3).any()
    b.max_q, b.max_kv = 6, 30
    want, slack = ref.attention(b.q, b.cache, b.q_start, b.kv_len, b.scale, max_kv=30)
    ref.assert_near(b.run(wl), want, slack, "max_kv")
    b.max_kv = 1 << 30
    b.kv_len[0] = 1 << 30
    o = b.run(wl, mask="full")
    b.q_start[1], b.q_start[2] = -5, 1 << 30
    b.run(wl)
    b.q_start[0], b.q_start[1] = 7, 2
    b.run(wl)
    torch.cuda.synchronize()


def test_output_over_the_queries(wl):
    for rows in ([1, 1, 1], [50, 70, 1]):
        for fmt in (BF, E4, F32):
            b = Batch(wl, [40, 900, 0], rows, 8, 2, 128, 32, fmt, seed=7, extra=1, wide=16)
            want = b.run(wl).clone()
            b.run(wl, o=b.q)
            torch.cuda.synchronize()
            n = sum(rows)
            assert torch.equal(b.q[:n], want[:n])


def test_empty_refusals_and_determinism(wl):
    b = Batch(wl, [2000, 30], [1, 1], 4, 1, 128, 16, BF, seed=9)
    assert wl.wl_attention(b.q[:0], b.cache, b.q_start, b.kv_len, 1, 100, 1.0).shape == (0, b.q.shape[1])
    first = b.run(wl).clone()
    for _ in range(3):
        assert torch.equal(b.run(wl), first)
    words = torch.zeros(b.T, 1, dtype=torch.int32, device=DEV)
    for bad in (dict(mask="tree"), dict(mask="other"), dict(tree=words, mask="causal"), dict(q_pos=words[:, 0]), dict(tree=words[:1])):
        with pytest.raises(ValueError):
            b.run(wl, **bad)
    for bad in (dict(window=-1), dict(window=4, mask="full")):
        with pytest.raises(wl.WlError):
            b.run(wl, **bad)
    with pytest.raises(ValueError):
        wl.wl_attention(b.q.float(), b.cache, b.q_start.long(), b.kv_len, 1, 100, 1.0)
    call = wl.attention_call(b.q, b.cache, b.q_start, b.kv_len, 1, 4000, 1.0)
    need = wl.lib.wl_attention_workspace_bytes(call.args)
    if need:
        call.ws = wl.new_workspace(need, DEV)[:need - 256]
        with pytest.raises(wl.WlError) as e:
            call.launch()
        assert e.value.status == wl.WL_ERR_WORKSPACE


@pytest.mark.parametrize("rows,hq", [([1, 1, 1], 4), ([9, 2, 40], 8)])
def test_replay_follows_lengths(wl, rows, hq):
    """A captured call reads queries, lengths and tables at each replay; two graphs
    that share a workspace run one after the other."""
    b = Batch(wl, [3000, 200, 64], rows, hq, 1, 128, 32, BF, seed=10)
    b.max_kv += 64
    args = (b.q, b.cache, b.q_start, b.kv_len, b.max_q, b.max_kv, b.scale)
    ws = wl.new_workspace(1 << 27, DEV)
    calls = [wl.attention_call(*args, ws=ws), wl.attention_call(*args, ws=ws, window=100)]
    eager = [wl.attention_call(*args), wl.attention_call(*args, window=100)]
    graphs = []
    for c in calls:
        c.launch()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.launch()
        graphs.append(g)
    lens = b.kv_len.clone()
    for step in range(4):
        b.q.copy_(torch.randn(b.q.shape, generator=b.g).to(BF))
        b.kv_len.copy_(lens - 37 * step)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        got = [c.out.clone() for c in calls]
        for c, o in zip(eager, got):
            assert torch.equal(c.launch(), o)
        torch.cuda.synchronize()


def test_far_pages_of_a_large_pool(wl):
    """Element offsets past 2^32, at pages of a pool that long."""
    page, n_kv, d, n_pages = 1024, 8, 256, 2200
    table = ints([[n_pages - 1, 2100], [0, 1]])
    c = wl.new_cache(n_pages, n_kv, page, d, table, I8)
    g = torch.Generator().manual_seed(1)
    n = 1100
    k, v = (torch.randn(n, n_kv * d, generator=g).to(BF).to(DEV) for _ in range(2))
    slot = torch.arange(n, dtype=torch.int32, device=DEV)
    for s in range(2):
        wl.wl_cache_write(c, k, v, ints([s] * n), slot)
    for rows in (1, 40):
        q = torch.randn(rows, n_kv * d, generator=g).to(BF).to(DEV)
        o = wl.wl_attention(torch.cat((q, q)), c, ints([0, rows, 2 * rows]), ints([n, n]), rows, n, d ** -0.5)
        torch.cuda.synchronize()
        assert torch.equal(o[:rows], o[rows:]) and torch.isfinite(o).all() and (o != 0).any()


@pytest.mark.parametrize("fmt", [BF, I8, F32])
@pytest.mark.parametrize("rows, n_seq", [(1, 64), (1, 65), (5, 7), (40, 3), (40, 64), (70, 2)])
def test_uneven_sequences_far_below_the_limit(wl, rows, n_seq, fmt):
    """Lengths from one key to thousands, some sequences idle, and a max_kv that none
    of them comes near: pieces follow the lengths, up to 64 sequences."""
    g = torch.Generator().manual_seed(rows * 100 + n_seq)
    ctx = [int(v) for v in torch.randint(0, 300, (n_seq,), generator=g)]
    ctx[n_seq // 2], ctx[-1] = 2900, 0
    new = [0 if i % 5 == 4 else 1 + int(torch.randint(0, rows, (1,), generator=g)) for i in range(n_seq)]
    b = Batch(wl, ctx, new, 4, 1, 128, 16, fmt)
    b.check(wl)
    tree, pos = b.tree()
    b.check(wl, "tree", mask="tree", tree=tree, q_pos=pos)
    b.check(wl, "window", window=600)
    # a longer page table, whose further entries are no pages
    c = b.cache
    table = torch.nn.functional.pad(c.table, (0, (1 << 16) - c.table.shape[1]), value=-1)
    b.cache = wl.Cache(c.k, c.v, table, c.k_scale, c.v_scale)
    b.max_q, b.max_kv = rows, 1 << 20
    b.check(wl, "max_kv of a million")


@pytest.fixture
def far(monkeypatch):
    """A max_kv at which calls of more than 64 rows per head are taken to be large:
    32 rows per wave, and eight waves at 129 to 256 rows over int8 and e4m3."""
    monkeypatch.setattr(Batch, "far", True)


@pytest.mark.parametrize("fmt", [BF, I8, E4, F32])
@pytest.mark.parametrize("case", [c for c in range(len(CASES)) if max(CASES[c][1]) > 1 and not CASES[c][6]])
def test_causal_under_a_large_limit(wl, far, case, fmt):
    test_causal(wl, case, fmt)


@pytest.mark.parametrize("fmt", [BF, I8, E4, F32])
@pytest.mark.parametrize("d, rows, hq", [(64, [70, 1, 64], 4), (128, [24, 25, 3], 8), (256, [64, 33, 0], 3), (256, [90, 30, 100], 2),
                                         (96, [256, 17, 129], 1), (256, [48, 31, 35], 4), (256, [40, 200, 16], 1)])
def test_shares_of_the_rows(wl, far, d, rows, hq, fmt):
    """Rows of a head from a wave's to several workgroups', by sequences that differ."""
    print(f"attention rows {rows} {hq} {d} {fmt}", flush=True)
    b = Batch(wl, [33, 400, 77], rows, hq, 1, d, 32, fmt, seed=21, extra=1)
    b.check(wl)
    words, pos = b.tree()
    b.check(wl, "tree", tree=words, q_pos=pos, window=60)
    b.check(wl, "full", mask="full")


@pytest.mark.parametrize("fmt", [BF, I8, E4, F32])
def test_unseen_and_absent_keys_under_a_large_limit(wl, far, fmt):
    for rows in ([150, 40], [100, 3], [60, 60]):
        test_nan_and_infinity_of_unseen_keys(wl, fmt, rows)
    test_pages_that_are_none(wl, fmt)
    test_queries_without_keys(wl, fmt)


@pytest.mark.parametrize("fmt", [BF, E4, F32])
@pytest.mark.parametrize("scale", [0.0, -0.3, 1.5])
def test_scales_under_a_large_limit(wl, far, scale, fmt):
    test_scales(wl, scale, fmt)


@pytest.mark.parametrize("fmt, d, keys, bad", [
    (F32, 64, 129, [128]), (BF, 256, 513, [512]), (I8, 128, 513, [512]), (E4, 256, 513, [512]),   # the newest key, alone in its piece
    (F32, 128, 192, range(64, 128)), (BF, 128, 768, range(256, 512)), (I8, 64, 768, range(0, 256)),   # a piece of NaN between others
    (F32, 128, 300, [70]), (BF, 64, 2000, [300]), (E4, 128, 5000, [4999])])                       # one of many
@pytest.mark.parametrize("limit", [0, 1 << 16])
def test_visible_nan_reaches_the_output_through_the_join(wl, fmt, d, keys, bad, limit):
    """One token over divided keys: a NaN in a visible key makes every score of the row's
    softmax NaN, whatever the other pieces hold and however large their scores are."""
    print(f"attention NaN {fmt} {d} {keys} {limit}", flush=True)
    for loud in (1.0, 300.0):
        b = Batch(wl, [keys - 1], [1], 4, 1, d, 16, fmt, seed=31)
        b.max_kv, b.scale = max(limit, keys), b.scale * loud
        if limit:
            table = torch.nn.functional.pad(b.cache.table, (0, limit // 16 - b.cache.table.shape[1]), value=-1)
            b.cache = wl.Cache(b.cache.k, b.cache.v, table, b.cache.k_scale, b.cache.v_scale)
        assert wl.lib.wl_attention_workspace_bytes(wl.attention_call(b.q, b.cache, b.q_start, b.kv_len, 1, b.max_kv, 1.0).args), "undivided"
        o = b.run(wl)
        torch.cuda.synchronize()
        assert torch.isfinite(o).all()
        k = torch.full((len(bad), d), float("nan"), dtype=b.q.dtype, device=DEV)
        wl.wl_cache_write(b.cache, k, torch.ones_like(k), ints([0] * len(bad)), ints(list(bad)))
        o = b.run(wl)
        torch.cuda.synchronize()
        assert torch.isnan(o).all(), loud


@pytest.mark.parametrize("fmt", [BF, E4, F32])
def test_queries_of_nan_are_not_walked_key_by_key(wl, fmt):
    """A prompt of NaN ends with the first key that each row sees: a wave would walk 16
    rows one after the other, a quarter of a microsecond a key, 15 ms in all."""
    b = Batch(wl, [0], [4096], 4, 1, 64, 64, fmt, seed=32)
    b.q[5:].fill_(float("nan"))
    for _ in range(2):
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda.synchronize()
        start.record()
        o = b.run(wl)
        end.record()
        torch.cuda.synchronize()
    assert torch.isnan(o[5:]).all() and torch.isfinite(o[:5]).all()
    assert start.elapsed_time(end) < 2
