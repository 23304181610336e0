"""The latent cache (written, read back) and the attention over it against their
definitions in 64 bits, at the bars derived in serve_ref."""
from __future__ import annotations

import random

import pytest
import torch

from tests import layer_ref, serve_ref
from tests.layer_ref import CHAIN, EPS32, f64

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def wl():
    from linear_02_amd import wl as mod
    return mod


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def table_of(lens, page, rng, spare=3, width=None):
    """Pages of every sequence in shuffled order, -1 behind the last."""
    need = [-(-n // page) for n in lens]
    ids = list(range(sum(need) + spare))
    rng.shuffle(ids)
    rows, at = [], 0
    for n in need:
        rows.append(ids[at:at + n] + [-1] * ((width or max(max(need), 1)) - n))
        at += n
    return rows, len(ids)


def fill(cache, g):
    """Normal values in every row of a cache's pool, on the device."""
    x = torch.randn(*cache.rows.shape[:2], cache.latent + cache.rot, generator=g)
    if cache.rows.dtype != torch.uint8:
        cache.rows.copy_(x)
        return
    most = x[..., :cache.latent].abs().amax(-1)
    codes = (x[..., :cache.latent] * 448 / most[..., None]).clamp(-448, 448).to(E4M3)
    cache.rows.copy_(torch.cat((codes.view(torch.uint8), x[..., cache.latent:].to(BF).view(torch.uint8)), -1))
    cache.scale.copy_(most / 448)


# ---- written and read back --------------------------------------------------------


@pytest.mark.parametrize("fmt", [BF, F32, E4M3])
@pytest.mark.parametrize("L,R,H,N", [(512, 64, 16, 128), (128, 32, 1, 64), (256, 64, 7, 96), (512, 32, 128, 0)])
@pytest.mark.parametrize("T", [1, 37, 300])
def test_write_and_read(wl, fmt, L, R, H, N, T):
    rng, g = random.Random(L + R + T), torch.Generator().manual_seed(L + R + T)
    dt = F32 if fmt == F32 else BF
    for k, (norm, style, scale, with_pos) in enumerate(((True, False, 1.0, False), (False, True, 1.25, True))):
        page = (16, 64)[k]
        table, n_pages = table_of([200, 0, 500], page, rng)
        cache = wl.new_latent_cache(n_pages, page, L, R, i32(table), fmt)
        cache.rows.zero_()
        if cache.scale is not None:
            cache.scale.zero_()
        places = [(s, j) for s, n in ((0, 200), (2, 500)) for j in range(n)]
        rng.shuffle(places)
        seq, slot = [p[0] for p in places[:T]], [p[1] for p in places[:T]]
        skipped = set()
        if T > 10:      # sequences and slots that there are not
            for t, (a, b) in enumerate(((-1, 3), (3, 0), (0, -1), (0, 260), (1, 0), (2, 1 << 30))):
                seq[t], slot[t] = a, b
                skipped.add(t)
        wide = torch.randn(T, L + R + 24, generator=g).to(dt).to(DEV)
        c = wide[:, 8:8 + L + R]
        q = torch.randn(T, H * (N + R) + 8, generator=g).to(dt).to(DEV)[:, :H * (N + R)]
        w = (torch.randn(L, generator=g) * 0.3).to(dt).to(DEV) if norm else None
        freq, m = wl.rope_frequencies(R, 10000.0, scaling="plain", device=DEV)
        pos = i32([rng.randrange(-5, 1000000) for _ in range(T)]) if with_pos else None
        q_out = torch.full_like(q, 7.0)
        rope = wl.Rope(freq, interleaved=style, scale=scale)
        wl.wl_latent_write(cache, c, i32(seq), i32(slot), q=q, n_q=H, rope=rope, pos=pos, norm=w, eps=1e-6, offset=1.0, q_out=q_out)
        back = torch.full((T, L + R), 9.0, dtype=dt, device=DEV)
        wl.wl_latent_read(cache, i32(seq), i32(slot), out=back)
        p = pos if with_pos else i32(slot)
        none = [t for t in range(T) if not 0 <= seq[t] < 3]
        live = [t for t in range(T) if t not in skipped]
        # Q: the last R of every head turned
        x = f64(q).view(T, H, N + R)
        turned, mag = layer_ref.rotate(x[..., N:].reshape(T, H * R), R, p, freq, scale, style)
        ref = torch.cat((x[..., :N], turned.view(T, H, R)), -1).flatten(1)
        slack = torch.cat((torch.zeros(T, H, N), mag.view(T, H, R)), -1).flatten(1) * 8 * EPS32
        ok = [t for t in range(T) if t not in none]
        if ok:
            layer_ref.assert_near(q_out[ok], ref[ok], slack[ok], "q")
        assert (q_out[none] == 7.0).all()
        # the rows
        z = f64(c)
        latent, turned_key = z[:, :L], layer_ref.rotate(c[:, L:], R, p, freq, scale, style)
        if norm:
            latent = layer_ref.rms(latent, f64(w), 1e-6, 1.0)[0]
        key, kmag = turned_key
        got = f64(back)
        assert (back[list(skipped)] == 9.0).all()
        layer_ref.assert_near(back[live][:, L:], key[live], 8 * EPS32 * kmag[live], "key")
        if fmt == E4M3:
            # the code's own step at worst (2^-4 of the value, 2^-10 of the top one below its smallest exponent), and bf16
            most = latent.abs().amax(1, keepdim=True)
            bar = (2 ** -4 + 2 ** -8) * latent.abs() * (1 + 2 ** -4) + most / 448 * 2 ** -10 + CHAIN * EPS32 * most
            assert ((got[live][:, :L] - latent[live]).abs() <= bar[live]).all()
            if not norm:        # the codes themselves
                codes, sc = layer_ref.codes(z[:, :L], E4M3)
                assert (got[live][:, :L] - (codes * sc[:, None])[live]).abs().le((codes * sc[:, None]).abs()[live] * 2 ** -8 * 1.01).all()
        else:
            layer_ref.assert_near(back[live][:, :L], latent[live], CHAIN * EPS32 * latent[live].abs(), "latent")


def test_write_in_place_and_without_q(wl):
    g = torch.Generator().manual_seed(1)
    table, n_pages = table_of([50], 16, random.Random(1))
    freq, _ = wl.rope_frequencies(64, device=DEV)
    c, q = torch.randn(50, 576, generator=g).to(BF).to(DEV), torch.randn(50, 4 * 192, generator=g).to(BF).to(DEV)
    seq, slot = i32([0] * 50), i32(list(range(50)))
    for style in (False, True):
        a, b = (wl.new_latent_cache(n_pages, 16, 512, 64, i32(table)) for _ in range(2))
        rope, mine = wl.Rope(freq, interleaved=style), q.clone()
        out = wl.wl_latent_write(a, c, seq, slot, q=q, n_q=4, rope=rope)
        assert wl.wl_latent_write(a, c, seq, slot, q=mine, n_q=4, rope=rope, q_out=mine) is mine and torch.equal(mine, out)
        assert wl.wl_latent_write(b, c, seq, slot, rope=rope) is None
        assert torch.equal(wl.wl_latent_read(a, seq, slot), wl.wl_latent_read(b, seq, slot))
        assert torch.equal(wl.wl_latent_write(b, c, seq, slot, q=q, n_q=4), q)
        assert torch.equal(wl.wl_latent_read(b, seq, slot), c)      # neither norm nor rotation


def test_rows_of_zeros_and_infinities_in_codes(wl):
    cache = wl.new_latent_cache(2, 16, 128, 32, i32([[1]]), E4M3)
    c = torch.zeros(4, 160, dtype=BF)
    c[1, 5], c[2, 7], c[3, :128] = float("inf"), float("nan"), 1e-38
    seq, slot = i32([0] * 4), i32([0, 1, 2, 3])
    wl.wl_latent_write(cache, c.to(DEV), seq, slot)
    back = wl.wl_latent_read(cache, seq, slot).cpu().float()
    assert (back[0] == 0).all() and back[1, :128].isnan().all() and back[2, :128].isnan().all()
    assert ((back[3, :128] - 1e-38).abs() < 1e-39).all()


# ---- attention ------------------------------------------------------------------------


class Batch:
    """Sequences of (earlier keys, new tokens) over a filled cache."""

    def __init__(self, wl, seqs, H, L=512, R=64, N=128, V=128, fmt=BF, page=16, seed=0, weights=True, gap=0, tail=0):
        g, rng = torch.Generator().manual_seed(seed), random.Random(seed)
        dt = F32 if fmt == F32 else BF
        lens, rows = [a + b for a, b in seqs], [b for _, b in seqs]
        table, n_pages = table_of(lens, page, rng)
        self.cache = wl.new_latent_cache(n_pages, page, L, R, i32(table), fmt)
        fill(self.cache, g)
        self.T = gap + sum(rows) + tail
        if not weights:
            N = V = L
        self.w = (torch.randn(H, N + V, L, generator=g) * L ** -0.5).to(dt).to(DEV) if weights else None
        self.q = (torch.randn(self.T, H * (N + R), generator=g) * (1.0 if weights else (192 / (L + R)) ** 0.5)).to(dt).to(DEV)
        self.starts = [gap + sum(rows[:i]) for i in range(len(rows) + 1)]
        self.lens, self.rows, self.H, self.V, self.scale = lens, rows, H, V, (N + R) ** -0.5
        self.rng = rng

    def trees(self):
        """A tree of drafted tokens for every sequence: masks and positions."""
        words, bits, pos = -(-max(self.rows) // 32), [[0]] * self.starts[0], [0] * self.starts[0]
        bits = [[0] * words for _ in bits]
        for n, total in zip(self.rows, self.lens):
            seen, depth = [], []
            for i in range(n):
                p = self.rng.randrange(-1, i)
                seen.append((seen[p] if p >= 0 else 0) | 1 << i)
                depth.append(depth[p] + 1 if p >= 0 else 0)
            bits += [[(v >> 32 * k & 0xffffffff) - (1 << 32) * (v >> 32 * k + 31 & 1) for k in range(words)] for v in seen]
            pos += [total - n + e for e in depth]
        pad = self.T - len(bits)
        return i32(bits + [[0] * words] * pad), i32(pos + [0] * pad)

    def run(self, wl, max_q=None, max_kv=None, **kw):
        o = torch.full((self.T, self.H * self.V), 5.0, dtype=self.q.dtype, device=DEV)
        wl.wl_latent_attention(self.q, self.cache, self.w, i32(self.starts), i32(self.lens), max_q or max(self.rows),
                               max_kv if max_kv is not None else max(self.lens), self.scale, o=o, **kw)
        return o

    def check(self, wl, what="", max_q=None, max_kv=None, form="auto", expanded=False, **kw):
        o = self.run(wl, max_q, max_kv, form=form, **kw)
        ref, slack = serve_ref.latent_attention(self.q, self.cache, self.w, i32(self.starts), i32(self.lens), self.scale,
                                                max_kv=max_kv, max_q=max_q, expanded=expanded, **kw)
        mine = ~ref[:, 0].isnan()
        assert (o[~mine.to(DEV)] == 5.0).all(), f"{what}: rows of nobody"
        got = o[mine.to(DEV)]
        layer_ref.assert_near(got, ref[mine], slack[mine], what)
        if got.numel() >= 256 and got.dtype == BF and float(ref[mine].norm()) > 0:
            rel = float((f64(got) - ref[mine]).norm() / ref[mine].norm())
            assert rel <= serve_ref.REL_BF16, f"{what}: {rel}"
        return o


SHAPES = [(512, 64, 128, 128), (256, 32, 64, 64), (128, 64, 96, 32)]


@pytest.mark.parametrize("fmt", [BF, E4M3, F32])
@pytest.mark.parametrize("L,R,N,V", SHAPES)
@pytest.mark.parametrize("H,seqs", [
    (16, [(0, 1)]), (16, [(999, 1)]), (1, [(30, 1), (0, 1), (31, 1), (32, 1), (33, 1)]), (20, [(100, 1), (0, 3), (250, 2)]),
    (128, [(70, 1), (15, 1)]), (4, [(5, 7), (100, 0), (64, 33), (0, 16)]), (7, [(200, 17)])])
def test_attention_causal(wl, fmt, L, R, N, V, H, seqs):
    Batch(wl, seqs, H, L, R, N, V, fmt, seed=H + len(seqs), gap=2, tail=1).check(wl, "causal", form="absorbed")


@pytest.mark.parametrize("fmt", [BF, E4M3, F32])
@pytest.mark.parametrize("window", [0, 1, 40])
def test_attention_trees_windows_and_full(wl, fmt, window):
    b = Batch(wl, [(80, 9), (0, 40), (300, 1), (33, 24)], 12, fmt=fmt, page=32, seed=3)
    tree, pos = b.trees()
    b.check(wl, "tree", tree=tree, q_pos=pos, window=window, form="absorbed")
    b.check(wl, "tree without positions", tree=tree, window=window, form="absorbed")
    b.check(wl, "causal", window=window, form="absorbed")
    if not window:
        b.check(wl, "full", mask="full", form="absorbed")


@pytest.mark.parametrize("fmt", [BF, E4M3, F32])
@pytest.mark.parametrize("L,R", [(512, 64), (512, 32), (128, 32)])
def test_attention_in_the_latent_space(wl, fmt, L, R):
    """Without weights."""
    Batch(wl, [(90, 3), (500, 1), (0, 5)], 16, L, R, fmt=fmt, weights=False, seed=4, gap=1).check(wl, "latent")


@pytest.mark.parametrize("fmt", [BF, E4M3, F32])
def test_long_caches_divided(wl, fmt):
    b = Batch(wl, [(5000, 1), (17, 1), (2600, 1)], 16, fmt=fmt, page=64, seed=5)
    b.check(wl, "divided")
    b.check(wl, "divided, far max_kv", max_kv=1 << 20)
    Batch(wl, [(4000, 6)], 8, fmt=fmt, page=128, seed=6).check(wl, "few rows over a long cache")
    Batch(wl, [(3000, 2)], 128, 512, 64, 64, 64, fmt=fmt, page=64, seed=7).check(wl, "many heads")


@pytest.mark.parametrize("fmt", [BF, E4M3, F32])
def test_more_sequences_than_lanes(wl, fmt):
    rng = random.Random(8)
    Batch(wl, [(rng.randrange(0, 700), rng.choice((0, 1, 1, 2))) for _ in range(70)], 4, 256, 64, 64, 64, fmt, seed=8).check(wl, "70 sequences")


@pytest.mark.parametrize("fmt", [BF, E4M3, F32])
@pytest.mark.parametrize("n_seq,H,V", [(70, 32, 64), (130, 16, 32), (40, 48, 96)])
def test_joins_of_many_units(wl, fmt, n_seq, H, V):
    """Divided keys of more than 128 units of 16 tokens and a head, below and above a lane a sequence."""
    rng = random.Random(n_seq)
    seqs = [(rng.choice((0, 20, 300, 1500)), rng.choice((0, 1, 1, 2))) for _ in range(n_seq)]
    Batch(wl, seqs, H, 128, 64, 64, V, fmt, page=32, seed=n_seq, gap=1, tail=20).check(wl, "many units", max_kv=4000, form="absorbed")


@pytest.mark.parametrize("fmt", [BF, E4M3, F32])
def test_captured_and_replayed_over_changing_lengths(wl, fmt):
    """Lengths and rows that change between replays, the same call made eagerly beside them."""
    b = Batch(wl, [(900, 2), (37, 1), (400, 3)], 12, fmt=fmt, page=32, seed=16, tail=3)
    starts, lens = i32(b.starts), i32(b.lens)
    call = wl.latent_attention_call(b.q, b.cache, b.w, starts, lens, 3, 1000, b.scale)
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        call.launch()
    torch.cuda.current_stream().wait_stream(s)
    for k, (first, rows) in enumerate([([902, 38, 403], b.starts), ([0, 38, 1], b.starts), ([500, 1, 403], [0, 3, 3, 4]), ([902, 0, 20], [2, 2, 3, 6])]):
        starts.copy_(i32(rows))
        lens.copy_(i32(first))
        b.q.copy_(torch.randn(b.q.shape, generator=torch.Generator().manual_seed(k)))
        call.out.fill_(5.0)
        g.replay()
        o = torch.full_like(call.out, 5.0)
        wl.wl_latent_attention(b.q, b.cache, b.w, starts, lens, 3, 1000, b.scale, o=o)
        assert torch.equal(call.out, o)
        assert (o[rows[-1]:] == 5.0).all() and (o[:rows[0]] == 5.0).all()


@pytest.mark.parametrize("fmt", [BF, E4M3, F32])
def test_limits_of_rows_and_keys(wl, fmt):
    """Rows beyond max_q have no result, keys beyond max_kv or the table are not seen, a sequence shorter than its
    new tokens has rows that see nothing."""
    b = Batch(wl, [(60, 9), (10, 4)], 6, fmt=fmt, seed=9, gap=1)
    b.check(wl, "max_q", max_q=5, form="absorbed")
    b.check(wl, "max_kv", max_kv=37, form="absorbed")
    b.check(wl, "no keys", max_kv=0, form="absorbed")
    b.lens = [3, 1000]
    o = b.check(wl, "short and long", max_kv=1000, form="absorbed")
    assert (o[1:7] == 0).all()


def test_missing_pages(wl):
    for fmt in (BF, E4M3, F32):
        b = Batch(wl, [(100, 2), (40, 1)], 8, fmt=fmt, seed=10)
        t = b.cache.table
        t[0, 2], t[0, 4], t[1, 0], t[1, 1], t[1, 2] = -1, 1 << 20, -5, 1 << 30, -1
        o = b.check(wl, "missing pages", form="absorbed")
        assert (o[2] == 0).all()


@pytest.mark.parametrize("fmt", [BF, E4M3, F32])
def test_unseen_keys_have_no_influence(wl, fmt):
    """NaN and infinities in rows that no query sees, or that some do not see."""
    b = Batch(wl, [(70, 4), (33, 1)], 9, fmt=fmt, seed=11)
    clean = b.check(wl, "clean", window=20, form="absorbed")
    ref, slack = serve_ref.latent_attention(b.q, b.cache, b.w, i32(b.starts), i32(b.lens), b.scale, window=20)
    last = [b.cache.table[s, (n - 1) // 16].item() for s, n in enumerate(b.lens)]
    bad = float("nan")
    rows = b.cache.rows
    as_bad = (lambda r: r.fill_(0x7F)) if fmt == E4M3 else (lambda r: r.fill_(bad))
    used = {int(p) for p in b.cache.table.flatten().tolist() if p >= 0}
    for p in range(rows.shape[0]):
        if p not in used:
            as_bad(rows[p])
    for s, n in enumerate(b.lens):
        as_bad(rows[last[s], (n - 1) % 16 + 1:])            # behind the last key
    as_bad(rows[b.cache.table[0, 0].item()])                # below the window
    if b.cache.scale is not None:
        b.cache.scale[b.cache.table[0, 0].item()] = float("inf")
    assert torch.equal(b.run(wl, window=20, form="absorbed"), clean)
    # the last key of sequence 0 is seen by its last query alone
    as_bad(rows[last[0], (b.lens[0] - 1) % 16])
    o = b.run(wl, window=20, form="absorbed")
    assert o[3].isnan().all() and torch.equal(o[4:], clean[4:])
    # the others share its tile of keys: summed anew, in another order, within the same bar
    layer_ref.assert_near(o[:3], ref[:3], slack[:3], "rows beside one that sees it")


def test_weightless_keys_of_minus_infinity(wl):
    """A key of -inf has weight 0 where its score is -inf."""
    b = Batch(wl, [(40, 1)], 2, 128, 32, weights=False, seed=12)
    b.q.abs_()
    page, off = b.cache.table[0, 1].item(), 3
    clean_rows = b.cache.rows.clone()
    b.cache.rows[page, off, 128:] = -float("inf")
    o = b.run(wl)
    b.cache.rows.copy_(clean_rows)
    b.cache.table[0, 1] = b.cache.table[0, 1]
    ref = serve_ref.latent_attention(b.q, b.cache, None, i32(b.starts), i32(b.lens), b.scale)[0]
    c, key, _ = serve_ref.latent_rows(b.cache, 0, 41)
    q = f64(b.q).view(1, 2, 160)[0]
    sc = (q[:, :128] @ c.T + q[:, 128:] @ key.T) * b.scale
    sc[:, 19] = -torch.inf
    ref = (sc.softmax(-1) @ c).flatten()
    assert float((f64(o)[0] - ref).norm() / ref.norm()) <= serve_ref.REL_BF16


def test_scales(wl):
    for scale in (0.0, -0.1, 3.0):
        for fmt in (BF, F32):
            b = Batch(wl, [(150, 2)], 5, fmt=fmt, seed=13)
            b.scale = scale
            b.check(wl, f"scale {scale}", form="absorbed") if abs(scale) < 1 else b.run(wl)


def test_strided_rows(wl):
    b = Batch(wl, [(50, 3), (10, 2)], 4, seed=14)
    wide = torch.full((5, b.q.shape[1] + 40), float("nan"), dtype=BF, device=DEV)
    wide[:, 16:16 + b.q.shape[1]] = b.q
    out = torch.full((5, 4 * 128 + 16), 3.0, dtype=BF, device=DEV)
    ref = b.run(wl)
    wl.wl_latent_attention(wide[:, 16:16 + b.q.shape[1]], b.cache, b.w, i32(b.starts), i32(b.lens), 3, 53, b.scale, o=out[:, 8:520])
    assert torch.equal(out[:, 8:520], ref) and (out[:, :8] == 3).all() and (out[:, 520:] == 3).all()


def test_repeatable(wl):
    b = Batch(wl, [(3000, 2), (100, 3)], 16, page=64, seed=15)
    first = b.run(wl)
    for _ in range(20):
        assert torch.equal(b.run(wl), first)
