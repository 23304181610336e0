"""wl_rope, wl_cache_write and wl_cache_read against their 64-bit definitions."""
from __future__ import annotations

import math

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


def draw(seed, *shape, dtype=BF, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype).to(DEV)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


# (T, q heads, k heads, d, rotated)
SHAPES = [(1, 4, 1, 256, 256), (1, 1, 0, 8, 8), (3, 7, 1, 96, 96), (5, 2, 2, 64, 16), (2, 0, 3, 24, 16), (130, 32, 8, 128, 64),
          (3000, 2, 1, 16, 16), (9, 5, 5, 200, 184)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_rope(wl, shape, interleaved, dtype):
    T, nq, nk, d, rot = SHAPES[shape]
    print(f"rope {SHAPES[shape]} interleaved={interleaved} {dtype}", flush=True)
    pos = ints([(t * 7919 + 123456) % 1000003 * (-1) ** t for t in range(T)])
    freq, scale = wl.rope_frequencies(rot, scaling="parts", factor=8.0, device=DEV)
    rope = wl.Rope(freq, interleaved=interleaved, scale=scale)
    qkv = draw(1, T, (nq + 2 * nk) * d + 8, dtype=dtype)         # rows with K and V beside Q
    q = qkv[:, :nq * d] if nq else None
    k = qkv[:, nq * d:(nq + nk) * d] if nk else None
    for weights in (False, True):
        wq, wk = (draw(2, d, dtype=dtype, std=0.3), draw(3, d, dtype=dtype, std=0.3)) if weights else (None, None)
        got = wl.wl_rope(q, k, pos, rope, d, q_norm=wq if nq else None, k_norm=wk if nk else None, eps=1e-5, offset=1.0)
        torch.cuda.synchronize()
        for out, x, w in ((got[0], q, wq), (got[1], k, wk)):
            if x is None:
                continue
            r, mag = ref.rotate(x, d, pos, freq, scale, interleaved, w, 1e-5, 1.0)
            ref.assert_near(out, r, (ref.CHAIN + 16) * ref.EPS32 * mag, f"weights={weights}")


def test_rope_in_place_and_back(wl):
    T, d = 33, 128
    freq, _ = wl.rope_frequencies(d, device=DEV)
    pos = torch.arange(T, dtype=torch.int32, device=DEV) + 5000
    qkv = draw(1, T, 6 * d, dtype=F32)
    before = qkv.clone()
    q, k = qkv[:, :4 * d], qkv[:, 4 * d:5 * d]
    want = wl.wl_rope(q, k, pos, wl.Rope(freq), d)
    wl.wl_rope(q, k, pos, wl.Rope(freq), d, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(qkv[:, 5 * d:], before[:, 5 * d:])
    wl.wl_rope(q, k, -pos, wl.Rope(freq), d, q_out=q, k_out=k)   # the transpose turns back
    torch.cuda.synchronize()
    pair = before.abs().cpu().double() + 8
    assert ((qkv - before).abs().cpu().double() <= 64 * ref.EPS32 * pair).all()


def test_rope_gradient_against_differences(wl):
    """The gradient of sum(g . rope(x)) is rope(g) at the negated positions."""
    T, d = 3, 64
    freq, scale = wl.rope_frequencies(32, scaling="parts", factor=4.0, device=DEV)
    rope, pos = wl.Rope(freq, interleaved=True, scale=scale), ints([3, 70000, -9])
    x, g = draw(1, T, d, dtype=F32), draw(2, T, d, dtype=F32)
    grad = wl.wl_rope(g, None, -pos, rope, d)[0]
    for at in (0, 1, 17, 31, 32, 63):
        e = torch.zeros_like(x)
        e[:, at] = 1.0
        # the operation is linear: the difference over a step of 1 is exact up to fp32
        diff = ((wl.wl_rope(x + e, None, pos, rope, d)[0] - wl.wl_rope(x, None, pos, rope, d)[0]) * g).sum(1)
        assert ((diff - grad[:, at]).abs() <= 1e-4 * (g.abs().sum(1) + 1)).all()


def place(cache, T, seed):
    """Tokens with distinct places in a cache whose table is shuffled."""
    g = torch.Generator().manual_seed(seed)
    n_seq, room = cache.table.shape[0], cache.table.shape[1] * cache.k.shape[2]
    at = torch.randperm(n_seq * room, generator=g)[:T]
    return ints((at // room).tolist()), ints((at % room).tolist())


def make(wl, fmt, n_kv, page, d, n_seq=3, max_pages=5):
    n = n_seq * max_pages
    table = torch.randperm(n + 2, generator=torch.Generator().manual_seed(9))[:n].int().view(n_seq, max_pages).to(DEV)
    c = wl.new_cache(n + 2, n_kv, page, d, table, fmt)
    for t in (c.k, c.v):
        t.view(torch.uint8).fill_(0x55)
    for t in (c.k_scale, c.v_scale):
        if t is not None:
            t.fill_(0.25)
    return c


WRITES = [(BF, BF, 1, 16, 256, 1, 4), (BF, I8, 8, 64, 128, 70, 32), (BF, E4, 3, 32, 96, 9, 6), (F32, F32, 2, 16, 64, 33, 2),
          (F32, I8, 1, 128, 16, 5, 0), (F32, E4, 2, 16, 256, 240, 4), (BF, E4, 1, 1024, 256, 40, 4), (BF, I8, 5, 16, 48, 2, 5)]


@pytest.mark.parametrize("case", range(len(WRITES)))
def test_write_and_read(wl, case):
    dtype, fmt, n_kv, page, d, T, nq = WRITES[case]
    print(f"cache write {WRITES[case]}", flush=True)
    c = make(wl, fmt, n_kv, page, d)
    seq, slot = place(c, T, case)
    qkv = draw(1, T, (nq + 2 * n_kv) * d, dtype=dtype)
    q, k, v = qkv.split([nq * d, n_kv * d, n_kv * d], 1)
    freq, _ = wl.rope_frequencies(d if d % 16 == 0 else d - 8, device=DEV)
    wk, wq = draw(2, d, dtype=dtype, std=0.2), draw(3, d, dtype=dtype, std=0.2)
    others = c.k.view(torch.uint8).clone()
    qo = wl.wl_cache_write(c, k, v, seq, slot, q=q if nq else None, rope=wl.Rope(freq), k_norm=wk,
                           q_norm=wq if nq else None, offset=1.0)
    kr, vr = wl.wl_cache_read(c, seq, slot, dtype=dtype)
    torch.cuda.synchronize()
    rk, mk = ref.rotate(k, d, slot, freq, 1.0, False, wk, 1e-6, 1.0)
    slack = (ref.CHAIN + 16) * ref.EPS32 * mk
    if nq:
        rq, mq = ref.rotate(q, d, slot, freq, 1.0, False, wq, 1e-6, 1.0)
        ref.assert_near(qo, rq, (ref.CHAIN + 16) * ref.EPS32 * mq, "q")
    if fmt in (BF, F32):
        ref.assert_near(kr, rk, slack, "k")
        assert torch.equal(vr, v)
    else:
        # a code is off by at most half a step of its format
        most = rk.view(T, n_kv, d).abs().amax(-1, keepdim=True).expand(-1, -1, d).flatten(1)
        step = most / 127 / 2 if fmt == I8 else torch.maximum(rk.abs() * 2 ** -4, most / 448 * 2 ** -10)
        ref.assert_near(kr, rk, slack + (step + 2 * slack) * (1 + 2 ** -6), "k")
        # V is stored as it is: codes and scales are the definition's
        want, scale = ref.codes(v.view(T, n_kv, d), fmt)
        page_id = c.table.cpu()[seq.cpu().long(), slot.cpu().long() // page].long()
        off = slot.cpu().long() % page
        pool = c.v.cpu()
        have = pool.view(torch.uint8)[page_id, :, off].view(fmt).float().double()
        assert torch.equal(have, want)
        assert torch.equal(c.v_scale.cpu()[page_id, :, off].double(), scale.float().double())
        ref.assert_near(vr, (want * scale.float().double()[..., None]).flatten(1), 2 * ref.EPS32 * v.cpu().double().abs(), "v")
    # nothing else of the cache was written
    mask = torch.ones(c.k.shape[:3], dtype=torch.bool, device=DEV)
    mask[c.table[seq.long(), slot.long() // page].long(), :, slot.long() % page] = False
    assert torch.equal(c.k.view(torch.uint8).view(*c.k.shape[:3], -1)[mask], others.view(*c.k.shape[:3], -1)[mask])


def test_ties_go_to_the_even_code(wl):
    """Rows of bf16 values that lie exactly between two codes."""
    for fmt, top in ((I8, 127.0), (E4, 448.0)):
        d = 16
        c = make(wl, fmt, 1, 16, d)
        rows = []
        for most in (top, top / 2, 2 * top, top * 2 ** -90, top * 2 ** 90):
            half = (torch.arange(d, dtype=torch.float64) + 0.5) if fmt == I8 else 16 + (torch.arange(d, dtype=torch.float64) % 8) * 2 + 1
            half[0] = top
            rows.append(half * most / top * torch.where(torch.arange(d) % 2 == 0, 1, -1))
        v = torch.stack(rows).to(BF).to(DEV)
        n = len(rows)
        seq, slot = ints([0] * n), ints(list(range(n)))
        wl.wl_cache_write(c, v, v, seq, slot)
        torch.cuda.synchronize()
        want, _ = ref.codes(v, fmt)
        page = int(c.table[0, 0])
        assert torch.equal(c.v.cpu().view(torch.uint8)[page, 0, :n].view(fmt).float().double(), want)


def test_rows_of_zeros_infinities_and_nan(wl):
    for fmt in (I8, E4):
        c = make(wl, fmt, 1, 16, 32)
        v = draw(1, 4, 32)
        v[0], v[1, 3], v[2, 4] = 0, float("inf"), float("nan")
        seq, slot = ints([1] * 4), ints([0, 1, 2, 3])
        wl.wl_cache_write(c, v, v, seq, slot)
        k, w = wl.wl_cache_read(c, seq, slot)
        torch.cuda.synchronize()
        for t in (k, w):
            assert (t[0] == 0).all() and torch.isnan(t[1]).all() and torch.isnan(t[2]).all() and torch.isfinite(t[3]).all()


def test_padding_and_places_that_are_none(wl):
    T, d, n_kv = 8, 64, 2
    c = make(wl, BF, n_kv, 16, d, n_seq=2, max_pages=2)
    c.table[1, 1] = -1
    c.table[1, 0] = c.k.shape[0]                      # no page either
    seq, slot = ints([0, -1, 2, 0, 0, 1, 1, 0]), ints([3, 0, 1, -5, 32, 20, 2, 31])
    k, v, q = draw(1, T, n_kv * d), draw(2, T, n_kv * d), draw(3, T, 4 * d)
    before = c.k.clone(), c.v.clone()
    qo = torch.full_like(q, 7.0)
    wl.wl_cache_write(c, k, v, seq, slot, q=q, q_out=qo)
    ko, vo = torch.full_like(k, 5.0), torch.full_like(v, 5.0)
    wl.wl_cache_read(c, seq, slot, k_out=ko, v_out=vo)
    torch.cuda.synchronize()
    skipped = torch.tensor([False, True, True] + [False] * 5, device=DEV)
    assert (qo[skipped] == 7).all() and torch.equal(qo[~skipped], q[~skipped])
    stored = torch.tensor([True, False, False, False, False, False, False, True], device=DEV)
    assert torch.equal(ko[stored], k[stored]) and torch.equal(vo[stored], v[stored])
    assert (ko[~stored] == 5).all() and (vo[~stored] == 5).all()
    changed = (c.k != before[0]).flatten(3).any(-1).any(1)
    page = c.table[0].long()
    assert int(changed.sum()) == 2 and changed[page[0], 3] and changed[page[1], 15]


def test_far_pages_of_a_large_pool(wl):
    """Element offsets past 2^31 and 2^32."""
    page, n_kv, d = 1024, 8, 256
    n_pages = 2200                                       # 4.6e9 one-byte elements in each pool
    table = ints([[n_pages - 1, 0], [1500, 1024]])
    c = wl.new_cache(n_pages, n_kv, page, d, table, I8)
    seq, slot = ints([0, 0, 1, 1]), ints([1023, 1024, 0, 2047])
    v = draw(1, 4, n_kv * d)
    wl.wl_cache_write(c, v, v, seq, slot)
    k, w = wl.wl_cache_read(c, seq, slot)
    torch.cuda.synchronize()
    for s, p, o in ((0, n_pages - 1, 1023), (1, 0, 0), (2, 1500, 0), (3, 1024, 1023)):
        assert torch.equal((c.k[p, :, o].float() * c.k_scale[p, :, o][:, None]).flatten().to(BF), k[s])
        most = v[s].float().view(n_kv, d).abs().amax(1, keepdim=True).expand(-1, d).flatten()
        assert ((w[s].float() - v[s].float()).abs() <= most / 127 / 2 * 1.01 + v[s].float().abs() / 128).all()


def test_empty_refusals_and_replay(wl):
    c = make(wl, E4, 2, 16, 64)
    k = draw(1, 4, 128)
    seq, slot = place(c, 4, 1)
    assert wl.wl_cache_write(c, k[:0], k[:0], seq[:0], slot[:0]) is None
    assert wl.wl_cache_read(c, seq[:0], slot[:0])[0].shape == (0, 128)
    freq, _ = wl.rope_frequencies(64, device=DEV)
    for bad in (dict(seq=seq[:3]), dict(seq=seq.long()), dict(k=k[:, :64]), dict(v=k.float()), dict(rope=wl.Rope(freq.float()))):
        kw = dict(k=k, v=k, seq=seq, slot=slot) | bad
        with pytest.raises(ValueError):
            wl.wl_cache_write(c, **kw)
    with pytest.raises(wl.WlError):
        wl.wl_cache_write(c, k, k, seq, slot, rope=wl.Rope(freq[:3]))
    with pytest.raises(wl.WlError):
        wl.wl_rope(k, None, None, wl.Rope(freq), 64)
    call = wl.cache_write_call(c, k, k, seq, slot, q=k, rope=wl.Rope(freq))
    read = wl.cache_read_call(c, seq, slot)
    call.launch(), read.launch()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call.launch(), read.launch()
    for seed in (3, 4, 5):
        k.copy_(draw(seed, 4, 128))
        slot.copy_((slot + 1) % 80)
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (call.out, *read.out)]
        call.launch(), read.launch()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (call.out, *read.out)))
