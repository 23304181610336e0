"""Latent attention of many (token, head) rows, and by every kernel over keys whose scores rise along the
sequence, against the definition in 64 bits. max_kv is far above the lengths, as a recorded step has it."""
from __future__ import annotations

import random

import pytest
import torch

from tests import layer_ref, serve_ref
from tests.test_gpu_latent import BF, E4M3, F32, Batch, i32, wl  # noqa: F401

pytestmark = pytest.mark.gpu
FAR = 1 << 17   # keys, far above all lengths here


SHAPES = [(512, 64, 128, 128), (512, 32, 64, 96), (256, 64, 64, 64), (256, 32, 96, 32), (128, 64, 64, 64)]


@pytest.mark.parametrize("fmt", [BF, E4M3])
@pytest.mark.parametrize("L,R,N,V", SHAPES)
def test_causal(wl, fmt, L, R, N, V):  # noqa: F811
    """Tiles that are full, that end inside a wave and that have one row; sequences of no rows and of few keys."""
    for k, (H, seqs) in enumerate(((120, [(70, 1), (0, 1), (300, 1)]), (43, [(500, 3), (0, 0), (31, 1), (5, 6)]), (12, [(0, 43), (90, 11)]))):
        b = Batch(wl, seqs, H, L, R, N, V, fmt, page=(16, 32, 64)[k], seed=L + k, gap=1, tail=2)
        b.check(wl, f"{H} heads", max_kv=FAR, form="absorbed")


@pytest.mark.parametrize("fmt", [BF, E4M3])
@pytest.mark.parametrize("L", [256, 512])
@pytest.mark.parametrize("window", [0, 1, 40])
def test_trees_windows_and_full(wl, fmt, L, window):  # noqa: F811
    b = Batch(wl, [(80, 9), (0, 40), (300, 1), (33, 24)], 11, L, 64, 64, 64, fmt, page=32, seed=3)
    tree, pos = b.trees()
    kw = dict(max_kv=FAR, form="absorbed")
    b.check(wl, "tree", tree=tree, q_pos=pos, window=window, **kw)
    b.check(wl, "tree without positions", tree=tree, window=window, **kw)
    if not window:
        b.check(wl, "full", mask="full", **kw)


@pytest.mark.parametrize("fmt", [BF, E4M3])
def test_causal_windows(wl, fmt):  # noqa: F811
    """Of 64 sequences, and of 70, whose pieces lanes do not plan."""
    rng = random.Random(5)
    for n_seq, window in ((64, 40), (70, 17)):
        b = Batch(wl, [(rng.choice((0, 20, 150)), rng.choice((0, 1, 3, 7))) for _ in range(n_seq)], 64, 512, 64, 64, 64, fmt, page=32, seed=n_seq, tail=500)
        b.check(wl, f"{n_seq} sequences", max_q=max(b.rows) + 1, max_kv=FAR, window=window, form="absorbed")


@pytest.mark.parametrize("fmt", [BF, E4M3])
@pytest.mark.parametrize("L", [256, 512])
def test_without_weights(wl, fmt, L):  # noqa: F811
    b = Batch(wl, [(90, 3), (500, 1), (0, 5)], 30, L, 64, fmt=fmt, weights=False, seed=4, gap=1)
    b.check(wl, "latent", max_kv=FAR)


@pytest.mark.parametrize("fmt", [BF, E4M3])
def test_more_sequences_than_lanes(wl, fmt):  # noqa: F811
    rng = random.Random(8)
    b = Batch(wl, [(rng.randrange(0, 500), rng.choice((0, 1, 2))) for _ in range(66)], 40, 512, 64, 64, 64, fmt, seed=8, page=32)
    b.check(wl, "66 sequences", max_kv=5000, form="absorbed")


@pytest.mark.parametrize("fmt", [BF, E4M3])
@pytest.mark.parametrize("scale", [0.0, -0.1])
def test_scales(wl, fmt, scale):  # noqa: F811
    b = Batch(wl, [(150, 2), (40, 1)], 50, fmt=fmt, seed=13)
    b.scale = scale
    b.check(wl, f"scale {scale}", max_kv=FAR, form="absorbed")


@pytest.mark.parametrize("fmt", [BF, E4M3])
@pytest.mark.parametrize("L", [256, 512])
def test_missing_pages(wl, fmt, L):  # noqa: F811
    b = Batch(wl, [(100, 2), (40, 1)], 40, L, 64, 64, 64, fmt, seed=10)
    t = b.cache.table
    t[0, 2], t[0, 4], t[1, 0], t[1, 1], t[1, 2] = -1, 1 << 20, -5, 1 << 30, -1
    o = b.check(wl, "missing pages", max_kv=b.cache.table.shape[1] * 16, form="absorbed")
    assert (o[2] == 0).all()
    wide = torch.full((2, FAR // 16), -1, dtype=torch.int32, device=t.device)
    wide[:, :t.shape[1]] = t
    b.cache = wl.LatentCache(b.cache.rows, wide, L, 64, b.cache.scale)
    o = b.check(wl, "missing pages, far max_kv", max_kv=FAR, form="absorbed")
    assert (o[2] == 0).all()


@pytest.mark.parametrize("fmt", [BF, E4M3])
@pytest.mark.parametrize("L", [256, 512])
def test_unseen_keys_have_no_influence(wl, fmt, L):  # noqa: F811
    """NaN and infinities in rows that no query sees, or that some do not see: trees, whose new tokens see one another
    or not, under a window."""
    b = Batch(wl, [(70, 4), (33, 1)], 40, L, 64, 64, 64, fmt, seed=11)
    tree = i32([[1], [3], [5], [9], [1]])     # tokens 1, 2 and 3 follow token 0
    kw = dict(tree=tree, window=20, max_kv=FAR, form="absorbed")
    clean = b.check(wl, "clean", **kw)
    ref, slack = serve_ref.latent_attention(b.q, b.cache, b.w, i32(b.starts), i32(b.lens), b.scale, tree=tree, window=20)
    rows = b.cache.rows
    as_bad = (lambda r: r.fill_(0x7F)) if fmt == E4M3 else (lambda r: r.fill_(float("nan")))
    last = [b.cache.table[s, (n - 1) // 16].item() for s, n in enumerate(b.lens)]
    for s, n in enumerate(b.lens):
        as_bad(rows[last[s], (n - 1) % 16 + 1:])            # behind the last key
    as_bad(rows[b.cache.table[0, 0].item()])                # below the window
    if b.cache.scale is not None:
        b.cache.scale[b.cache.table[0, 0].item()] = float("inf")
    assert torch.equal(b.run(wl, **kw), clean)
    as_bad(rows[b.cache.table[0, 72 // 16].item(), 72 % 16])  # token 2's key, which tokens 0, 1 and 3 do not see
    o = b.run(wl, **kw)
    assert o[2].isnan().all() and torch.equal(o[4:], clean[4:])
    for i in (0, 1, 3):                                     # summed anew, in another order
        layer_ref.assert_near(o[i], ref[i], slack[i], f"row {i}")


@pytest.mark.parametrize("fmt", [BF, E4M3])
def test_captured_and_replayed_over_changing_lengths(wl, fmt):  # noqa: F811
    b = Batch(wl, [(900, 2), (37, 1), (400, 3)], 48, fmt=fmt, page=32, seed=16, tail=3)
    starts, lens = i32(b.starts), i32(b.lens)
    call = wl.latent_attention_call(b.q, b.cache, b.w, starts, lens, 3, FAR, b.scale)
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
        wl.wl_latent_attention(b.q, b.cache, b.w, starts, lens, 3, FAR, b.scale, o=o)
        assert torch.equal(call.out, o)
        want, slack = serve_ref.latent_attention(b.q, b.cache, b.w, starts, lens, b.scale, max_q=3)
        mine = ~want[:, 0].isnan()
        layer_ref.assert_near(o[mine.to(o.device)], want[mine], slack[mine], f"replay {k}")
        assert (o[~mine.to(o.device)] == 5.0).all()


# ---- scores that rise along the keys -----------------------------------------------------


def rising(b, per_tile):
    """Key j of every sequence adds per_tile j / 32 to a score (a power of two), times a factor of -1 to 1 of the
    row's own: j = 128 a + c in two elements of the rotated key, which bf16 holds exactly, as 128 a and c.
    A running reference that moves when a score passes it by 2^8 moves again and again, at other keys in
    every row, while most of the weight lies in the last few tiles; in rows whose scores fall, never."""
    page, L, R = b.cache.rows.shape[1], b.cache.latent, b.cache.rot
    for s, n in enumerate(b.lens):
        j = torch.arange(n)
        page_of = b.cache.table.cpu()[s][j // page].long()
        key = torch.stack((j // 128 * 128, j % 128), 1)
        if b.cache.rows.dtype == torch.uint8:
            host = b.cache.rows.cpu()
            host[page_of, j % page, L:L + 4] = key.to(BF).view(torch.uint8)
            b.cache.rows.copy_(host)
        else:
            host = b.cache.rows.cpu()
            host[page_of, j % page, L:L + 2] = key.to(host.dtype)
            b.cache.rows.copy_(host)
    step = per_tile / 32 / 1.4426950408889634 / b.scale
    g = torch.Generator().manual_seed(99)
    factor = torch.tensor([1.0, 0.75, 0.5, -1.0, 0.0])[torch.randint(5, (b.T, b.H), generator=g)]
    q = b.q.view(b.T, b.H, -1)
    q[:, :, q.shape[2] - R:][:, :, :2] = (factor * step)[:, :, None].to(q.dtype).to(q.device)


# (token, head) rows of a sequence: 16, 32, 64 and more, each in the kernels that take so many
@pytest.mark.parametrize("fmt", [BF, E4M3, F32])
@pytest.mark.parametrize("L", [128, 256, 512])
@pytest.mark.parametrize("H,seqs,max_kv", [
    (8, [(1500, 2), (300, 1)], None), (14, [(1400, 2), (700, 1)], None), (30, [(1600, 2), (90, 1)], None), (64, [(1500, 2), (400, 1)], None),
    (64, [(1500, 2), (400, 1)], FAR), (33, [(900, 5), (1700, 3), (40, 1)], FAR)])
@pytest.mark.parametrize("weights", [True, False])
def test_rising_scores(wl, fmt, L, H, seqs, max_kv, weights):  # noqa: F811
    b = Batch(wl, seqs, H, L, 64, 64, 64, fmt, page=64, seed=L + H, weights=weights)
    rising(b, 3.0)
    b.check(wl, "rising", max_kv=max_kv, form="absorbed")


@pytest.mark.parametrize("n_seq", [3, 70])
@pytest.mark.parametrize("fmt", [BF, E4M3, F32])
def test_rising_scores_of_many_sequences(wl, fmt, n_seq):  # noqa: F811
    """Pieces of the keys whose references differ by far, joined."""
    rng = random.Random(n_seq)
    b = Batch(wl, [(rng.choice((100, 2500) if n_seq < 64 else (30, 600)), 1) for _ in range(n_seq)], 40, 256, 64, 64, 64, fmt, page=64, seed=n_seq)
    rising(b, 2.0)
    b.check(wl, "rising", max_kv=4096, form="absorbed")


@pytest.mark.parametrize("D,L", [(64, 256), (128, 512)])
def test_rising_scores_expanded(wl, D, L):  # noqa: F811
    b = Batch(wl, [(1500, 140), (300, 33)], 3, L, 64, D, D, page=64, seed=D)
    rising(b, 3.0)
    b.check(wl, "rising", form="expanded", expanded=True)
