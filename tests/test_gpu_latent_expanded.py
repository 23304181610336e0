"""Latent attention in the expanded form against its definition in 64 bits, and against the
absorbed form."""
from __future__ import annotations

import random

import pytest
import torch

from tests import layer_ref, serve_ref
from tests.test_gpu_latent import BF, DEV, E4M3, Batch, i32, wl  # noqa: F401

pytestmark = pytest.mark.gpu


def run(b, wl, what, **kw):
    return b.check(wl, what, form="expanded", expanded=True, **kw)


@pytest.mark.parametrize("L,R,D", [(512, 64, 128), (256, 32, 64), (128, 64, 128), (512, 32, 64)])
@pytest.mark.parametrize("H,seqs", [(1, [(0, 1)]), (3, [(100, 130), (0, 0), (0, 37), (31, 1), (5, 128)]), (8, [(500, 20), (127, 129)])])
def test_causal(wl, L, R, D, H, seqs):  # noqa: F811
    run(Batch(wl, seqs, H, L, R, D, D, seed=H + D, gap=3, tail=2), wl, "causal")


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("window", [0, 1, 50])
def test_masks(wl, page, window):  # noqa: F811
    b = Batch(wl, [(300, 60), (0, 33), (140, 9)], 4, page=page, seed=3)
    tree, pos = b.trees()
    run(b, wl, "tree", tree=tree, q_pos=pos, window=window)
    run(b, wl, "causal", window=window)
    if not window:
        run(b, wl, "full", mask="full")


def test_limits_of_rows_and_keys(wl):  # noqa: F811
    b = Batch(wl, [(60, 9), (10, 4)], 6, seed=9, gap=1)
    run(b, wl, "max_q", max_q=5)
    run(b, wl, "max_kv", max_kv=37)
    run(b, wl, "no keys", max_kv=0)
    b.lens = [3, 1000]
    o = run(b, wl, "short and long", max_kv=1000)
    assert (o[1:7] == 0).all()


def test_missing_pages(wl):  # noqa: F811
    b = Batch(wl, [(100, 20), (40, 1)], 8, seed=10)
    t = b.cache.table
    t[0, 2], t[0, 4], t[1, 0], t[1, 1], t[1, 2] = -1, 1 << 20, -5, 1 << 30, -1
    o = run(b, wl, "missing pages")
    assert (o[20] == 0).all()


def test_unseen_keys_have_no_influence(wl):  # noqa: F811
    b = Batch(wl, [(150, 4), (33, 1)], 5, seed=11)
    clean = run(b, wl, "clean", window=20)
    ref, slack = serve_ref.latent_attention(b.q, b.cache, b.w, i32(b.starts), i32(b.lens), b.scale, window=20, expanded=True)
    rows, bad = b.cache.rows, float("nan")
    last = [b.cache.table[s, (n - 1) // 16].item() for s, n in enumerate(b.lens)]
    for s, n in enumerate(b.lens):
        rows[last[s], (n - 1) % 16 + 1:] = bad              # behind the last key
    rows[b.cache.table[0, 0].item()] = bad                  # below the window, and below the first key formed
    rows[b.cache.table[0, 8].item(), :2] = -float("inf")    # below the window, among the keys formed
    layer_ref.assert_near(b.run(wl, window=20, form="expanded"), ref, slack, "unseen")
    rows[last[0], (b.lens[0] - 1) % 16] = bad               # seen by the last query of sequence 0 alone
    o = b.run(wl, window=20, form="expanded")
    assert o[3].isnan().all() and torch.equal(o[4:], clean[4:])
    layer_ref.assert_near(o[:3], ref[:3], slack[:3], "rows beside one that sees it")


def test_heads_in_groups(wl):  # noqa: F811
    """Room for more keys than the workspace takes of all heads at once."""
    b = Batch(wl, [(90, 40), (0, 70)], 12, seed=12)
    n, wide = b.cache.table.shape[1], torch.full((2, 65536), -1, dtype=torch.int32, device=DEV)
    wide[:, :n] = b.cache.table
    ref = b.run(wl, form="expanded")
    far = wl.LatentCache(b.cache.rows, wide, 512, 64)
    args = (b.q, far, b.w, i32(b.starts), i32(b.lens), 70, 1 << 20, b.scale)
    call = wl.latent_attention_call(*args, form="expanded")
    need = wl.lib.wl_latent_attention_workspace_bytes(call.args)
    assert (1 << 32) < need <= (8 << 30) + wl.SYNC_BYTES + 4096
    assert torch.equal(call.launch(), ref)
    call = None
    wl.WORKSPACE._bufs.clear()
    torch.cuda.empty_cache()


def test_chosen_for_prompts(wl):  # noqa: F811
    """Left to choose, a prompt takes the expanded form's workspace, a token and a code cache the absorbed one's."""
    b = Batch(wl, [(10, 300)], 64, seed=13)
    need = lambda form, max_q: wl.lib.wl_latent_attention_workspace_bytes(  # noqa: E731
        wl.latent_attention_call(b.q, b.cache, b.w, i32(b.starts), i32(b.lens), max_q, 310, b.scale, form=form).args)
    assert need("auto", 300) == need("expanded", 300) != need("absorbed", 300)
    assert need("auto", 4) == need("absorbed", 4)
    o = b.run(wl)
    assert torch.equal(o, b.run(wl, form="expanded"))
    a = b.run(wl, form="absorbed")
    assert float((o.float() - a.float()).norm() / a.float().norm()) <= 2 * serve_ref.REL_BF16
    c = Batch(wl, [(10, 300)], 64, fmt=E4M3, seed=13)
    assert torch.equal(c.run(wl), c.run(wl, form="absorbed"))
    with pytest.raises(wl.WlError):
        c.run(wl, form="expanded")


def test_long_prompt(wl):  # noqa: F811
    """Every row of a prompt of several tiles, of a few heads."""
    rng = random.Random(1)
    b = Batch(wl, [(700, 500), (3, 260 + rng.randrange(8))], 2, page=64, seed=14)
    run(b, wl, "prompt")


def test_repeatable_and_captured(wl):  # noqa: F811
    b = Batch(wl, [(100, 200), (30, 250)], 16, seed=15)
    first = b.run(wl, form="expanded")
    for _ in range(10):
        assert torch.equal(b.run(wl, form="expanded"), first)
    call = wl.latent_attention_call(b.q, b.cache, b.w, i32(b.starts), i32(b.lens), 250, 300, b.scale, form="expanded")
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        call.launch()
    torch.cuda.current_stream().wait_stream(s)
    for k in range(4):
        b.q.copy_(torch.randn(b.q.shape, generator=torch.Generator().manual_seed(k)))
        g.replay()
        assert torch.equal(call.out, b.run(wl, form="expanded", max_q=250, max_kv=300))
