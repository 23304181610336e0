"""A latent cache whose pool passes 2^32 bytes (and 2^31 elements): its last pages give the same as those of a
small pool, in every kernel."""
from __future__ import annotations

import pytest
import torch

from tests.test_gpu_latent import BF, DEV, E4M3, F32, Batch, i32, wl  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [BF, E4M3, F32])
def test_far_pages(wl, fmt):  # noqa: F811
    b = Batch(wl, [(1500, 3), (700, 1)], 20, fmt=fmt, page=1024, seed=1)
    small, n = b.cache, b.cache.rows.shape[0]
    pages = max((1 << 32) // small.rows.element_size(), 1 << 31) // small.rows[0].numel() + n + 1
    rows = torch.empty(pages, *small.rows.shape[1:], dtype=small.rows.dtype, device=DEV)
    rows[-n:] = small.rows
    scale = None
    if small.scale is not None:
        scale = torch.empty(pages, small.scale.shape[1], device=DEV)
        scale[-n:] = small.scale
    table = torch.where(small.table >= 0, small.table + (pages - n), small.table).to(torch.int32)
    far = wl.LatentCache(rows, table, small.latent, small.rot, scale)
    # written and read back
    g = torch.Generator().manual_seed(2)
    T = 70
    c = torch.randn(T, small.latent + small.rot, generator=g).to(small.dtype).to(DEV)
    seq, slot = i32([t % 2 for t in range(T)]), i32([9 * t for t in range(T)])
    back = []
    for cache in (small, far):
        wl.wl_latent_write(cache, c, seq, slot)
        back.append(wl.wl_latent_read(cache, seq, slot))
    assert torch.equal(*back) and torch.equal(rows[-n:], small.rows)
    # attention: few rows, more of them, many, without weights, expanded, and a row done again key by key
    outs = []
    for cache in (small, far):
        b.cache, o = cache, []
        for heads in (4, 10, 20):
            q = b.q.view(b.T, 20, -1)[:, :heads].flatten(1).contiguous()
            o.append(wl.wl_latent_attention(q, cache, b.w[:heads].contiguous(), i32(b.starts), i32(b.lens), 3, 1503, b.scale, form="absorbed"))
        latent = torch.randn(b.T, 20 * (small.latent + small.rot), generator=torch.Generator().manual_seed(3)).to(small.dtype).to(DEV)
        o.append(wl.wl_latent_attention(latent, cache, None, i32(b.starts), i32(b.lens), 3, 1503, 0.05))
        if fmt == BF:
            o.append(b.run(wl, form="expanded"))
        page, off = cache.table[0, 1].item(), 1502 - 1024      # the last key: its query's row alone is NaN
        kept = cache.rows[page, off].clone()
        cache.rows[page, off].fill_(0x7F if fmt == E4M3 else float("inf"))
        o.append(b.run(wl, form="absorbed"))
        assert o[-1][2].isnan().any() and not o[-1][[0, 1, 3]].isnan().any()
        o[-1] = o[-1].nan_to_num(7.0)
        cache.rows[page, off] = kept
        outs.append(o)
    for x, y in zip(*outs):
        assert torch.equal(x, y)
