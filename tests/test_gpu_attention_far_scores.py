"""Scores far beyond any that a model has, up to 2^100, of finite queries and keys: the largest takes all the
weight, in wl_attention and wl_latent_attention."""
from __future__ import annotations

import pytest
import torch

from tests import layer_ref, serve_ref
from tests.layer_ref import f64
from tests.test_gpu_attention import BF, E4, F32, I8
from tests.test_gpu_attention import Batch as Heads
from tests.test_gpu_latent import Batch, i32, wl  # noqa: F401

pytestmark = pytest.mark.gpu


def near(o, ref, what):
    """Outputs are one value vector each, in its own rounding (and that of what it is formed from)."""
    assert torch.isfinite(o).all(), what
    assert float(((f64(o) - ref).norm(dim=1) / ref.norm(dim=1)).max()) <= 2.0 ** -7, what


@pytest.mark.parametrize("fmt", [BF, E4, F32])
@pytest.mark.parametrize("H,rows", [(5, 3), (13, 2), (16, 9), (3, 140)])
@pytest.mark.parametrize("size", [2.0 ** 35, -2.0 ** 60, 2.0 ** 100])
def test_latent(wl, fmt, H, rows, size):  # noqa: F811
    b = Batch(wl, [(200, rows), (20, 1)], H, 256, 64, 64, 64, fmt, page=32, seed=H)
    b.q *= abs(size)
    b.scale = b.scale if size > 0 else -b.scale
    for form in ("absorbed", "expanded") if fmt == BF else ("absorbed",):
        o = b.run(wl, form=form)
        ref, _ = serve_ref.latent_attention(b.q, b.cache, b.w, i32(b.starts), i32(b.lens), b.scale, expanded=form == "expanded")
        near(o.view(-1, 64), ref.view(-1, 64), form)


@pytest.mark.parametrize("fmt", [BF, E4, I8, F32])
@pytest.mark.parametrize("rows", [[1, 1], [20, 3], [150, 40]])
@pytest.mark.parametrize("size", [2.0 ** 35, 2.0 ** 100])
def test_heads(wl, fmt, rows, size):  # noqa: F811
    b = Heads(wl, [200, 20], rows, 8, 2, 128, 16, fmt, seed=rows[0])
    b.q = b.q * size
    o = b.run(wl)
    ref, _ = layer_ref.attention(b.q, b.cache, b.q_start, b.kv_len, b.scale)
    near(o.view(-1, 128), ref.view(-1, 128), "heads")
