"""wl_attention in calls of more than 32 tiles of 64 query rows: weights as single bf16
values, 32 rows per wave under a large max_kv (eight waves at 129 to 256 rows over int8
and e4m3), 16 under a tight one. The tests of small calls, in batches with further
sequences that have nothing to do."""
from __future__ import annotations

import pytest
import torch

import test_gpu_attention as small
from test_gpu_attention import BF, CASES, E4, F32, I8, TREES, wl  # noqa: F401

pytestmark = pytest.mark.gpu


# Idle sequences: with those of a test more than 32, so as many tiles at least; above 64
# of them the keys are divided by max_kv.
@pytest.fixture(params=[(40, False), (40, True), (70, True)], ids=["tight", "far", "far-unplanned"])
def many(request, monkeypatch):
    base = small.Batch
    idle, limit = request.param

    class Many(base):
        far = limit

        def __init__(self, wl, ctx, rows, *args, **kw):
            super().__init__(wl, list(ctx) + [0] * idle, list(rows) + [0] * idle, *args, **kw)

    monkeypatch.setattr(small, "Batch", Many)


@pytest.mark.parametrize("fmt", [BF, I8, E4])
@pytest.mark.parametrize("case", [c for c in range(len(CASES)) if max(CASES[c][1]) * CASES[c][2] // CASES[c][3] > 64])
def test_causal(wl, many, case, fmt):  # noqa: F811
    small.test_causal(wl, case, fmt)


@pytest.mark.parametrize("fmt", [BF, I8, E4])
@pytest.mark.parametrize("case", [c for c in range(len(TREES)) if max(TREES[c][1]) * TREES[c][2] // TREES[c][3] > 64])
def test_tree(wl, many, case, fmt):  # noqa: F811
    small.test_tree(wl, case, fmt)


@pytest.mark.parametrize("fmt", [BF, I8, E4])
@pytest.mark.parametrize("d, rows, hq", [(64, [70, 1, 64], 4), (128, [24, 25, 3], 8), (256, [64, 33, 0], 3), (256, [90, 30, 100], 2),
                                         (96, [256, 17, 129], 1), (256, [48, 31, 35], 4), (256, [40, 200, 16], 1),
                                         (64, [40, 9, 33], 4), (128, [150, 40, 130], 1)])
def test_shares_of_the_rows(wl, many, d, rows, hq, fmt):  # noqa: F811
    small.test_shares_of_the_rows(wl, None, d, rows, hq, fmt)


@pytest.mark.parametrize("fmt", [BF, I8, E4])
def test_unseen_and_absent_keys(wl, many, fmt):  # noqa: F811
    for rows in ([150, 40], [100, 3], [60, 60]):
        small.test_nan_and_infinity_of_unseen_keys(wl, fmt, rows)
    small.test_pages_that_are_none(wl, fmt)


@pytest.mark.parametrize("fmt", [BF, I8, E4])
@pytest.mark.parametrize("scale", [0.0, -0.3, 1.5])
def test_scales(wl, many, scale, fmt):  # noqa: F811
    small.test_scales(wl, scale, fmt)


@pytest.mark.parametrize("fmt", [BF, I8, E4])
def test_queries_without_keys(wl, many, fmt):  # noqa: F811
    small.test_queries_without_keys(wl, fmt)


@pytest.mark.parametrize("fmt", [BF, I8, E4])
@pytest.mark.parametrize("d, rows", [(64, [160, 70, 1]), (128, [300, 2, 129]), (256, [200, 80, 256])])
def test_undivided(wl, many, d, rows, fmt):  # noqa: F811
    """Tiles enough for every place on the card: one piece each."""
    b = small.Batch(wl, [50, 3, 200], rows, 8, 8, d, 32, fmt, seed=42, extra=1)
    call = wl.attention_call(b.q, b.cache, b.q_start, b.kv_len, b.max_q, b.max_kv, 1.0)
    assert wl.lib.wl_attention_workspace_bytes(call.args) == 0, "divided"
    b.check(wl, window=90)
    words, pos = b.tree()
    b.check(wl, "tree", tree=words, q_pos=pos)


@pytest.mark.parametrize("fmt", [BF, I8, E4])
def test_visible_nan_through_the_join(wl, many, fmt):  # noqa: F811
    """70 tokens over divided keys, the newest key NaN: the last row alone sees it."""
    b = small.Batch(wl, [3000], [70], 4, 1, 128, 16, fmt, seed=41)
    assert wl.lib.wl_attention_workspace_bytes(
        wl.attention_call(b.q, b.cache, b.q_start, b.kv_len, b.max_q, b.max_kv, 1.0).args), "undivided"
    k = torch.full((1, 128), float("nan"), dtype=b.q.dtype, device=b.q.device)
    wl.wl_cache_write(b.cache, k, torch.ones_like(k), small.ints([0]), small.ints([3069]))
    o = b.run(wl)
    torch.cuda.synchronize()
    assert torch.isnan(o[69]).all() and torch.isfinite(o[:69]).all()
