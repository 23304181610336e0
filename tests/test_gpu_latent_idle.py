"""Latent attention where workgroups have no keys: sequences of none, pieces behind a sequence's
end, windows that leave pieces empty. In the kernels whose waves take keys of their own these join
nothing, beside workgroups that do."""
from __future__ import annotations

import random

import pytest
import torch

from tests.test_gpu_latent import BF, E4M3, F32, Batch, wl  # noqa: F401

pytestmark = pytest.mark.gpu
FORMATS = [BF, E4M3, F32]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("L", [128, 256, 512])
@pytest.mark.parametrize("H,weights", [(8, True), (5, False), (16, True), (12, False)])
def test_pieces_without_keys(wl, fmt, L, H, weights):  # noqa: F811
    """More sequences than lanes, of up to 2 tokens each (16 rows of 8 and 5 heads, 17 to 32 of 16 and
    12), whose keys are divided by a max_kv far above most of them."""
    rng = random.Random(L + H)
    seqs = [(rng.choice((0, 0, 3, 40, 700)), rng.choice((0, 1, 2))) for _ in range(66)]
    b = Batch(wl, seqs, H, L, 64, 64, 64, fmt, page=32, seed=L + H, weights=weights, gap=1, tail=3)
    first = b.check(wl, "causal", max_kv=5000)
    for _ in range(10):
        assert torch.equal(b.run(wl, max_kv=5000), first)
    tree, pos = b.trees()
    b.check(wl, "tree", max_kv=5000, tree=tree, q_pos=pos, window=25)
    b.check(wl, "window", max_kv=5000, window=25)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("H,weights", [(6, True), (6, False), (20, True)])
def test_sequences_without_keys(wl, fmt, H, weights):  # noqa: F811
    """Up to 64 sequences, whose pieces follow from their lengths: rows over no key at all are zeros."""
    b = Batch(wl, [(0, 1), (900, 1), (0, 1), (30, 1)], H, 512, 64, 64, 64, fmt, page=32, seed=H, weights=weights, tail=1)
    b.lens = [0, 901, -4, 31]
    o = b.check(wl, "idle sequences", max_kv=1000)
    assert (o[0] == 0).all() and (o[2] == 0).all() and (o[1] != 0).any()
    b.lens = [0, 0, 0, 0]
    assert (b.check(wl, "no keys", max_kv=1000)[:4] == 0).all()
