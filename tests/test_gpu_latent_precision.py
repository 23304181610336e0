"""How far latent attention in bf16 is from its definition in 64 bits, against what its output's own
rounding costs.

A rounding to bf16 is off by up to half a step, uniformly: 2^-7 / sqrt(12) of a power of two in the root mean
square, times sqrt(E[1 / m^2]) = 0.74 for a mantissa m in [1, 2) of density 1 / (m ln 2), so 0.00166 of the
value. Roundings of random sign add up in squares: k of them, each of a factor of the output, come to sqrt(k)
of the output's own, which is what is measured here. A sum of 512 random squares or more scatters by less than
1 / sqrt(512) = 5 %."""
from __future__ import annotations

import pytest
import torch

from tests import serve_ref
from tests.layer_ref import f64
from tests.test_gpu_latent import BF, E4M3, Batch, i32, wl  # noqa: F401

pytestmark = pytest.mark.gpu
ONE, TWO = 1.1, 1.5     # roundings: the output's, and one of its factors (sqrt(2)); three come to 1.73


def off(wl, b, form="absorbed", max_kv=None, **kw):  # noqa: F811
    """Error of the outputs over the error of the definition rounded to bf16."""
    o = f64(b.run(wl, max_kv=max_kv, form=form, **kw))
    ref, _ = serve_ref.latent_attention(b.q, b.cache, b.w, i32(b.starts), i32(b.lens), b.scale, expanded=form == "expanded", **kw)
    mine = ~ref[:, 0].isnan()
    assert ref[mine].numel() >= 512
    return float((o[mine] - ref[mine]).norm() / (ref[mine].to(BF).double() - ref[mine]).norm())


def batch(wl, H, seqs, L, R, N, V, fmt, weights):  # noqa: F811
    return Batch(wl, seqs, H, L, R, N, V, fmt, page=64, seed=H + L, weights=weights)


SHAPES = [(512, 64, 128, 128), (512, 32, 64, 64), (256, 64, 64, 64), (128, 64, 96, 32)]
SHORT, LONG = [(30, 2), (9, 1)], [(3000, 2), (700, 1)]


@pytest.mark.parametrize("fmt", [BF, E4M3])
@pytest.mark.parametrize("L,R,N,V", SHAPES)
@pytest.mark.parametrize("seqs", [SHORT, LONG])
def test_few_rows(wl, fmt, L, R, N, V, seqs):  # noqa: F811
    """Up to 16 rows: queries, weights and outputs in the latent space keep fp32's precision, divided keys or not."""
    assert off(wl, batch(wl, 8, seqs, L, R, N, V, fmt, True)) <= ONE


@pytest.mark.parametrize("fmt", [BF, E4M3])
@pytest.mark.parametrize("L,R,N,V", SHAPES)
@pytest.mark.parametrize("H", [14, 30, 64])
@pytest.mark.parametrize("seqs", [[(30, 2), (9, 1)], [(300, 2), (200, 1)], [(3000, 2), (700, 1)]])
def test_more_rows(wl, fmt, L, R, N, V, H, seqs):  # noqa: F811
    """28, 60 and 128 rows: the output's is the only rounding to bf16."""
    assert off(wl, batch(wl, H, seqs, L, R, N, V, fmt, True)) <= ONE


@pytest.mark.parametrize("fmt", [BF, E4M3])
@pytest.mark.parametrize("L,H", [(512, 8), (512, 64), (256, 14), (128, 64)])
@pytest.mark.parametrize("small", [2.0 ** -30, 1.0])
def test_queries_of_any_size(wl, fmt, L, H, small):  # noqa: F811
    """Queries of rows far apart in size, and some elements of each far below its largest."""
    b = batch(wl, H, [(200, 2), (50, 1)], L, 64, 64, 64, fmt, True)
    q = b.q.view(b.T, H, -1)
    q[:, ::2, :64] *= small
    q[:, :, 5] *= 2.0 ** -12
    q[0, 1, :64] = 0
    assert off(wl, b) <= ONE


@pytest.mark.parametrize("fmt", [BF, E4M3])
@pytest.mark.parametrize("L", [128, 256, 512])
@pytest.mark.parametrize("H", [8, 14, 64])
def test_without_weights(wl, fmt, L, H):  # noqa: F811
    """Queries are as given then, and outputs are rounded once."""
    for seqs in (SHORT, LONG):
        assert off(wl, batch(wl, H, seqs, L, 64, 64, 64, fmt, False), form="auto") <= ONE


@pytest.mark.parametrize("L,R,D", [(512, 64, 128), (256, 32, 64), (128, 64, 128), (512, 32, 64)])
@pytest.mark.parametrize("seqs", [[(20, 33), (0, 9)], [(300, 140)], [(1500, 20), (40, 130)]])
def test_expanded(wl, L, R, D, seqs):  # noqa: F811
    """Expanded keys and values and the weights are fp16: 2^-11 each, an eighth of the output's rounding."""
    assert off(wl, batch(wl, 3, seqs, L, R, D, D, BF, True), form="expanded") <= ONE


@pytest.mark.parametrize("mask", ["causal", "full"])
def test_expanded_rows_of_any_size(wl, mask):  # noqa: F811
    """Latents of rows far apart in size: each expanded row has a scale of its own, and weights times these stay
    within fp16, whether the large rows come first or last, with high scores or low ones."""
    for seed, sizes in enumerate(([0, 6, 3], [0, -20, -40], [20, 0, -20], [0, 15, 30], [40, 0, -40], [-30, 0, 30])):
        b = batch(wl, 4, [(180, 70), (100, 30)], 256, 64, 64, 64, BF, True)
        rows = b.cache.rows
        g = torch.Generator().manual_seed(seed)
        which = torch.randint(3, rows.shape[:2], generator=g)
        rows[..., :256] *= (2.0 ** torch.tensor(sizes, dtype=torch.float64))[which].to(rows.device)[..., None].to(BF)
        # the latents' part of a score is kept near 1 for the largest
        q = b.q.view(b.T, 4, -1)
        q[:, :, :64] *= 2.0 ** -max(sizes)
        q[:, :, 64:] *= 4.0
        assert off(wl, b, form="expanded", mask=mask) <= ONE, sizes


@pytest.mark.parametrize("form", ["expanded", "absorbed"])
@pytest.mark.parametrize("size", [100, 40, -100])
def test_rows_that_some_queries_do_not_see(wl, form, size):  # noqa: F811
    """A latent 2^100 times the others', seen by its own query alone in a tree, takes nothing from the others'."""
    b = batch(wl, 3, [(70, 4), (33, 1)], 256, 64, 128, 128, BF, True)
    b.cache.rows[b.cache.table[0, 72 // 64].item(), 72 % 64, :256] *= 2.0 ** size
    tree = i32([[1], [3], [5], [9], [1]])     # tokens 1, 2 and 3 follow token 0
    o = f64(b.run(wl, form=form, tree=tree, max_kv=128))
    ref, _ = serve_ref.latent_attention(b.q, b.cache, b.w, i32(b.starts), i32(b.lens), b.scale, tree=tree)
    rows = torch.tensor([0, 1, 3, 4])
    assert float((o[rows] - ref[rows]).norm() / (ref[rows].to(BF).double() - ref[rows]).norm()) <= ONE
