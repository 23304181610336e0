"""How far latent attention in bf16 is from its definition in 64 bits, against what its output's own
rounding costs.

A rounding to bf16 is off by up to half a step, uniformly: 2^-7 / sqrt(12) of a power of two in the root mean
square, times sqrt(E[1 / m^2]) = 0.74 for a mantissa m in [1, 2) of density 1 / (m ln 2), so 0.00166 of the
value. Roundings of random sign add up in squares: k of them, each of a factor of the output, come to sqrt(k)
of the output's own, which is what is measured here. A sum of 512 random squares or more scatters by less than
1 / sqrt(512) = 5 %."""
from __future__ import annotations

import pytest

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
