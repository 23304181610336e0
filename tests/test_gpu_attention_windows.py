"""wl_attention under windows up to the largest int, with queries in front of their sequence's first slot."""
from __future__ import annotations

import pytest

from test_gpu_attention import BF, E4, F32, I8, Batch, wl  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [BF, I8, E4, F32])
@pytest.mark.parametrize("rows", [[6, 3], [40, 150], [260, 9]])
@pytest.mark.parametrize("window", [(1 << 31) - 1, (1 << 31) - 5, 1 << 30])
def test_large_windows(wl, fmt, rows, window):  # noqa: F811
    o = Batch(wl, [-3, 200], rows, 4, 2, 128, 16, fmt, seed=rows[0], extra=1).check(wl, window=window)
    assert (o[:3] == 0).all() and (o[3:rows[0]] != 0).any(1).all()
