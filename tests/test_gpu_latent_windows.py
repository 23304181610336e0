"""Windows that reach far beyond a sequence: queries in front of its first slot, windows up to the
largest int."""
from __future__ import annotations

import pytest

from tests.test_gpu_latent import BF, E4M3, F32, Batch, wl  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form,fmt", [("expanded", BF), ("absorbed", BF), ("absorbed", E4M3), ("absorbed", F32)])
@pytest.mark.parametrize("window", [(1 << 31) - 1, (1 << 31) - 5, 1 << 30])
def test_large_windows(wl, form, fmt, window):  # noqa: F811
    b = Batch(wl, [(60, 40), (200, 150), (0, 3)], 3, fmt=fmt, seed=21)
    b.lens = [37, 149, 3]       # the first queries of two sequences have slots below 0
    o = b.check(wl, "window", window=window, form=form, expanded=form == "expanded")
    assert (o[:3] == 0).all() and (o[3:40] != 0).any(1).all()
