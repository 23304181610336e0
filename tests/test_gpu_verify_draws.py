"""Draws whose border lies within fp64's rounding of a running sum: a token without weight is never
drawn, and the drawn one lies beside the border."""
from __future__ import annotations

import pytest
import torch

from tests.test_gpu_verify_no_rows import DEV, i32, wl  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("with_draft", [True, False])
@pytest.mark.parametrize("first", [0, 4 * 62, 4 * 300])
def test_running_sums_that_fall(wl, with_draft, first):  # noqa: F811
    """Groups of 16 bytes with weights 2^-53, 2^-53, 1, 0, .., 1 and u = 1/2, so that u times the whole is 1 in fp64.
    Summed as ((a + b) + c) + 0 the running sum is 1 + 2^-52 from c on, as (c + b) + a it is 1 there: a scan
    over lanes brackets each lane's sum in its own way, and may pass 1 at a lane whose own weights are 0."""
    V = 4 * 512
    for far in (8, 40, 100, 200):
        p = torch.zeros(1, V)
        p[0, first], p[0, first + 4], p[0, first + 8], p[0, first + 4 * far] = 2.0 ** -53, 2.0 ** -53, 1.0, 1.0
        p = p.to(DEV)
        out, n, _ = wl.wl_verify_drafts(p, i32([0]), i32([0, 1]), torch.full((1, 2), 0.5, device=DEV), probabilities=True,
                                        draft=p.clone() if with_draft else None)
        assert n.tolist() == [1] and out.tolist()[0] in (first + 8, first + 4 * far), far
