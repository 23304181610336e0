"""Verification of batches without rows."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def wl():
    from linear_02_amd import wl as mod
    return mod


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("n_seq", [1, 7, 1000])
@pytest.mark.parametrize("with_draft", [True, False])
def test_no_rows(wl, n_seq, with_draft):
    """An empty batch keeps 0 tokens of every sequence, whatever the last call left there."""
    target, token, u = torch.zeros(0, 50, device=DEV), i32([]), torch.zeros(0, 2, device=DEV)
    n_out, length = i32([-7] * n_seq), i32(list(range(n_seq)))
    call = wl.verify_drafts_call(target, token, i32([0] * (n_seq + 1)), u, draft=target.clone() if with_draft else None,
                                 length=length, n_out=n_out)
    out, n, path = call.launch()
    assert out.numel() == path.numel() == 0 and n is n_out
    assert (n_out == 0).all() and torch.equal(length, i32(list(range(n_seq))))
    step = wl.LayerStep([call])
    for _ in range(3):
        n_out.fill_(-7)
        step.launch()
        assert (n_out == 0).all()
