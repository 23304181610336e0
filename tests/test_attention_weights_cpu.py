"""The bar on attention's weights: a weight held as a bf16 and its remainder passes it,
one held as a single bf16 does not."""
from __future__ import annotations

import pytest
import torch

import weights_ref as wr


@pytest.mark.parametrize("n, d", [(64, 256), (500, 128), (2000, 64), (3000, 256)])
def test_the_bar_tells_one_bf16_from_two(n, d):
    g = torch.Generator().manual_seed(n)
    k, v = (t.double() for t in wr.keys(g, n, 1, d))
    q = wr.queries(g, 8, 1, d).double()
    scale = d ** -0.5 / 2
    o, slack = wr.attention(q, k, v, scale, wr.TWO)
    s = (q @ k.T).float() * torch.tensor(scale, dtype=torch.float32)
    p = (s - s.amax(-1, keepdim=True)).exp()
    head = p.to(torch.bfloat16)
    rest = (p - head.float()).to(torch.bfloat16)
    total = p.sum(-1, keepdim=True)
    two = ((head.double() + rest.double()) @ v / total.double()).to(torch.bfloat16)
    one = (head.double() @ v / total.double()).to(torch.bfloat16)
    as_summed = (head.double() @ v / head.double().sum(-1, keepdim=True)).to(torch.bfloat16)
    assert wr.excess(two, o, slack) <= 1
    assert wr.excess(one, o, slack) > 1 and wr.excess(as_summed, o, slack) > 1
    o, slack = wr.attention(q, k, v, scale, 2 * wr.ONE)
    assert wr.excess(one, o, slack) <= 1 and wr.excess(as_summed, o, slack) <= 1
