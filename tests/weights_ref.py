"""Inputs and a bar that tell how many bits attention's weights are held in.

Keys come in pairs with nearly the same score and opposite values, so the output is
a small difference of large terms and its own rounding hides little. Queries and
keys are small multiples of powers of two: every product q . k is exact in fp32, and
what is left of an error is that of the weights.

A weight as one bf16 is off by at most half a step, 2^-8 of it; as a bf16 and a bf16
remainder by at most 2^-8 of 2^-8.
"""
from __future__ import annotations

import torch

import layer_ref as ref

ONE, TWO = ref.half_step(torch.bfloat16), ref.half_step(torch.bfloat16) ** 2


def keys(g, n, n_kv, d):
    """K, V fp32 [n][n_kv * d], n even."""
    k = torch.randint(-8, 9, (n // 2, n_kv, d), generator=g).float() / 8
    v = torch.randint(0, 2, (n // 2, n_kv, d), generator=g).float() * 2 - 1
    near = k.clone()
    near[..., 0] = near[..., 0].sign() * (near[..., 0].abs() - 0.125) + (near[..., 0] == 0) * 0.125
    return torch.stack((k, near), 1).reshape(n, -1), torch.stack((v, -v), 1).reshape(n, -1)


def queries(g, rows, n_q, d):
    return torch.randint(-2, 3, (rows, n_q * d), generator=g).float()


def bar(w, v, scores, n, held):
    """Largest error beyond the output's own rounding: of the weights as they are held,
    of the scores (a scale or two, the power of two: a handful of fp32 roundings of the
    score), of fp32 sums over the keys and the few factors beside them."""
    most = scores.abs().amax(-1, keepdim=True)
    return (held + 2 * 8 * ref.EPS32 * most + (n / 16 + ref.CHAIN) * ref.EPS32) * (w @ v.abs())


def attention(q, k, v, scale, held):
    """(o, slack) of rows q [m][d] over keys and values [n][d], all visible, in 64 bits."""
    s = q @ k.T * scale
    w = torch.softmax(s, -1)
    return w @ v, bar(w, v, s, k.shape[0], held)


def excess(got, o, slack):
    """Largest error as a share of what is allowed."""
    g = ref.f64(got)
    allowed = ref.half_step(got.dtype) * o.abs() * (1 + 2 ** -7) + slack
    return float(((g - o).abs() / allowed).max())
