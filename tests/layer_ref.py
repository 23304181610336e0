"""64-bit references of the operations between the projections, on the CPU, and
the bars their outputs are held to.

A rounding to a type is off by at most half a step, finfo(type).eps / 2 of the
value; EPS32 = 2^-24 is that of fp32, in which the kernels compute. Bars add, to
the output's own rounding, a small number of fp32 roundings of the magnitudes
that enter (64 covers the longest chain of a row sum: 32 elements per lane, six
lane steps, 16 waves, and the few products around it), and for attention what
its documented roundings allow.
"""
from __future__ import annotations

import torch

EPS32 = 2.0 ** -24
CHAIN = 64


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def f64(t):
    return t.detach().cpu().double()


def assert_near(got, ref, slack, what):
    """|got - ref| <= half a step of got's type at ref + slack, per element."""
    g = f64(got)
    assert torch.isfinite(g).all(), f"{what}: non-finite output"
    err, bar = (g - ref).abs(), half_step(got.dtype) * ref.abs() * (1 + 2 ** -7) + slack + 1e-38
    worst = (err / bar).max() if err.numel() else torch.tensor(0.0)
    assert worst <= 1, f"{what}: error {float(worst):.3f} of the bar at {int((err / bar).argmax())}"


def rms(z, w, eps, offset):
    inv = 1 / (z.square().mean(-1, keepdim=True) + eps).sqrt()
    return z * inv * ((w if w is not None else 1 - offset) + offset), inv


def norm(x, y, post, pre, gate, eps, offset, rs, bs):
    """(x', n) and the magnitudes that enter each."""
    x, y, post, pre, gate = (None if t is None else f64(t) for t in (x, y, post, pre, gate))
    out, mag = rs * x, abs(rs) * x.abs()
    if y is not None:
        p = y if post is None else rms(y, post, eps, offset)[0]
        p = bs * (p if gate is None else p * gate)
        out, mag = out + p, mag + p.abs()
    n, inv = rms(out, pre, eps, offset)
    w = (pre if pre is not None else torch.ones(1)) + (offset if pre is not None else 0)
    return out, n, mag, mag * inv * w.abs()


def rotate(x, d, pos, freq, scale, interleaved, w=None, eps=0.0, offset=0.0):
    """Heads of d rotated, and the magnitude of each element's pair."""
    z = f64(x).view(x.shape[0], -1, d)
    if w is not None:
        z, _ = rms(z, f64(w), eps, offset)
    out, mag = z.clone(), z.abs()
    if freq is not None:
        r = freq.numel()
        ang = torch.outer(pos.cpu().double(), f64(freq))[:, None]
        a = slice(0, 2 * r, 2) if interleaved else slice(0, r)
        b = slice(1, 2 * r, 2) if interleaved else slice(r, 2 * r)
        c, s = ang.cos() * scale, ang.sin() * scale
        out[..., a], out[..., b] = z[..., a] * c - z[..., b] * s, z[..., a] * s + z[..., b] * c
        m = (z[..., a].abs() + z[..., b].abs()) * abs(scale)
        mag[..., a], mag[..., b] = m, m
    return out.flatten(1), mag.flatten(1)


def codes(x, fmt):
    """(codes as values, scale) of rows [..., d] in 64 bits: ties to even."""
    x = f64(x)
    top = 127.0 if fmt == torch.int8 else 448.0
    most = x.abs().amax(-1, keepdim=True)
    z = torch.where(most > 0, x * top / most.clamp(min=1e-300), torch.zeros_like(x))
    if fmt == torch.int8:
        return z.round(), most.squeeze(-1) / top
    step = 2.0 ** ((torch.frexp(z).exponent - 1).clamp(min=-6).double() - 3)
    return (z / step).round() * step, most.squeeze(-1) / top


def cache_rows(cache, s, n):
    """K, V [n][n_kv][d] of the first n slots of sequence s in 64 bits, and which have a page."""
    page = cache.k.shape[2]
    table = cache.table.cpu()
    j = torch.arange(n)
    pid = table[s, j // page].long()
    has = (pid >= 0) & (pid < cache.k.shape[0])
    pid, off = pid.clamp(0, cache.k.shape[0] - 1), j % page
    out = []
    for pool, scale in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        p = pool.cpu()
        x = (p.view(torch.uint8)[pid, :, off].view(p.dtype).float() if p.dtype.itemsize == 1 else p[pid, :, off]).double()
        out.append(x if scale is None else x * scale.cpu().double()[pid, :, off][..., None])
    return out[0], out[1], has


def attention(q, cache, q_start, kv_len, scale, mask=None, window=0, tree=None, q_pos=None, max_kv=None):
    """(o, slack): slack is the bar beyond the output's own rounding. Rows outside
    every sequence are NaN in o."""
    mask = mask or ("causal" if tree is None else "tree")
    d, n_kv = cache.k.shape[3], cache.k.shape[1]
    n_q = q.shape[1] // d
    g = n_q // n_kv
    qd = f64(q).view(-1, n_q, d)
    o = torch.full_like(qd, float("nan"))
    slack = torch.zeros_like(qd)
    starts, lens = q_start.tolist(), kv_len.tolist()
    # the weights' rounding and their sum's (bf16), then fp32 sums of the keys
    w_err = 2 * half_step(torch.bfloat16) if q.dtype == torch.bfloat16 else 0.0
    for s in range(len(lens)):
        lo, hi = starts[s], starts[s + 1]
        total, m = lens[s], hi - lo
        n = min(total, cache.table.shape[1] * cache.k.shape[2], total if max_kv is None else max_kv)
        if m == 0:
            continue
        n = max(n, 0)
        k, v, has = cache_rows(cache, s, n)
        ctx, j = total - m, torch.arange(n)
        at = ctx + torch.arange(m)[:, None]
        if mask == "full":
            see = torch.ones(m, n, dtype=torch.bool)
        elif mask == "causal":
            see = (j <= at) & ((j > at - window) if window else True)
        else:
            words = tree[lo:hi].cpu().long() & 0xFFFFFFFF
            e = (j - ctx).clamp(0, 32 * words.shape[1] - 1)
            bit = (words[:, e // 32] >> (e % 32) & 1).bool() & (j - ctx < 32 * words.shape[1])
            p = at if q_pos is None else q_pos[lo:hi].cpu().long()[:, None]
            early = (j > p - window).expand(m, -1) if window else torch.ones(m, n, dtype=torch.bool)
            see = torch.where(j < ctx, early, bit)
        see = see & has
        for h in range(n_q):
            kk, vv = k[:, h // g], v[:, h // g]
            used = see.any(0)
            kk, vv = (torch.where(used[:, None], t, torch.zeros(())) for t in (kk, vv))
            sc = qd[lo:hi, h] @ kk.T * scale
            sc = torch.where(see, sc, -torch.inf)
            big = sc.amax(1, keepdim=True) if n else torch.full((m, 1), -torch.inf, dtype=torch.float64)
            w = torch.where(sc == -torch.inf, 0.0, (sc - torch.where(big == -torch.inf, 0.0, big)).exp())
            l = w.sum(1, keepdim=True)
            w = torch.where(l > 0, w / l.clamp(min=1e-300), 0.0)
            # keys not seen contribute nothing, whatever they hold
            o[lo:hi, h] = torch.stack([w[i][see[i]] @ v[:, h // g][see[i]] for i in range(m)])
            ds = (d + 8) * EPS32 * abs(scale) * (qd[lo:hi, h].abs() @ kk.abs().T).masked_fill(~see, 0).amax(1, keepdim=True) if n else 0.0
            ds = ds + 2 * EPS32 * (torch.where(see, sc, torch.zeros(())).abs().amax(1, keepdim=True) if n else 0.0)
            slack[lo:hi, h] = (w_err + 2 * ds + (n / 16 + CHAIN) * EPS32) * (w @ vv.abs())
    return o.flatten(1), slack.flatten(1)
