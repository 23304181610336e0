"""64-bit references of the operations around a serving batch, on the CPU, and the
bars their outputs are held to (half_step, EPS32 and CHAIN as in layer_ref).

What latent attention rounds to bf16, each off by at most 2^-8 of the value: queries in
the latent space or expanded keys (which move a score), outputs in the latent space or
expanded values, the weights of the second product and their sum. Per element the bar
adds these up at their worst. Since they are of random sign, the whole output is also
held to REL_BF16 in the 2-norm: a rounding is off by at most 2^-8 and about 2^-8 / 2.3 =
0.0017 in the mean square; four of them (the output's own among them), of scores of about
1, come to 0.0034.
"""
from __future__ import annotations

import torch

from tests.layer_ref import CHAIN, EPS32, f64, half_step

REL_BF16 = 0.005


def plan(table, held, free, n_free, past, n_new, T, page):
    """One wl_batch_plan on lists: (q_start, kv_len, seq, slot); table, held and free
    (a list without what lies above the top) are changed."""
    room = len(table[0])
    past, n_new = [max(p, 0) for p in past], [max(n, 0) for n in n_new]
    want = [-(-(p + n) // page) for p, n in zip(past, n_new)]
    lacked = asked = 0
    starts, lens, seq, slot, back = [0], [], [], [], []
    height = len(free)
    ok = []
    for w, h in zip(want, held):
        lack = max(w - h, 0) if w <= room else 0
        lacked += lack
        ok.append(w <= room and (lack == 0 or lacked <= height))
    for s, n in enumerate(n_new):
        asked += n if ok[s] else 0
        served = ok[s] and (n == 0 or asked <= T)
        if served:
            seq += [s] * n
            slot += list(range(past[s], past[s] + n))
            for j in range(held[s], want[s]):
                table[s][j] = free.pop()
            held[s] = max(held[s], want[s])
        lens.append(past[s] + n if served else past[s])
        starts.append(len(seq))
        keep = min(-(-lens[s] // page), room, held[s])
        back += table[s][keep:held[s]]
        table[s][keep:held[s]] = [-1] * (held[s] - keep)
        held[s] = keep
    free += back
    pad = T - len(seq)
    return starts, lens, seq + [-1] * pad, slot + [-1] * pad


def weights(x, kind, t):
    """fp64 weights of one row: powers of logits over t, or the given ones."""
    x = f64(x)
    if kind == "probabilities":
        return torch.where(x > 0, x, torch.zeros_like(x))
    x = torch.where(x.isnan(), torch.full_like(x, -torch.inf), x)
    top = x.max()
    if top == -torch.inf:
        return torch.zeros_like(x)
    w = torch.where(x == top, torch.ones_like(x), ((x - top) / t).exp())
    return torch.where(x == -torch.inf, torch.zeros_like(x), w)


def largest(x, kind):
    """The first of the largest entries, -1 where there is nothing."""
    x = f64(x)
    x = torch.where(x.isnan(), torch.full_like(x, -torch.inf), x) if kind == "logits" else torch.where(x > 0, x, torch.zeros_like(x))
    top = x.max()
    return -1 if top == (-torch.inf if kind == "logits" else 0) else int((x == top).nonzero()[0])


def drawn(w, u):
    """(token, how far u times the whole is from the nearest border, as part of the whole)"""
    run = w.cumsum(0)
    total = float(run[-1])
    if total == 0:
        return -1, 1.0
    aim = float(u) * total
    x = int(torch.searchsorted(run, torch.tensor([aim], dtype=torch.float64), right=True)[0])
    x = min(x, int((w > 0).nonzero()[-1]))
    return x, float((run - aim).abs().min()) / total if aim else 1.0   # which weights are 0 is no rounding's to decide


def verify(target, token, starts, u, draft=None, parent=None, temperature=None, kind="logits", max_q=1024):
    """(out, n_out, path) as lists with None in rows outside every sequence, and the nearest
    distance of a decision from its border."""
    T = len(token)
    out, path, n_out, near = [None] * T, [None] * T, [], 1.0
    for s in range(len(starts) - 1):
        lo = min(max(starts[s], 0), T)
        m = min(min(max(starts[s + 1], lo), T) - lo, max_q)
        out[lo:lo + m], path[lo:lo + m] = [-1] * m, [-1] * m
        t = 1.0 if temperature is None else float(temperature[s])
        at = n = 0
        while n < m:
            r = lo + at
            path[lo + n] = at
            if draft is not None:
                nxt = token[r + 1] if at + 1 < m else None
                if t > 0:
                    p, q = weights(target[r], kind, t), weights(draft[r], kind, t)
                    if kind == "logits":
                        p, q = (w / w.sum().clamp(min=1e-300) for w in (p, q))   # a row of nothing stays nothing
                    stay = False
                    if nxt is not None and 0 <= nxt < p.numel():
                        a, b = float(u[r][0]) * float(q[nxt]), float(p[nxt])
                        stay, near = a < b, min(near, abs(a - b) / max(a, b) if a or b else 1.0)
                    left = (p - q).clamp(min=0)
                    x, d = drawn(left if nxt is not None and float(left.sum()) > 0 else p, u[r][1])
                else:
                    x, d = largest(target[r], kind), 1.0
                    stay = nxt is not None and x == nxt and x >= 0
                if stay:
                    out[lo + n], at, n = nxt, at + 1, n + 1
                    continue
                out[lo + n], n, near = x, n + 1, min(near, d)
                break
            x, d = (drawn(weights(target[r], kind, t), u[r][1]) if t > 0 else (largest(target[r], kind), 1.0))
            out[lo + n], n, near = x, n + 1, min(near, d)
            follow = [i for i in range(at + 1, m) if x >= 0 and token[lo + i] == x and (i - 1 if parent is None else parent[lo + i]) == at]
            if not follow:
                break
            at = follow[0]
        n_out.append(n)
    return out, n_out, path, near


def latent_rows(cache, s, n):
    """(latents, keys, which have a page) of the first n slots of sequence s in 64 bits."""
    page = cache.rows.shape[1]
    table, pool, j = cache.table.cpu(), cache.rows.cpu(), torch.arange(n)
    pid = table[s, j // page].long()
    has = (pid >= 0) & (pid < pool.shape[0])
    pid, off, L = pid.clamp(0, pool.shape[0] - 1), j % page, cache.latent
    rows = pool[pid, off]
    if rows.dtype == torch.uint8:
        c = rows[:, :L].contiguous().view(torch.float8_e4m3fn).float().double() * cache.scale.cpu().double()[pid, off][:, None]
        return c, rows[:, L:].contiguous().view(torch.bfloat16).double(), has
    return rows[:, :L].double(), rows[:, L:].double(), has


def latent_attention(q, cache, w, q_start, kv_len, scale, mask=None, window=0, tree=None, q_pos=None, max_kv=None,
                     max_q=None, expanded=False):
    """(o, slack): slack is the bar beyond the output's own rounding. Rows outside every
    sequence are NaN in o."""
    mask = mask or ("causal" if tree is None else "tree")
    L, R = cache.latent, cache.rot
    H = q.shape[1] // (L + R) if w is None else w.shape[0]
    qd = f64(q).view(q.shape[0], H, -1)
    N = qd.shape[2] - R
    V = L if w is None else w.shape[1] - N
    o = torch.full((q.shape[0], H, V), float("nan"), dtype=torch.float64)
    slack = torch.zeros_like(o)
    starts, lens = q_start.tolist(), kv_len.tolist()
    b = half_step(torch.bfloat16) if q.dtype == torch.bfloat16 else 0.0
    for s in range(len(lens)):
        lo, m = starts[s], starts[s + 1] - starts[s]
        rows = m if max_q is None else min(m, max_q)
        if rows <= 0:
            continue
        total = lens[s]
        n = max(min(total, cache.table.shape[1] * cache.rows.shape[1], total if max_kv is None else max_kv), 0)
        c, key, has = latent_rows(cache, s, n)
        ctx, j = total - m, torch.arange(n)
        at = ctx + torch.arange(rows)[:, None]
        if mask == "full":
            see = torch.ones(rows, n, dtype=torch.bool)
        elif mask == "causal":
            see = (j <= at) & ((j > at - window) if window else True)
        else:
            words = tree[lo:lo + rows].cpu().long() & 0xFFFFFFFF
            e = (j - ctx).clamp(0, 32 * words.shape[1] - 1)
            bit = (words[:, e // 32] >> (e % 32) & 1).bool() & (j - ctx < 32 * words.shape[1])
            p = at if q_pos is None else q_pos[lo:lo + rows].cpu().long()[:, None]
            early = (j > p - window).expand(rows, -1) if window else torch.ones(rows, n, dtype=torch.bool)
            see = torch.where(j < ctx, early, bit)
        see = see & has
        used = see.any(0)
        c, key = (torch.where(used[:, None], t, torch.zeros(())) for t in (c, key))   # nothing else has any influence
        for h in range(H):
            x = qd[lo:lo + rows, h]
            wk = torch.eye(L, dtype=torch.float64) if w is None else f64(w[h, :N])
            wv = torch.eye(L, dtype=torch.float64) if w is None else f64(w[h, N:])
            ql = x[:, :N] @ wk
            sc = (ql @ c.T + x[:, N:] @ key.T) * scale
            part = ql.abs() @ c.abs().T if not expanded else x[:, :N].abs() @ (c @ wk.T).abs().T
            sums = (x[:, :N].abs() @ wk.abs() @ c.abs().T + x[:, N:].abs() @ key.abs().T)
            sc = torch.where(see, sc, -torch.inf)
            big = sc.amax(1, keepdim=True) if n else torch.full((rows, 1), -torch.inf, dtype=torch.float64)
            p = torch.where(sc == -torch.inf, 0.0, (sc - torch.where(big == -torch.inf, 0.0, big)).exp())
            l = p.sum(1, keepdim=True)
            p = torch.where(l > 0, p / l.clamp(min=1e-300), 0.0)
            o[lo:lo + rows, h] = (p @ c) @ wv.T
            if not n:
                continue
            hide = lambda t: t.masked_fill(~see, 0).amax(1, keepdim=True)  # noqa: E731
            ds = abs(scale) * (b * hide(part) * (w is not None) + (L + N + R + 8) * EPS32 * hide(sums)) + 2 * EPS32 * hide(torch.where(see, sc, torch.zeros(())).abs())
            rel = 2 * b + 2 * ds + (n / 16 + L + CHAIN) * EPS32
            if expanded:
                slack[lo:lo + rows, h] = (rel + b) * (p @ (c @ wv.T).abs()) + (L + 8) * EPS32 * (p @ c.abs() @ wv.abs().T)
            else:
                slack[lo:lo + rows, h] = ((rel + (b if w is not None else 0.0) + (L + 8) * EPS32) * (p @ c.abs())) @ wv.abs().T
    return o.flatten(1), slack.flatten(1)
