"""Verification of drafted tokens against its definition in 64 bits: whole numbers, equal.
A decision that lies within 1e-9 of its border could go either way; none of these does."""
from __future__ import annotations

import random

import pytest
import torch

from tests import serve_ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def wl():
    from linear_02_amd import wl as mod
    return mod


def make(seed, rows, V, dtype, kind, with_draft, tree, t, gap=0):
    """Rows of every sequence (with `gap` rows of nobody in front), their logits or probabilities, drafted tokens."""
    g, rng = torch.Generator().manual_seed(seed), random.Random(seed)
    T = gap + sum(rows)
    x = torch.randn(T, V, generator=g) * 2
    x.scatter_(1, torch.randint(V, (T, 2), generator=g), 2 + torch.log(torch.tensor(float(V))).item())
    y = x + torch.randn(T, V, generator=g) * 0.7
    parent = [-1] * gap + [p for n in rows for p in ([-1] + [rng.randrange(max(0, i - 4), i) for i in range(1, n)])[:n]]
    starts = [gap + sum(rows[:i]) for i in range(len(rows) + 1)]
    if kind == "probabilities":
        x, y = x.softmax(-1), y.softmax(-1)
    x, y = x.to(dtype), y.to(dtype)
    token = [0] * T
    for s, n in enumerate(rows):
        for i in range(1, n):
            up = starts[s] + (parent[starts[s] + i] if tree else i - 1)
            if with_draft and rng.random() < 0.9:
                token[starts[s] + i] = int((y[up].float() if kind == "logits" else y[up].float().log()).add(
                    -torch.empty(V).exponential_(generator=g).log()).argmax())
            else:
                token[starts[s] + i] = int(x[up].float().topk(min(3, V)).indices[rng.randrange(min(3, V))])
    u = torch.rand(T, 2, generator=g)
    temperature = None if t is None else torch.tensor([t if s % 3 != 2 else 0.0 for s in range(len(rows))])
    return x, (y if with_draft else None), token, starts, (parent if tree else None), u, temperature


def check(wl, args, kind, max_q=1024, ld=0, what=""):
    x, y, token, starts, parent, u, temperature = args
    out, n_out, path, near = serve_ref.verify(x, token, starts, u.tolist(), y, parent, temperature, kind, max_q)
    assert near > 1e-9, "a decision at its border"
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    V = x.shape[1]

    def place(t):
        if t is None:
            return None
        wide = torch.full((t.shape[0], V + ld), float("nan"), dtype=t.dtype, device=DEV)
        wide[:, :V] = t.to(DEV)
        return wide[:, :V]
    T = len(token)
    length = i32([100 + s for s in range(len(n_out))])
    got_out, got_n, got_path = i32([-77] * T), i32([-77] * len(n_out)), i32([-77] * T)
    wl.wl_verify_drafts(place(x), i32(token), i32(starts), u.to(DEV), draft=place(y), parent=None if parent is None else i32(parent),
                        temperature=None if temperature is None else temperature.to(DEV), probabilities=kind == "probabilities",
                        max_q=max_q, length=length, out=got_out, n_out=got_n, path=got_path)
    assert got_n.tolist() == n_out, what
    assert got_out.tolist() == [-77 if v is None else v for v in out], what
    assert got_path.tolist() == [-77 if v is None else v for v in path], what
    assert length.tolist() == [100 + s + n for s, n in enumerate(n_out)], what
    return n_out


@pytest.mark.parametrize("V", [1, 2, 7, 8, 1000, 4099, 32001])
@pytest.mark.parametrize("dtype,kind", [(BF, "logits"), (F32, "logits"), (F32, "probabilities")])
@pytest.mark.parametrize("form", ["draft", "chain", "tree"])
def test_against_definition(wl, V, dtype, kind, form):
    for seed, t in ((1, None), (2, 0.7), (3, 1.0)):
        args = make(seed + V, [5, 1, 3, 8, 0, 2, 4], V, dtype, kind, form == "draft", form == "tree", t, gap=2)
        check(wl, args, kind, ld=seed - 1, what=f"seed {seed}")


@pytest.mark.parametrize("form", ["draft", "tree"])
def test_many_rows_and_long_ones(wl, form):
    args = make(5, [40, 17, 33, 64], 5003, BF, "logits", form == "draft", form == "tree", 0.9)
    assert max(check(wl, args, "logits", ld=5)) > 1
    args = make(6, [3, 2], 262147, BF, "logits", form == "draft", form == "tree", 1.0)
    check(wl, args, "logits")


def test_rows_beyond_max_q(wl):
    for form in (True, False):
        check(wl, make(11, [9, 4, 12], 300, F32, "logits", form, not form, 1.0, gap=1), "logits", max_q=5)


@pytest.mark.parametrize("with_draft", [True, False])
def test_odd_values(wl, with_draft):
    """-inf, NaN and +inf logits; rows of nothing; u = 0 and just below 1."""
    inf, nan = float("inf"), float("nan")
    x, y, token, starts, parent, u, t = make(21, [3, 3, 3, 3, 3], 500, F32, "logits", with_draft, False, None)
    x[0, 10:] = -inf
    x[3, ::2] = nan
    x[6, 77] = inf
    x[9] = -inf
    x[12] = nan
    u[:6] = 0.0
    u[6:] = 1 - 2.0 ** -24
    for temperature in (None, torch.tensor([0.0] * 5), torch.tensor([1e-30, 1e30, 2.0, 5.0, -1.0])):
        check(wl, (x, y, token, starts, parent, u, temperature), "logits")
    x[6, 77] = 3.0
    check(wl, (x, y, token, starts, parent, u, torch.tensor([inf, 0.3, inf, inf, nan])), "logits")


def test_probabilities_with_nothing_left(wl):
    """Drafts at least as likely as the target everywhere: the token behind a refused one is drawn from the target."""
    V = 1000
    g = torch.Generator().manual_seed(3)
    p = torch.rand(4, V, generator=g)
    q = p * 2
    u = torch.full((4, 2), 0.75)
    args = (p, q, [0, 5, 6, 7], [0, 4], None, u, None)
    n = check(wl, args, "probabilities")
    assert n == [1]
    p[:] = 0
    p[0, 5], p[1, 6], p[2, 7] = 1.0, 1.0, -1.0
    check(wl, (p, q, [0, 5, 6, 7], [0, 4], None, u, None), "probabilities")


def test_tokens_outside_the_vocabulary(wl):
    x, y, token, starts, parent, u, t = make(31, [4, 4], 64, F32, "logits", True, False, 1.0)
    token[1], token[5] = 64, -3
    check(wl, (x, y, token, starts, None, u, t), "logits")
    check(wl, (x, None, token, starts, None, u, t), "logits")
    x[:] = -float("inf")      # no token anywhere: a drafted -1 is not followed
    check(wl, (x, None, [0, -1, -1, -1] * 2, starts, [-1, 0, 1, 2] * 2, u, t), "logits")
    check(wl, (x, y, [0, -1, -1, -1] * 2, starts, None, u, torch.tensor([0.0, 0.0])), "logits")


def test_wild_parents(wl):
    """Parents out of reach, later rows, themselves: such rows are never next."""
    x, _, token, starts, parent, u, t = make(41, [6, 6], 40, F32, "logits", False, True, 1.0)
    token = [3] * 12
    x[:, 3] += 30
    parent = [-1, 1, 5, -9, 1 << 30, 0, -1, 0, 0, 9, 2, 4]
    n = check(wl, (x, None, token, starts, parent, u, t), "logits")
    assert n == [2, 2]


def test_repeatable_and_in_a_graph(wl):
    for form in ("draft", "tree"):
        x, y, token, starts, parent, u, t = make(51, [5, 4, 5], 20011, BF, "logits", form == "draft", form == "tree", 0.8)
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
        x2 = x.flip(0).contiguous()
        target, tok, start, uu = x.to(DEV), i32(token), i32(starts), u.to(DEV)
        call = wl.verify_drafts_call(target, tok, start, uu, draft=None if y is None else y.to(DEV),
                                     parent=None if parent is None else i32(parent), temperature=t.to(DEV))
        g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
            call.launch()
        torch.cuda.current_stream().wait_stream(s)
        for k in range(6):
            data = (x, x2)[k % 2]
            target.copy_(data)
            g.replay()
            torch.cuda.synchronize()
            out, n_out, path, near = serve_ref.verify(data, token, starts, u.tolist(), y, parent, t)
            assert near > 1e-9
            assert call.out[0].tolist() == out and call.out[1].tolist() == n_out and call.out[2].tolist() == path
