"""The batch's plan (rows, slots, page tables, the stack of free pages) against a plain
one on lists: whole numbers, equal."""
from __future__ import annotations

import random

import pytest
import torch

from tests import serve_ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def wl():
    from linear_02_amd import wl as mod
    return mod


def lists(pages):
    """table, held, free, n_free on the host; what lies above the top has to be -1."""
    torch.cuda.synchronize()
    n, free = int(pages.n_free), pages.free.tolist()
    assert all(v == -1 for v in free[n:]), "above the top of the stack"
    return pages.table.tolist(), pages.held.tolist(), free[:n]


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def check(wl, pages, past, n_new, T, page, what=""):
    table, held, free = lists(pages)
    ref = serve_ref.plan(table, held, free, len(free), past, n_new, T, page)
    out = wl.wl_batch_plan(pages, i32(past), i32(n_new), T)
    got = [t.tolist() for t in out]
    for name, g, r in zip(("q_start", "kv_len", "seq", "slot"), got, ref):
        assert g == list(r), f"{what}: {name}"
    t, h, f = lists(pages)
    assert h == held and f == free and t == table, f"{what}: pages"
    return out


@pytest.mark.parametrize("n_seq,T", [(1, 1), (2, 7), (64, 100), (65, 8192), (1000, 3000), (1024, 500), (1025, 2000), (2500, 9000)])
@pytest.mark.parametrize("page,n_pages,max_pages", [(16, 4000, 40), (64, 900, 12)])
def test_steps_of_a_batch(wl, n_seq, T, page, n_pages, max_pages):
    """Growing, rolling back, dropping and filling slots anew, until pages or rows run out."""
    rng = random.Random(n_seq * 31 + T + page)
    pages = wl.new_pages(n_seq, max_pages, n_pages, page, DEV)
    past = [0] * n_seq
    for step in range(7):
        fresh = [rng.choice((0, 1, 1, 3, rng.randrange(1, 2 * page + 2))) for _ in past]
        if step == 2:
            fresh[rng.randrange(n_seq)] = max_pages * page + 1     # longer than a row of the table
        if step == 3:
            past = [0 if rng.random() < 0.5 else p for p in past]  # half of them dropped
        _, kv, _, _ = check(wl, pages, past, fresh, T if step != 4 else 0, page, f"step {step}")
        past = [max(k - rng.choice((0, 0, 1, 5)), 0) for k in kv.tolist()]


def test_no_rows_takes_pages_back(wl):
    pages = wl.new_pages(3, 8, 20, 16, DEV)
    check(wl, pages, [0, 0, 0], [40, 1, 128], 169, 16)
    assert pages.held.tolist() == [3, 1, 8] and int(pages.n_free) == 8
    check(wl, pages, [17, 0, 128], [0, 0, 0], 0, 16)
    assert pages.held.tolist() == [2, 0, 8] and int(pages.n_free) == 10


def test_order_of_service(wl):
    """One that the stack does not cover holds up those behind it that lack pages, not the others; too few rows hold
    up all behind that have any."""
    pages = wl.new_pages(5, 8, 6, 16, DEV)
    check(wl, pages, [0] * 5, [16, 0, 0, 16, 1], 40, 16)             # 3 pages
    out = check(wl, pages, [16, 0, 0, 15, 1], [1, 60, 1, 1, 20], 40, 16)
    assert out[0].tolist() == [0, 1, 1, 1, 2, 2]                     # 1: lacks 4 of 2; 2 and 4 lack pages behind it
    out = check(wl, pages, [17, 0, 0, 16, 1], [3, 0, 9, 0, 1], 11, 16)
    assert out[0].tolist() == [0, 3, 3, 3, 3, 3]


def test_negative_numbers_and_wild_state(wl):
    pages = wl.new_pages(4, 4, 10, 16, DEV)
    check(wl, pages, [-5, 0, -1, 3], [3, -7, 20, 1], 30, 16)
    # A state that no plan leaves: nothing is read or written outside the tensors.
    wild = wl.Pages(i32([[9, 1 << 30, -7, 3]] * 3), i32([900, -4, 2]), i32([5, -3, 1 << 30, 2]), i32([77]), 16)
    guard = wild.free.clone()
    out = wl.wl_batch_plan(wild, i32([0, 2147483647, 60]), i32([2147483647, 2147483647, 4]), 8)
    torch.cuda.synchronize()
    assert 0 <= int(wild.n_free) <= 4 and all(0 <= h <= 4 for h in wild.held.tolist()) and guard.shape == wild.free.shape
    assert out[0].tolist()[0] == 0 and max(out[0].tolist()) <= 8


def test_prompts_in_many_workgroups(wl):
    rng = random.Random(5)
    n_seq, page = 300, 16
    pages = wl.new_pages(n_seq, 700, 120000, page, DEV)
    fresh = [rng.randrange(1, 900) for _ in range(n_seq)]
    T = sum(fresh) + 37
    check(wl, pages, [0] * n_seq, fresh, T, page)
    past = [rng.randrange(0, f) for f in fresh]
    check(wl, pages, past, [rng.randrange(0, 600) for _ in fresh], T, page)


def test_replayed_in_a_graph(wl):
    """A captured plan follows the numbers in its tensors, replay by replay."""
    rng = random.Random(9)
    for n_seq, T in ((20, 64), (1200, 9000)):
        page = 16
        pages = wl.new_pages(n_seq, 40, 6000, page, DEV)
        past, fresh = i32([0] * n_seq), i32([1] * n_seq)
        call = wl.batch_plan_call(pages, past, fresh, T)
        g = torch.cuda.CUDAGraph()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
            call.launch()
        torch.cuda.current_stream().wait_stream(s)
        now = [0] * n_seq
        for _ in range(4):
            add = [rng.randrange(0, 30) for _ in now]
            table, held, free = lists(pages)
            ref = serve_ref.plan(table, held, free, len(free), now, add, T, page)
            past.copy_(i32(now)), fresh.copy_(i32(add))
            g.replay()
            torch.cuda.synchronize()
            assert [t.tolist() for t in call.out] == [list(r) for r in ref]
            assert lists(pages) == (table, held, free)
            now = [max(k - rng.randrange(0, 9), 0) for k in ref[1]]
