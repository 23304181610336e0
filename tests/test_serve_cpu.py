"""The operations around a serving batch without a GPU: the library's own checks
refuse bad arguments before anything reaches HIP. Pointers are addresses that are never
read."""
from __future__ import annotations

import ctypes

import pytest

from tests.test_layer_cpu import P, at, struct


@pytest.fixture(scope="module")
def wl():
    import os

    from linear_02_amd import build
    if not os.path.exists(build.LIBRARY):
        build.build()
    from linear_02_amd import wl as mod
    return mod


BIG = 1 << 40


def refused(wl, status):
    return wl.lib.wl_last_error() != b"" or status == 0


PLAN = dict(table=P[0], held=P[1], free_pages=P[2], n_free=P[3], past=P[4], n_new=P[5], q_start=P[6], kv_len=P[7], seq=P[8],
            slot=P[9], T=40, n_seq=3, max_pages=8, n_pages=20, page=16)


@pytest.mark.parametrize("bad,status", [
    *[({k: None}, 1) for k in ("table", "held", "free_pages", "n_free", "past", "n_new", "q_start", "kv_len", "seq", "slot")],
    *[({k: PLAN[k] + 2}, 1) for k in ("table", "n_free", "past", "slot")],
    (dict(T=-1), 1), (dict(T=(1 << 24) + 1), 2), (dict(n_seq=0), 1), (dict(n_seq=65537), 2), (dict(max_pages=0), 1), (dict(n_pages=0), 1),
    (dict(page=8), 1), (dict(page=48), 1), (dict(page=2048), 1), (dict(max_pages=1 << 30), 1), (dict(max_pages=(1 << 26) + 1), 2),
    (dict(past=P[7]), 1), (dict(n_new=P[1] + 8), 1), (dict(seq=P[9] + 4), 1), (dict(kv_len=P[0] + 92), 1), (dict(held=P[2] + 76), 1)])
def test_plan_refuses(wl, bad, status):
    a = struct(wl.BatchPlanArgs, **(PLAN | bad))
    assert wl.lib.wl_batch_plan(ctypes.byref(a), P[20], BIG, None) == status and refused(wl, status)
    assert wl.lib.wl_batch_plan_workspace_bytes(ctypes.byref(a)) == 0


def test_plan_workspace(wl):
    a = struct(wl.BatchPlanArgs, **PLAN)
    need = wl.lib.wl_batch_plan_workspace_bytes
    assert need(ctypes.byref(a)) == 0
    b = struct(wl.BatchPlanArgs, **(PLAN | dict(n_seq=65536, T=1 << 20)))
    n = need(ctypes.byref(b))
    assert n > wl.SYNC_BYTES and wl.lib.wl_batch_plan(ctypes.byref(b), P[20], n - 1, None) == 4
    assert wl.lib.wl_batch_plan(ctypes.byref(b), None, n, None) == 4 and wl.lib.wl_batch_plan(ctypes.byref(b), P[20] + 16, n, None) == 1
    assert wl.lib.wl_batch_plan(ctypes.byref(b), P[9] - wl.SYNC_BYTES - 256, n, None) == 1      # over slot
    assert wl.lib.wl_batch_plan(None, None, 0, None) == 1 and need(None) == 0


def cache(wl, **kw):
    base = dict(rows=P[0], scale=P[1], table=P[2], n_pages=8, page=16, latent=512, rot=64, n_seq=3, max_pages=4, format=0)
    return struct(wl.LatentCacheStruct, **(base | kw))


def write_args(wl, pool, **kw):
    return struct(wl.LatentWriteArgs, **(dict(cache=at(pool), c=P[5], norm=P[6], q=P[7], q_out=P[8], seq=P[9], slot=P[10], T=4, n_q=2,
                                              nope=128, ldc=576, ldq=384, ldq_out=384) | kw))


def read_args(wl, c, **kw):
    return struct(wl.LatentReadArgs, **(dict(cache=at(c), seq=P[9], slot=P[10], out=P[8], T=4, ld=576) | kw))


def attention_args(wl, c, **kw):
    return struct(wl.LatentAttentionArgs, **(dict(cache=at(c), q=P[5], w=P[6], o=P[8], q_start=P[9], kv_len=P[10], T=4, n_q=2, nope=128,
                                                  value=128, ldq=384, ldo=256, max_q=2, max_kv=40, scale=0.125) | kw))


@pytest.mark.parametrize("bad,status", [
    (dict(rows=None), 1), (dict(rows=P[0] + 8), 1), (dict(table=None), 1), (dict(page=8), 1), (dict(page=24), 1), (dict(page=2048), 1),
    (dict(latent=0), 1), (dict(latent=384), 2), (dict(rot=0), 1), (dict(rot=48), 2), (dict(n_pages=0), 1), (dict(n_seq=0), 1),
    (dict(max_pages=0), 1), (dict(format=4), 2), (dict(format=1), 2), (dict(format=2), 2), (dict(format=3, scale=None), 1),
    (dict(format=3, scale=P[1] + 4), 1)])
def test_cache_refuses(wl, bad, status):
    c = cache(wl, **bad)
    assert wl.lib.wl_latent_write(ctypes.byref(write_args(wl, c)), None) == status
    assert wl.lib.wl_latent_read(ctypes.byref(read_args(wl, c)), None) == status
    a = attention_args(wl, c)
    assert wl.lib.wl_latent_attention(ctypes.byref(a), P[20], BIG, None) == status and refused(wl, status)
    assert wl.lib.wl_latent_attention_workspace_bytes(ctypes.byref(a)) == 0


@pytest.mark.parametrize("bad,rot,status", [
    (dict(cache=None), {}, 1), (dict(c=None), {}, 1), (dict(ldc=568), {}, 1), (dict(ldc=580), {}, 1), (dict(seq=None), {}, 1),
    (dict(slot=P[10] + 2), {}, 1), (dict(T=-1), {}, 1), (dict(T=(1 << 23)), {}, 2), (dict(n_q=-1), {}, 1), (dict(n_q=5000), {}, 1),
    (dict(nope=12), {}, 1), (dict(nope=264), {}, 1), (dict(nope=-8), {}, 1), (dict(norm=P[6] + 2), {}, 1), (dict(q=None), {}, 1),
    (dict(ldq=376), {}, 1), (dict(q_out=P[5]), {}, 1), (dict(q_out=P[0]), {}, 1), (dict(c=P[0]), {}, 1), (dict(q_out=P[7] + 16), {}, 1),
    (dict(dtype=1), {}, 2), (dict(dtype=9), {}, 2), ({}, dict(rot=32), 1), ({}, dict(style=2), 1), ({}, dict(freq=None), 1),
    ({}, dict(pos=P[13] + 2), 1)])
def test_write_refuses(wl, bad, rot, status):
    r = struct(wl.Rotary, **(dict(freq=P[12], pos=P[13], rot=64, style=0, scale=1.0) | rot))
    kept = cache(wl)
    a = write_args(wl, kept, **(dict(rotary=at(r)) | bad))
    assert wl.lib.wl_latent_write(ctypes.byref(a), None) == status and refused(wl, status)


@pytest.mark.parametrize("bad,status", [(dict(cache=None), 1), (dict(out=None), 1), (dict(out=P[8] + 8), 1), (dict(ld=568), 1),
                                        (dict(seq=None), 1), (dict(out=P[0]), 1), (dict(out=P[10]), 1), (dict(dtype=1), 2), (dict(T=-1), 1)])
def test_read_refuses(wl, bad, status):
    kept = cache(wl)
    a = read_args(wl, kept, **bad)
    assert wl.lib.wl_latent_read(ctypes.byref(a), None) == status and refused(wl, status)


@pytest.mark.parametrize("bad,status", [
    (dict(cache=None), 1), (dict(q=None), 1), (dict(o=None), 1), (dict(w=P[6] + 8), 1), (dict(q_start=None), 1), (dict(kv_len=None), 1),
    (dict(T=-1), 1), (dict(max_q=-1), 1), (dict(max_kv=-1), 1), (dict(max_kv=(1 << 30) + 1), 2), (dict(n_q=0), 1), (dict(n_q=5000), 2),
    (dict(nope=16), 1), (dict(value=40), 1), (dict(nope=288), 2), (dict(value=288), 2), (dict(w=None), 1), (dict(ldq=376), 1), (dict(ldo=252), 1),
    (dict(mask=3), 1), (dict(mask=-1), 1), (dict(window=-1), 1), (dict(window=4, mask=2), 1), (dict(mask=1), 1), (dict(form=3), 1),
    (dict(scale=float("nan")), 1), (dict(o=P[5]), 1), (dict(o=P[6]), 1), (dict(o=P[0]), 1), (dict(o=P[9] - 16), 1), (dict(dtype=1), 2),
    (dict(form=2, nope=96, value=96, ldq=384, ldo=256), 2), (dict(form=2, nope=128, value=64), 2)])
def test_attention_refuses(wl, bad, status):
    kept = cache(wl)
    a = attention_args(wl, kept, **bad)
    assert wl.lib.wl_latent_attention(ctypes.byref(a), P[20], BIG, None) == status and refused(wl, status)
    assert wl.lib.wl_latent_attention_workspace_bytes(ctypes.byref(a)) == 0


def test_attention_workspace(wl):
    c = cache(wl)
    a = attention_args(wl, c)
    f, n = wl.lib.wl_latent_attention, wl.lib.wl_latent_attention_workspace_bytes(ctypes.byref(a))
    assert n > wl.SYNC_BYTES and n % 256 == 0
    assert f(ctypes.byref(a), None, n, None) == 4 and f(ctypes.byref(a), P[20], n - 1, None) == 4 and f(ctypes.byref(a), P[20] + 8, n, None) == 1
    assert f(ctypes.byref(a), P[8] - wl.SYNC_BYTES - 256 & ~255, n, None) == 1      # over o
    fp32 = cache(wl, format=1)
    latent = attention_args(wl, fp32, w=None, nope=512, value=512, dtype=1, form=2)
    assert wl.lib.wl_latent_attention(ctypes.byref(latent), P[20], BIG, None) == 2
    crowd = cache(wl, n_seq=1 << 24)
    huge = attention_args(wl, crowd, n_q=128, ldq=128 * 192, ldo=128 * 128, max_q=4)
    assert f(ctypes.byref(huge), P[20], BIG, None) != 0


VERIFY = dict(target=P[0], draft=P[1], token=P[2], q_start=P[3], u=P[4], temperature=P[5], out=P[6], path=P[7], n_out=P[8], len=P[9],
              T=10, n_seq=2, vocab=1000, ld_target=1000, ld_draft=1001, max_q=5)


@pytest.mark.parametrize("bad,status", [
    *[({k: None}, 1) for k in ("target", "token", "q_start", "u", "out", "n_out")],
    (dict(target=P[0] + 2), 1), (dict(draft=P[1] + 8), 1), (dict(u=P[4] + 4), 1), (dict(path=P[7] + 2), 1), (dict(len=P[9] + 1), 1),
    (dict(temperature=P[5] + 2), 1), (dict(parent=P[10]), 1), (dict(draft=None, parent=P[10] + 2), 1), (dict(T=-1), 1), (dict(T=1 << 25), 2),
    (dict(n_seq=0), 1), (dict(vocab=0), 1), (dict(vocab=(1 << 30) + 1), 2), (dict(ld_target=999), 1), (dict(ld_draft=999), 1),
    (dict(T=1 << 22), 1), (dict(max_q=0), 1), (dict(max_q=1025), 1), (dict(kind=2), 1), (dict(dtype=5), 2), (dict(out=P[2]), 1),
    (dict(n_out=P[6] + 36), 1), (dict(len=P[8]), 1), (dict(path=P[6]), 1), (dict(out=P[0] + 64), 1), (dict(len=P[5] + 4), 1)])
def test_verify_refuses(wl, bad, status):
    a = struct(wl.VerifyArgs, **(VERIFY | bad))
    assert wl.lib.wl_verify_drafts(ctypes.byref(a), P[20], BIG, None) == status and refused(wl, status)
    assert wl.lib.wl_verify_drafts_workspace_bytes(ctypes.byref(a)) == 0


def test_verify_workspace(wl):
    a = struct(wl.VerifyArgs, **VERIFY)
    f, n = wl.lib.wl_verify_drafts, wl.lib.wl_verify_drafts_workspace_bytes(ctypes.byref(a))
    assert n > wl.SYNC_BYTES
    assert f(ctypes.byref(a), None, n, None) == 4 and f(ctypes.byref(a), P[20], n - 1, None) == 4 and f(ctypes.byref(a), P[20] + 8, n, None) == 1
    assert f(ctypes.byref(a), P[6] - wl.SYNC_BYTES - 256, n, None) == 1
    many = struct(wl.VerifyArgs, **(VERIFY | dict(n_seq=1 << 24, draft=None, q_start=1 << 40, temperature=1 << 41, n_out=1 << 42, len=1 << 43)))
    assert f(ctypes.byref(many), P[20], BIG, None) == 2 and b"workgroups" in wl.lib.wl_last_error()


def test_nothing_to_do(wl):
    c = cache(wl)
    assert wl.lib.wl_latent_write(ctypes.byref(struct(wl.LatentWriteArgs, cache=at(c))), None) == 0
    assert wl.lib.wl_latent_read(ctypes.byref(struct(wl.LatentReadArgs, cache=at(c))), None) == 0
    a = attention_args(wl, c, T=0, q=None, o=None, q_start=None)
    assert wl.lib.wl_latent_attention(ctypes.byref(a), None, 0, None) == 0 and wl.lib.wl_latent_attention_workspace_bytes(ctypes.byref(a)) == 0
    v = struct(wl.VerifyArgs, n_seq=1, vocab=5, max_q=1)
    assert wl.lib.wl_verify_drafts(ctypes.byref(v), None, 0, None) == 0 and wl.lib.wl_verify_drafts_workspace_bytes(ctypes.byref(v)) == 0
    for f in ("wl_latent_write", "wl_latent_read"):
        assert getattr(wl.lib, f)(None, None) == 1
    for f in ("wl_latent_attention", "wl_verify_drafts"):
        assert getattr(wl.lib, f)(None, None, 0, None) == 1 and getattr(wl.lib, f + "_workspace_bytes")(None) == 0


def test_steps_take_them(wl):
    ops = (wl.StepOp * 1)()
    c = cache(wl)
    for op, a in ((wl.OP_LATENT_WRITE, write_args(wl, c)), (wl.OP_LATENT_READ, read_args(wl, c)), (wl.OP_BATCH_PLAN, struct(wl.BatchPlanArgs, **PLAN))):
        ops[0].op, ops[0].args = op, ctypes.addressof(a)
        assert wl.lib.wl_step_ops_workspace_bytes(ops, 1) == wl.SYNC_BYTES
    for op, a, f in ((wl.OP_LATENT_ATTENTION, attention_args(wl, c), "wl_latent_attention"), (wl.OP_VERIFY_DRAFTS, struct(wl.VerifyArgs, **VERIFY), "wl_verify_drafts")):
        ops[0].op, ops[0].args = op, ctypes.addressof(a)
        assert wl.lib.wl_step_ops_workspace_bytes(ops, 1) == getattr(wl.lib, f + "_workspace_bytes")(ctypes.byref(a)) > wl.SYNC_BYTES
    for op in (8, 15, 21):
        ops[0].op = op
        assert wl.lib.wl_step_ops_workspace_bytes(ops, 1) == 0


@pytest.mark.parametrize("bad", [dict(n_out=P[6] + 2), dict(n_out=P[3] + 4), dict(n_out=P[5]), dict(n_out=P[9] - 4)])
def test_verify_of_no_rows_refuses(wl, bad):
    """With T == 0 the counts are still written."""
    a = struct(wl.VerifyArgs, **(VERIFY | dict(T=0) | bad))
    assert wl.lib.wl_verify_drafts(ctypes.byref(a), None, 0, None) == 1 and b"n_out" in wl.lib.wl_last_error()
    assert wl.lib.wl_verify_drafts_workspace_bytes(ctypes.byref(a)) == 0
