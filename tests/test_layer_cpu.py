"""The operations between the projections without a GPU: the library's own
checks refuse bad arguments before anything reaches HIP, and the rotary
frequencies are the formulas'. Pointers are addresses that are never read."""
from __future__ import annotations

import ctypes
import math

import pytest

P = [0x10000000 * (i + 1) for i in range(30)]


@pytest.fixture(scope="module")
def wl():
    import os

    from linear_02_amd import build
    if not os.path.exists(build.LIBRARY):
        build.build()
    from linear_02_amd import wl as mod
    return mod


def struct(t, **kw):
    s = t()
    for k, v in kw.items():
        assert any(f[0] == k for f in t._fields_), k
        setattr(s, k, v)
    return s


def at(s):
    return None if s is None else ctypes.addressof(s)


def cache(wl, **kw):
    base = dict(k=P[0], v=P[1], k_scale=P[2], v_scale=P[3], table=P[4], n_pages=8, page=16, n_kv=2, d=64, n_seq=3,
                max_pages=4, format=0)
    return struct(wl.CacheStruct, **(base | kw))


def rotary(wl, **kw):
    return struct(wl.Rotary, **(dict(freq=P[5], pos=P[6], rot=64, style=0, scale=1.0) | kw))


NORM = dict(x=P[7], y=P[8], post=P[9], pre=P[10], gate=P[11], x_out=P[12], n_out=P[13], T=4, d=64, gate_ld=64, dtype=0)


@pytest.mark.parametrize("bad,status", [
    (dict(x=None), 1), (dict(x=P[7] + 8), 1), (dict(d=0), 1), (dict(d=60), 1), (dict(d=40000), 2), (dict(dtype=2), 2),
    (dict(T=-1), 1), (dict(x_out=None, n_out=None), 1), (dict(gate_ld=56), 1), (dict(gate_ld=68), 1),
    (dict(post=P[9] + 2), 1), (dict(n_out=P[12]), 1), (dict(x_out=P[11]), 1), (dict(x_out=P[7] + 128), 1),
    (dict(n_out=P[10] - 64), 1), (dict(T=1 << 25), 1)])
def test_norm_refuses(wl, bad, status):
    a = struct(wl.NormArgs, **(NORM | bad))
    assert wl.lib.wl_norm_residual(ctypes.byref(a), None) == status and wl.lib.wl_last_error() != b""


def test_nothing_to_do(wl):
    for t, f, kw in ((wl.NormArgs, "wl_norm_residual", dict(d=64, x_out=P[1])), (wl.RopeArgs, "wl_rope", dict(d=64, n_q=1))):
        assert getattr(wl.lib, f)(ctypes.byref(struct(t, **kw)), None) == 0
    c = cache(wl)
    assert wl.lib.wl_cache_write(ctypes.byref(struct(wl.CacheWriteArgs, cache=at(c))), None) == 0
    assert wl.lib.wl_cache_read(ctypes.byref(struct(wl.CacheReadArgs, cache=at(c), k_out=P[9])), None) == 0
    a = struct(wl.AttentionArgs, cache=at(c), n_q=2, scale=1.0)
    assert wl.lib.wl_attention(ctypes.byref(a), None, 0, None) == 0
    for f in ("wl_norm_residual", "wl_rope", "wl_cache_write", "wl_cache_read"):
        assert getattr(wl.lib, f)(None, None) == 1
    assert wl.lib.wl_attention(None, None, 0, None) == 1 and wl.lib.wl_attention_workspace_bytes(None) == 0


@pytest.mark.parametrize("bad,rot,status", [
    (dict(q=None), {}, 1), (dict(k_out=None), {}, 1), (dict(n_q=0, n_k=0), {}, 1), (dict(n_q=-1), {}, 1), (dict(d=60), {}, 1),
    (dict(d=264), {}, 2), (dict(ldq=120), {}, 1), (dict(ldk_out=132), {}, 1), (dict(dtype=7), {}, 2),
    (dict(q_out=P[8]), {}, 1),                       # on top of k
    (dict(q_out=P[7], ldq_out=256), {}, 1),          # on top of q, other rows
    (dict(q_out=P[7] + 16), {}, 1), (dict(k_out=P[9]), {}, 1),
    ({}, dict(rot=0), 1), ({}, dict(rot=12), 1), ({}, dict(rot=72), 1), ({}, dict(style=2), 1), ({}, dict(freq=None), 1),
    ({}, dict(freq=P[5] + 4), 1), ({}, dict(pos=None), 1)])
def test_rope_refuses(wl, bad, rot, status):
    r = rotary(wl, **rot)
    a = struct(wl.RopeArgs, **(dict(q=P[7], k=P[8], q_out=P[9], k_out=P[10], rotary=at(r), T=4, n_q=2, n_k=2, d=64, ldq=128,
                                    ldk=128, ldq_out=128, ldk_out=128) | bad))
    assert wl.lib.wl_rope(ctypes.byref(a), None) == status and wl.lib.wl_last_error() != b""


CACHES = [(dict(k=None), 1), (dict(v=P[1] + 8), 1), (dict(table=None), 1), (dict(page=8), 1), (dict(page=48), 1),
          (dict(page=2048), 1), (dict(d=40), 1), (dict(d=272), 2), (dict(n_pages=0), 1), (dict(n_kv=0), 1), (dict(n_seq=0), 1),
          (dict(max_pages=0), 1), (dict(format=4), 2), (dict(format=1), 2), (dict(format=2, k_scale=None), 1),
          (dict(format=3, v_scale=P[3] + 4), 1)]


def write_args(wl, c, **kw):
    return struct(wl.CacheWriteArgs, **(dict(cache=at(c), k=P[7], v=P[8], q=P[9], q_out=P[10], seq=P[11], slot=P[12], T=4,
                                             n_q=4, ldk=128, ldv=128, ldq=256, ldq_out=256) | kw))


def attention_args(wl, c, **kw):
    return struct(wl.AttentionArgs, **(dict(cache=at(c), q=P[9], o=P[10], q_start=P[11], kv_len=P[12], T=4, n_q=4, ldq=256,
                                            ldo=256, max_q=2, max_kv=40, scale=0.125) | kw))


@pytest.mark.parametrize("bad,status", CACHES)
def test_cache_refuses(wl, bad, status):
    c = cache(wl, **bad)
    r = struct(wl.CacheReadArgs, cache=at(c), seq=P[11], slot=P[12], k_out=P[13], v_out=P[14], T=4, ldk=128, ldv=128)
    assert wl.lib.wl_cache_write(ctypes.byref(write_args(wl, c)), None) == status
    assert wl.lib.wl_cache_read(ctypes.byref(r), None) == status
    assert wl.lib.wl_attention(ctypes.byref(attention_args(wl, c)), P[20], 1 << 40, None) == status


@pytest.mark.parametrize("bad,status", [
    (dict(cache=None), 1), (dict(k=None), 1), (dict(seq=None), 1), (dict(slot=P[12] + 2), 1), (dict(ldv=64), 1), (dict(n_q=-1), 1),
    (dict(q_out=P[7]), 1), (dict(q_out=P[0]), 1), (dict(k=P[0]), 1), (dict(v=P[1] + 64), 1), (dict(dtype=1), 2), (dict(T=-2), 1),
    (dict(q_out=P[4] - 16), 1)])
def test_cache_write_refuses(wl, bad, status):
    c = cache(wl)
    assert wl.lib.wl_cache_write(ctypes.byref(write_args(wl, c, **bad)), None) == status and wl.lib.wl_last_error() != b""


def test_cache_write_refuses_pools_that_meet(wl):
    assert wl.lib.wl_cache_write(ctypes.byref(write_args(wl, c := cache(wl, v=P[0] + 64))), None) == 1
    assert wl.lib.wl_cache_write(ctypes.byref(write_args(wl, c := cache(wl, format=2, v_scale=P[2]))), None) == 1
    del c


@pytest.mark.parametrize("bad,status", [
    (dict(k_out=None, v_out=None), 1), (dict(v_out=P[13]), 1), (dict(k_out=P[0]), 1), (dict(ldk=120), 1), (dict(seq=None), 1)])
def test_cache_read_refuses(wl, bad, status):
    c = cache(wl)
    a = struct(wl.CacheReadArgs, **(dict(cache=at(c), seq=P[11], slot=P[12], k_out=P[13], v_out=P[14], T=4, ldk=128, ldv=128) | bad))
    assert wl.lib.wl_cache_read(ctypes.byref(a), None) == status and wl.lib.wl_last_error() != b""


@pytest.mark.parametrize("bad,status", [
    (dict(q=None), 1), (dict(o=P[10] + 4), 1), (dict(n_q=3), 1), (dict(n_q=0), 1), (dict(ldo=128), 1), (dict(mask=3), 1),
    (dict(window=-1), 1), (dict(mask=2, window=5), 1), (dict(mask=1), 1), (dict(mask=1, tree_words=1), 1), (dict(T=-1), 1),
    (dict(max_q=-1), 1), (dict(max_kv=-1), 1), (dict(scale=float("nan")), 1), (dict(kv_len=None), 1), (dict(o=P[0]), 1),
    (dict(o=P[9] + 512), 1), (dict(dtype=1), 2), (dict(mask=1, tree=P[10], tree_words=1), 1)])
def test_attention_refuses(wl, bad, status):
    c = cache(wl)
    a = attention_args(wl, c, **bad)
    assert wl.lib.wl_attention(ctypes.byref(a), P[20], 1 << 40, None) == status and wl.lib.wl_last_error() != b""
    assert wl.lib.wl_attention_workspace_bytes(ctypes.byref(a)) == 0


def test_sizes_beyond_a_launch_are_refused(wl):
    a = struct(wl.NormArgs, **(NORM | dict(T=(1 << 24) + 1, d=8, gate_ld=8, x_out=P[26], n_out=None)))
    assert wl.lib.wl_norm_residual(ctypes.byref(a), None) == 2 and b"T=" in wl.lib.wl_last_error()
    c = cache(wl, n_kv=1, d=16)
    w = write_args(wl, c, T=(1 << 24) + 1, n_q=0, ldk=16, ldv=16)
    assert wl.lib.wl_cache_write(ctypes.byref(w), None) == 2
    a = attention_args(wl, cache(wl), max_kv=(1 << 30) + 1)
    assert wl.lib.wl_attention(ctypes.byref(a), P[20], 1 << 40, None) == 2
    big = cache(wl, n_seq=1 << 23)                             # 2^23 sequences of 2 key/value heads
    a = attention_args(wl, big, q_start=P[24], kv_len=P[28])
    assert wl.lib.wl_attention(ctypes.byref(a), P[20], 1 << 40, None) == 2
    assert b"workgroups" in wl.lib.wl_last_error()


def test_two_to_the_32_threads_are_refused(wl):
    """2^23 workgroups of eight waves, which codes at 129 to 256 rows per head take."""
    c = cache(wl, n_kv=1, d=16, n_seq=1 << 23, max_pages=1, format=2, k=1 << 36, v=1 << 37, k_scale=1 << 38, v_scale=1 << 39,
              table=1 << 40)
    a = attention_args(wl, c, q=1 << 41, o=1 << 42, q_start=1 << 43, kv_len=1 << 44, T=200, max_q=200, n_q=1, ldq=16, ldo=16)
    assert wl.lib.wl_attention(ctypes.byref(a), None, 0, None) == 2, wl.lib.wl_last_error()
    assert b"workgroups" in wl.lib.wl_last_error()


def test_step_ops_refuse(wl):
    ops = (wl.StepOp * 1)()
    h = ctypes.c_void_p()
    make = lambda n=1, ws=P[20], size=1 << 40: wl.lib.wl_step_create_ops(ops, n, ws, size, ctypes.byref(h))  # noqa: E731
    assert make() == 1                                         # no arguments
    a = struct(wl.NormArgs, **NORM)
    ops[0].op, ops[0].args = 9, ctypes.addressof(a)
    assert make() == 1 and wl.lib.wl_step_ops_workspace_bytes(ops, 1) == 0
    ops[0].op = wl.OP_NORM
    assert wl.lib.wl_step_ops_workspace_bytes(ops, 1) == wl.SYNC_BYTES
    assert make(n=0) == 1 and make(size=100) == 4 and make(ws=P[20] + 4) == 1
    call = wl.Call()
    ops[0].op, ops[0].args = wl.OP_LINEAR, ctypes.addressof(call)
    call.op = wl.OP_QKV
    assert make() == 1
    assert wl.lib.wl_step_create_ops(None, 1, P[20], 1 << 40, ctypes.byref(h)) == 1 and h.value is None


def test_frequencies(wl):
    rot, base = 64, 10000.0
    f = [base ** (-2 * e / rot) for e in range(rot // 2)]
    got = lambda **kw: wl.rope_frequencies(rot, base, device="cpu", **kw)  # noqa: E731
    near = lambda a, b: all(abs(x - y) <= 1e-14 * abs(y) for x, y in zip(a.tolist(), b))  # noqa: E731
    assert near(got()[0], f) and got()[1] == 1.0
    assert near(got(scaling="linear", factor=8.0)[0], [v / 8 for v in f])
    slow = got(scaling="base", factor=8.0)[0]
    assert slow[0] == 1.0 and abs(float(slow[-1]) * 8 / f[-1] - 1) < 1e-12
    part, scale = got(scaling="parts", factor=8.0, original=4096.0, slow=1.0, fast=32.0)
    turns = [4096 * v / (2 * math.pi) for v in f]
    assert abs(scale - (0.1 * math.log(8) + 1)) < 1e-7
    for v, p, n in zip(f, part.tolist(), turns):
        assert abs(p - (v if n >= 32 else v / 8 if n <= 1 else v * (n - 1) / 31 + v / 8 * (32 - n) / 31)) <= 1e-14 * v
    for bad in (dict(rot=12), dict(rot=0), dict(rot=264), dict(rot=64, base=1.0), dict(rot=64, scaling="linear", factor=0.5),
                dict(rot=64, scaling="parts", fast=1.0), dict(rot=64, scaling="parts", original=0.0), dict(rot=64, base=float("nan"))):
        with pytest.raises(wl.WlError):
            wl.rope_frequencies(device="cpu", **bad)
    with pytest.raises(ValueError):
        wl.rope_frequencies(64, scaling="other", device="cpu")
