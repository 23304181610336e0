"""What the binding keeps alive: device memory whose addresses calls, steps and captured
graphs hold. Without a GPU, by weak references to host tensors in their place."""
from __future__ import annotations

import ctypes
import gc
import weakref

import pytest
import torch


@pytest.fixture(scope="module")
def wl():
    import os

    from linear_02_amd import build
    if not os.path.exists(build.LIBRARY):
        build.build()
    from linear_02_amd import wl as mod
    return mod


@pytest.fixture
def no_device(wl, monkeypatch):
    """Steps are checked and made on the host alone; rows of x without a look at its device."""
    for f in ("wl_step_create", "wl_step_create_ops"):
        monkeypatch.setattr(wl.lib, f, lambda *a: 0)
    monkeypatch.setattr(wl, "_io", lambda x, *a: x.shape[0])


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def theta():
    return dict(W0=bf16(64, 64), s=torch.ones(64), U=bf16(64, 4), V=bf16(64, 4), d_in=64, d_out=64, r=4)


def watch(*tensors):
    return [weakref.ref(t) for t in tensors]


def alive(refs):
    gc.collect()
    return [r() is not None for r in refs]


def norm(wl):
    x, out = bf16(4, 64), bf16(4, 64)
    args = wl.NormArgs(x=x.data_ptr(), n_out=out.data_ptr(), T=4, d=64)
    return wl.OpCall(wl.OP_NORM, None, args, (None, out), x.device, (x,)), watch(x, out)


def test_a_layer_step_outlives_the_list_it_was_made_from(wl, no_device):
    call, refs = norm(wl)
    th, x, y = theta(), bf16(4, 64), bf16(4, 64)
    refs += watch(x, y, th["W0"], th["s"], th["U"], th["V"])
    thetas = [th]
    calls = [call, (wl.OP_LINEAR, thetas, x, y)]
    step = wl.LayerStep(calls, ws=torch.zeros(1, dtype=torch.uint8))
    args = ctypes.addressof(call.args)
    calls.clear(), thetas.clear(), th.clear()
    call.args = call.out = call.keep = None
    del call, x, y
    assert all(alive(refs))
    assert args in [ctypes.addressof(a) for k in step._keep if isinstance(k, tuple) for a in k if isinstance(a, ctypes.Structure)]
    del step
    assert not any(alive(refs))


def test_a_step_outlives_the_thetas_it_was_made_from(wl, no_device):
    th, x, y = theta(), bf16(4, 64), bf16(4, 64)
    refs = watch(x, y, th["W0"], th["s"], th["U"], th["V"])
    thetas = [th]
    calls = [(wl.OP_LINEAR, thetas, x, y)]
    step = wl.Step(calls, ws=torch.zeros(1, dtype=torch.uint8))
    calls.clear(), thetas.clear(), th.clear()
    del x, y
    assert all(alive(refs))
    del step
    assert not any(alive(refs))


class OnDevice:
    """A host tensor that says it is on the device."""

    def __init__(self, t):
        self.t = t

    is_cuda, device = True, torch.device("cuda", 0)

    def get_device(self):
        return 0

    def new_empty(self, *a, **kw):
        return OnDevice(self.t.new_empty(*a, **kw))

    def __getattr__(self, name):
        return getattr(self.t, name)


def test_calls_keep_the_cache_and_frequencies_they_were_made_with(wl):
    def dev(*shape, dtype=torch.bfloat16):
        return OnDevice(torch.zeros(shape, dtype=dtype))

    k, v, table = dev(2, 1, 16, 64), dev(2, 1, 16, 64), dev(1, 2, dtype=torch.int32)
    freq = dev(32, dtype=torch.float64)
    refs = watch(k, v, table, freq)
    cache, rope = wl.Cache(k, v, table), wl.Rope(freq)
    i32 = dict(dtype=torch.int32)
    row = dev(3, 64)
    calls = [wl.cache_write_call(cache, row, dev(3, 64), dev(3, **i32), dev(3, **i32), q=dev(3, 64), rope=rope),
             wl.cache_read_call(cache, dev(3, **i32), dev(3, **i32)),
             wl.attention_call(row, cache, dev(2, **i32), dev(1, **i32), 3, 3, 1.0),
             wl.rope_call(row, None, dev(3, **i32), rope, 64)]
    cache.k = cache.v = cache.table = rope.freq = None
    struct = ctypes.addressof(cache.struct)
    assert [c.args.cache == struct for c in calls[:3]] == [True] * 3
    del k, v, table, freq, cache, rope
    for _ in range(3):                      # each of the three that hold the cache, alone at last
        assert all(alive(refs))
        calls.pop(0)
    assert alive(refs) == [False, False, False, True]
    calls.clear()
    assert not any(alive(refs))


@pytest.fixture
def streams(wl, monkeypatch):
    """Host memory for workspaces, on a stream and in a capture of the test's choice."""
    class At:
        stream, capture, prepared = 1, None, 0

    def prepared(nbytes, device):
        At.prepared += 1
        return torch.empty(nbytes, dtype=torch.uint8)

    monkeypatch.setattr(wl, "_raw_stream", lambda index: At.stream)
    monkeypatch.setattr(wl, "_capture", lambda stream: At.capture, raising=False)
    monkeypatch.setattr(wl, "_bytes", lambda n, device: torch.empty(n, dtype=torch.uint8), raising=False)
    monkeypatch.setattr(wl, "new_workspace", prepared)
    return At


CUDA0 = torch.device("cuda", 0)


def test_a_capture_has_a_workspace_of_its_own(wl, streams):
    w = wl.Workspace()
    eager = w.get(CUDA0, 1000)
    assert w.get(CUDA0, 500) is eager and streams.prepared == 1
    streams.capture = 7
    first = w.get(CUDA0, 1000)
    assert first is not eager and streams.prepared == 2        # prepared by a node of the graph
    assert w.get(CUDA0, 900) is first and streams.prepared == 2
    streams.stream = 2                                         # another stream in the same capture
    beside = w.get(CUDA0, 1000)
    assert beside is not first and streams.prepared == 3
    streams.stream, streams.capture = 1, 8                     # another graph on the same stream
    second = w.get(CUDA0, 1000)
    assert second is not first and streams.prepared == 4
    large = w.get(CUDA0, 1 << 21)
    assert large.numel() >= 1 << 21 and w.get(CUDA0, 1000) is large
    streams.capture = None
    assert w.get(CUDA0, 1000) is eager and streams.prepared == 5


def test_captured_attention_takes_memory_of_its_graph(wl, streams):
    got = []

    def launched(args, ws, nbytes, stream):
        got.append((ws, nbytes))
        return 0

    cache = wl.CacheStruct(k=1 << 20, v=1 << 30, table=1 << 34, n_pages=64, page=64, n_kv=1, d=64, n_seq=1, max_pages=64)
    args = wl.AttentionArgs(cache=ctypes.addressof(cache), q=1 << 35, o=1 << 36, q_start=1 << 37, kv_len=1 << 38, T=1, n_q=1, ldq=64,
                            ldo=64, max_q=1, max_kv=4096, scale=1.0)
    need = int(wl.lib.wl_attention_workspace_bytes(args))
    assert need > 0
    call = wl.OpCall(wl.OP_ATTENTION, launched, args, None, CUDA0, ())
    shared = wl.WORKSPACE.get(CUDA0, need)
    prepared = streams.prepared
    call._launch()
    assert got[-1][0] == shared.data_ptr() and streams.prepared == prepared
    streams.capture = 3
    call._launch()
    assert got[-1][0] != shared.data_ptr() and got[-1][1] >= need and streams.prepared == prepared
    call.ws = torch.empty(need, dtype=torch.uint8)
    call._launch()
    assert got[-1][0] == call.ws.data_ptr()
    wl.WORKSPACE._bufs.pop((0, streams.stream))


class Elsewhere:
    """A tensor of another device."""

    def __init__(self, t, index):
        self.t, self.device = t, torch.device("cuda", index)

    def __getattr__(self, name):
        return getattr(self.t, name)


def test_a_step_is_made_and_launched_on_its_calls_device(wl, no_device, monkeypatch):
    """One device per step, which need not be the current one."""
    at, seen = [0], []

    class On:
        def __init__(self, device):
            self.index = device.index

        def __enter__(self):
            at.append(self.index)

        def __exit__(self, *a):
            at.pop()

    monkeypatch.setattr(wl.torch.cuda, "current_device", lambda: at[-1])
    monkeypatch.setattr(wl.torch.cuda, "device", On)
    monkeypatch.setattr(wl, "_raw_stream", lambda index: index)
    for f in ("wl_step_create", "wl_step_create_ops", "wl_step_launch"):
        monkeypatch.setattr(wl.lib, f, lambda *a, f=f: seen.append((f, at[-1])) or 0)
    ws = torch.zeros(1, dtype=torch.uint8)

    def calls(*indexes):
        return [(wl.OP_LINEAR, [theta()], Elsewhere(bf16(4, 64), i), bf16(4, 64)) for i in indexes]

    for make, f in ((wl.Step, "wl_step_create"), (wl.LayerStep, "wl_step_create_ops")):
        for index in (0, 1):
            make(calls(index, index), ws=ws).launch()
            assert seen == [(f, index), ("wl_step_launch", index)] and at == [0]
            seen.clear()
        with pytest.raises(ValueError, match="call 1"):
            make(calls(0, 1), ws=ws)
        assert not seen
