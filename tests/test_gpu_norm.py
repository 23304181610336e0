"""wl_norm_residual against its 64-bit definition."""
from __future__ import annotations

import pytest
import torch

import layer_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def wl():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    from linear_02_amd import wl as mod
    return mod


def draw(seed, *shape, dtype, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype).to(DEV)


def check(wl, x, y, post, pre, gate, eps=1e-6, offset=1.0, rs=1.0, bs=1.0, **kw):
    rx, rn, mx, mn = ref.norm(x, y, post, pre, gate, eps, offset, rs, bs)
    xo, no = wl.wl_norm_residual(x, y=y, post=post, pre=pre, gate=gate, eps=eps, offset=offset, res_scale=rs,
                                 branch_scale=bs, **kw)
    torch.cuda.synchronize()
    if xo is not None:
        ref.assert_near(xo, rx, ref.CHAIN * ref.EPS32 * mx, "x'")
    if no is not None:
        ref.assert_near(no, rn, 2 * ref.CHAIN * ref.EPS32 * mn, "n")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,d", [(1, 8), (1, 1152), (3, 512), (5, 520), (2, 1032), (4, 2048), (3, 2056), (37, 5376),
                                 (2, 6152), (1, 8200), (2, 16392), (1, 32768), (600, 64)])
def test_sizes(wl, T, d, dtype):
    print(f"norm T={T} d={d} {dtype}", flush=True)
    x, y = draw(1, T, d, dtype=dtype, std=3), draw(2, T, d, dtype=dtype)
    check(wl, x, y, draw(3, d, dtype=dtype, std=0.2), draw(4, d, dtype=dtype, std=0.2), draw(5, T, d, dtype=dtype), rs=0.75, bs=-0.5)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_parts(wl, dtype):
    T, d = 7, 1152
    x, y = draw(1, T, d, dtype=dtype), draw(2, T, d, dtype=dtype)
    post, pre, gate = (draw(s, d, dtype=dtype, std=0.3) for s in (3, 4, 5))
    wide = draw(6, T, 2 * d + 8, dtype=dtype)
    check(wl, x, None, None, pre, None)                                   # a norm alone
    check(wl, x, None, None, None, None, offset=0.0)                      # without weights
    check(wl, x, y, None, None, None)
    check(wl, x, y, post, None, gate, offset=0.0)                         # a gate for each channel
    check(wl, x, y, None, pre, wide[:, 8:d + 8])                          # rows of a wider matrix
    check(wl, x, y, post, pre, None, want_x=False)
    check(wl, x, y, post, pre, None, want_n=False)
    check(wl, x, y, post, pre, None, eps=0.5, rs=0.0)


def test_in_place_and_other_outputs(wl):
    dtype, T, d = torch.bfloat16, 9, 2304
    post, pre = draw(3, d, dtype=dtype), draw(4, d, dtype=dtype)
    for a, b in (("x", "y"), ("y", "x"), ("x", None), (None, "y")):
        t = dict(x=draw(1, T, d, dtype=dtype), y=draw(2, T, d, dtype=dtype))
        want = wl.wl_norm_residual(t["x"].clone(), y=t["y"].clone(), post=post, pre=pre)
        xo, no = wl.wl_norm_residual(t["x"], y=t["y"], post=post, pre=pre, x_out=t.get(a), n_out=t.get(b))
        torch.cuda.synchronize()
        assert torch.equal(xo, want[0]) and torch.equal(no, want[1]), (a, b)


def test_rows_of_zeros_infinities_and_nan_stay_apart(wl):
    T, d = 4, 1152
    x = draw(1, T, d, dtype=torch.float32)
    x[0], x[2, 5], x[3, 7] = 0, float("nan"), float("inf")
    _, n = wl.wl_norm_residual(x)
    torch.cuda.synchronize()
    assert (n[0] == 0).all() and torch.isfinite(n[1]).all()
    assert torch.isnan(n[2]).all() and torch.isnan(n[3, 7]) and (n[3, :7] == 0).all()


def test_empty_and_refusals(wl):
    dtype = torch.bfloat16
    x = draw(1, 4, 64, dtype=dtype)
    assert wl.wl_norm_residual(x[:0])[0].shape == (0, 64)
    for bad in (dict(y=draw(1, 4, 72, dtype=dtype)), dict(post=draw(1, 72, dtype=dtype)), dict(pre=draw(1, 64, dtype=torch.float32)),
                dict(gate=draw(1, 3, 64, dtype=dtype)), dict(y=x.cpu())):
        with pytest.raises(ValueError):
            wl.wl_norm_residual(x, **bad)
    y = torch.empty(8, 64, dtype=dtype, device=DEV)
    with pytest.raises(wl.WlError) as e:
        wl.wl_norm_residual(y[:4], x_out=y[1:5])
    assert e.value.status == wl.WL_ERR_INVALID_ARG and "overlaps" in str(e.value)


def test_graph_and_stream(wl):
    T, d = 3, 1152
    x, y = draw(1, T, d, dtype=torch.bfloat16), draw(2, T, d, dtype=torch.bfloat16)
    call = wl.norm_call(x, y=y, post=draw(3, d, dtype=torch.bfloat16))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call.launch()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call.launch()
    for seed in (5, 6, 7):
        x.copy_(draw(seed, T, d, dtype=torch.bfloat16))
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in call.out]
        call.launch()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, call.out))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("offset", [3e7, -0.3, 1.0])
def test_an_absent_weight_is_one(wl, dtype, offset):
    """Without weights the offset has no part: n is the bare norm for any offset."""
    x, y = draw(1, 5, 1152, dtype=dtype), draw(2, 5, 1152, dtype=dtype)
    z = ref.f64(x) + ref.f64(y)
    inv = 1 / (z.square().mean(1, keepdim=True) + 1e-6).sqrt()
    xo, no = wl.wl_norm_residual(x, y=y, offset=offset)
    torch.cuda.synchronize()
    ref.assert_near(no, z * inv, 2 * ref.CHAIN * ref.EPS32 * (ref.f64(x).abs() + ref.f64(y).abs()) * inv, "n")
    assert torch.equal(no, wl.wl_norm_residual(x, y=y)[1])
