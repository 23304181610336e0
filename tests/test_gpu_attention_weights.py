"""How many bits wl_attention's weights keep on their way into the second product."""
from __future__ import annotations

import pytest
import torch

import layer_ref as ref
import weights_ref as wr

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, I8, E4 = torch.bfloat16, torch.float32, torch.int8, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def wl():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    from linear_02_amd import wl as mod
    return mod


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def worst(wl, fmt, d, n_seq, n_kv, group, rows, n, max_kv, held):
    """Largest error of a call of n_seq sequences of `rows` new tokens over n keys, all of
    them seen, as a share of the bar."""
    print(f"weights {fmt} d={d} {n_seq} x {rows} rows, {n_kv} x {group} heads, {n} keys, max_kv {max_kv}", flush=True)
    g = torch.Generator().manual_seed(rows + n)
    dtype, page = F32 if fmt == F32 else BF, 64
    pages = -(-n // page)
    table = torch.full((n_seq, max(max_kv // page, pages)), -1, dtype=torch.int32)
    table[:, :pages] = torch.arange(n_seq * pages, dtype=torch.int32).view(n_seq, pages)
    c = wl.new_cache(n_seq * pages, n_kv, page, d, table.to(DEV), fmt)
    for s in range(n_seq):
        k, v = (t.to(dtype).to(DEV) for t in wr.keys(g, n, n_kv, d))
        wl.wl_cache_write(c, k, v, ints([s] * n), torch.arange(n, dtype=torch.int32, device=DEV))
    q = wr.queries(g, n_seq * rows, n_kv * group, d).to(dtype).to(DEV)
    scale = d ** -0.5 / 2
    o = wl.wl_attention(q, c, ints([rows * s for s in range(n_seq + 1)]), ints([n] * n_seq), rows, max_kv, scale, mask="full")
    torch.cuda.synchronize()
    out = 0.0
    for s in range(n_seq):
        k, v, _ = ref.cache_rows(c, s, n)
        for h in range(n_kv * group):
            at = slice(s * rows, (s + 1) * rows), slice(h * d, (h + 1) * d)
            want = wr.attention(ref.f64(q)[at], k[:, h // group], v[:, h // group], scale, held)
            out = max(out, wr.excess(o[at], *want))
    return out


# d, sequences, key/value heads, query heads each, new tokens, keys
FEW = [(256, 1, 1, 4, 1, 1000), (128, 3, 2, 8, 4, 700), (64, 2, 1, 4, 8, 2048), (96, 1, 1, 1, 16, 64), (256, 2, 1, 4, 8, 3000),
       (128, 1, 2, 4, 16, 1024)]


@pytest.mark.parametrize("fmt", [BF, I8, E4, F32])
@pytest.mark.parametrize("case", range(len(FEW)))
@pytest.mark.parametrize("limit", [0, 1 << 17])
def test_up_to_64_rows_per_head_keep_the_remainder(wl, case, fmt, limit):
    d, n_seq, n_kv, group, rows, n = FEW[case]
    assert worst(wl, fmt, d, n_seq, n_kv, group, rows, n, max(limit, n), 0.0 if fmt == F32 else wr.TWO) <= 1


MORE = [(256, 1, 1, 4, 128, 512), (128, 1, 1, 2, 100, 1000), (64, 1, 2, 1, 200, 300), (256, 1, 1, 4, 48, 2048)]


@pytest.mark.parametrize("fmt", [BF, I8, E4])
@pytest.mark.parametrize("case", range(len(MORE)))
def test_the_limit_on_keys_does_not_decide_over_the_remainder(wl, case, fmt):
    """Few tiles of rows: the remainder is kept whether max_kv is the keys' number or far above it."""
    d, n_seq, n_kv, group, rows, n = MORE[case]
    for max_kv in (n, 1 << 17):
        assert worst(wl, fmt, d, n_seq, n_kv, group, rows, n, max_kv, wr.TWO) <= 1, max_kv
