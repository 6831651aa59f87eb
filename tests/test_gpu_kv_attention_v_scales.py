"""Rows whose softmax lies on pages of a small v scale, beside pages of a far
larger one that they give no weight, some of the weight, or do not see: the
value of such a row is that of its own keys (GPU only, both kernels).

The tolerance of an output value, with p_j the row's weights, A = sum_j p_j |v_j|
and C = 127 max_j p_j vs_j, the largest contribution the row's keys can make, all
of them from the keys that the row sees:
  scores    as in test_gpu_kv_attention (delta), and the page's v scale that enters
            them as two logarithms: values up to 2^6, an ulp (2^-18) each, their
            difference 2^-19 and its sums with score and maximum 2^-18 each:
            4.5 x 2^-18 ln 2 < 2^-16;
  weights   one rounding to fp16: 2^-11 of the weight, or 2^-25 of the largest
            contribution: n 2^-25 C;
  sums      (n + 8) 2^-24;
  output    its half step.
"""

import numpy as np
import pytest
import torch

import bit_ptq_vla_amd as q
import oracle
from test_gpu_kv_attention import DEV, DT, HALF_STEP, Cache, f64
from test_gpu_kv_attention_scales import batch_of

pytestmark = pytest.mark.gpu
SIZE = 4.0           # a query's elements; with codes near 100 and a scale of 0.01 a score is 4 sqrt(d)


def aligned(c, table, factor, d, seed=23):
    """Keys along one direction of +-1 (returned): codes 100 times it, times the
    page's factor, and noise.  A query along it scores 4 sqrt(d) factor."""
    g = np.random.default_rng(seed)
    way = np.where(g.random(d) < 0.5, -1.0, 1.0)
    page = c.host["k"].shape[2]
    for col, f in enumerate(factor):
        noise = g.integers(-3, 4, (page, d))
        c.host["k"][table[0, col], :] = np.clip(np.rint(100.0 * f * way) + noise, -127, 127).astype(np.int8)
    c.host["k_scale"][:] = 0.01
    return way


def check_rows(out, x, host, table, kv, hq, cap, dtype, rows):
    """rows of one causal sequence, each against its own keys."""
    pages, heads, page, d = host["k"].shape
    args = (table, [0, len(x)], [kv], hq, d ** -0.5, cap)
    ref = oracle.kv_attention(f64(x), host, *args).reshape(len(x), hq, d)
    a = oracle.kv_attention(f64(x), dict(host, v=np.abs(host["v"].astype(np.int16))), *args).reshape(len(x), hq, d)
    got = f64(out).reshape(len(x), hq, d)
    tiny = 2.0 ** -25 if dtype == "f16" else 0.0
    j = np.arange(kv)
    at = table[0, j // page].astype(np.int64)
    worst = 0.0
    for i in rows:
        seen = j <= kv - len(x) + i
        for h in range(hq):
            kh = h // (hq // heads)
            keys = host["k"][at[seen], kh, j[seen] % page].astype(np.float64) * host["k_scale"][at[seen], kh].astype(np.float64)[:, None]
            qi = f64(x)[i].reshape(hq, d)[h]
            s = keys @ qi * d ** -0.5
            b = np.max(np.abs(keys) @ np.abs(qi)) * d ** -0.5
            if cap:
                s = cap * np.tanh(s / cap)
                b = min(b, cap)
            p = np.exp(s - s.max())
            p /= p.sum()
            big = 127.0 * np.max(p * host["v_scale"][at[seen], kh].astype(np.float64))
            n = int(seen.sum())
            delta = (d + 8) * 2.0 ** -24 * b + (2.0 ** -21 * cap if cap else 0.0)
            rel = 2 * delta + 2.0 ** -16 + 2.0 ** -11 + (n + 8) * 2.0 ** -24
            tol = (rel * a[i, h] + HALF_STEP[dtype] * np.abs(ref[i, h])) * (1 + 2.0 ** -6) + n * 2.0 ** -25 * big + tiny
            err = np.abs(got[i, h] - ref[i, h])
            assert np.all(err <= tol), f"row {i} head {h}: {np.nanmax(err / np.maximum(tol, 1e-300)):.3g} of the tolerance"
            worst = max(worst, float(np.max(err / np.maximum(tol, 1e-300))))
    return worst


@pytest.mark.parametrize("wide", [False, True], ids=["rows16", "prompts"])
@pytest.mark.parametrize("octaves", [8, 14, 20, 26, 40, 60])
@pytest.mark.parametrize("dtype,hq,hkv,d,page,cap,large", [
    ("bf16", 1, 1, 128, 16, 0.0, 1), ("bf16", 1, 1, 128, 16, 0.0, 6), ("f16", 2, 1, 64, 16, 0.0, 3),
    ("f16", 2, 2, 256, 32, 50.0, 4), ("bf16", 1, 1, 64, 64, 50.0, 0),
])
def test_a_large_page_without_weight(dtype, hq, hkv, d, page, cap, large, octaves, wide):
    """One page with a v scale 2^octaves of the others' and keys that point away:
    rows in front of it do not see it, rows behind it give it e^-60 or less."""
    cols = 9 if page < 64 else 4
    c = Cache(cols + 2, page, hkv, d)
    table = c.table(1, cols)
    factor = [1.0] * cols
    factor[large] = -1.0
    way = aligned(c, table, factor, d)
    c.host["v_scale"][:] = 0.25
    c.host["v_scale"][table[0, large]] = 0.25 * 2.0 ** octaves
    c.upload()
    kv = cols * page - 5
    g = torch.Generator().manual_seed(3)
    x = (torch.from_numpy(np.tile(way, hq)) * SIZE * (1 + 0.1 * torch.rand((kv, hq * d), generator=g))).to(DT[dtype])
    out = q.qlin_kv_attention(x.to(DEV), c.cache, batch_of(table, [0, kv], [kv], page, wide), hq, softcap=cap)
    torch.cuda.synchronize()
    rows = [i for i in range(kv) if not (large == 0 and i < page)]         # rows that see a key of the others
    check_rows(out, x, c.host, table, kv, hq, cap, dtype, rows)


@pytest.mark.parametrize("wide", [False, True], ids=["rows16", "prompts"])
@pytest.mark.parametrize("octaves", [6, 10, 16, 30])
@pytest.mark.parametrize("large", [0, 2, 5])
def test_a_large_page_with_as_large_a_part(octaves, large, wide):
    """The large page's keys score octaves ln 2 below: both parts of the value count."""
    d, page, cols = 128, 16, 7
    c = Cache(cols + 1, page, 1, d)
    table = c.table(1, cols)
    factor = [1.0] * cols
    factor[large] = 1.0 - octaves * np.log(2.0) / (SIZE * d ** 0.5)
    way = aligned(c, table, factor, d)
    c.host["v_scale"][:] = 2.0 ** -5
    c.host["v_scale"][table[0, large]] = 2.0 ** (octaves - 5)
    c.upload()
    kv = cols * page
    x = torch.from_numpy(np.tile(way * SIZE, (kv, 1))).to(torch.bfloat16)
    out = q.qlin_kv_attention(x.to(DEV), c.cache, batch_of(table, [0, kv], [kv], page, wide), 1)
    torch.cuda.synchronize()
    check_rows(out, x, c.host, table, kv, 1, 0.0, "bf16", range(kv))


@pytest.mark.parametrize("octaves", [16, 40])
@pytest.mark.parametrize("large", [0, 37, 120])
def test_large_pages_over_split_keys(large, octaves):
    """Two tokens over split keys: the large page in a split, or a wave, of its own."""
    hq, hkv, d, page, cols = 2, 1, 128, 16, 160
    c = Cache(cols + 1, page, hkv, d)
    table = c.table(1, cols)
    factor = [1.0 - 0.01 * (i % 7) for i in range(cols)]
    factor[large] = -1.0
    way = aligned(c, table, factor, d)
    c.host["v_scale"][:] = 2.0 ** -6
    c.host["v_scale"][table[0, large]] = 2.0 ** (octaves - 6)
    c.upload()
    kv = cols * page - 9
    x = torch.from_numpy(np.tile(way * SIZE, (2, hq))).to(torch.bfloat16)
    b = batch_of(table, [0, 2], [kv], page, False)
    assert q.kv_attention_workspace_bytes(c.cache, b, hq) > 0
    out = q.qlin_kv_attention(x.to(DEV), c.cache, b, hq)
    torch.cuda.synchronize()
    check_rows(out, x, c.host, table, kv, hq, 0.0, "bf16", range(2))


@pytest.mark.parametrize("wide", [False, True], ids=["rows16", "prompts"])
def test_pages_of_scale_zero(wide):
    """Rows that see only pages of v scale 0 (whatever their codes) give 0; rows
    behind them count their keys in the sum."""
    d, page, cols = 64, 16, 8
    c = Cache(cols + 1, page, 1, d)
    table = c.table(1, cols)
    c.host["v_scale"][table[0, [0, 1, 4]]] = 0.0
    c.upload()
    kv = cols * page
    x = torch.from_numpy(np.random.default_rng(2).standard_normal((kv, d))).to(torch.bfloat16)
    out = q.qlin_kv_attention(x.to(DEV), c.cache, batch_of(table, [0, kv], [kv], page, wide), 1)
    torch.cuda.synchronize()
    assert not out[:2 * page].any()
    check_rows(out, x, c.host, table, kv, 1, 0.0, "bf16", range(2 * page, kv))
