"""The attention kernel for prompts on short inputs (GPU only).  It is taken by
the bounds a call states (rows and keys), so a batch whose bounds are far above
its lengths reaches it with any size: the cases of the general tests, run again
under such bounds, and sequences whose keys are split over several blocks.
Tolerances as there.
"""

import numpy as np
import pytest
import torch

import bit_ptq_vla_amd as q
import test_gpu_kv_attention as base
from test_gpu_kv_attention import CASES, DEV, Cache, check, i32, queries

pytestmark = pytest.mark.gpu
ROWS, KEYS = 200, 1 << 18


@pytest.fixture
def wide(monkeypatch):
    def batch_of(table, q_start, kv_len, page, prefix=None, max_kv=None):
        table = np.asarray(table)
        bounds = np.full((len(table), KEYS // page), -7, dtype=np.int32)      # no page: never to be read
        bounds[:, :table.shape[1]] = table
        return q.KvBatch(i32(bounds), i32(q_start), i32(kv_len), max_q=max(ROWS, int(np.diff(q_start).max())),
                         max_kv=KEYS, prefix_len=None if prefix is None else i32(prefix))

    monkeypatch.setattr(base, "batch_of", batch_of)


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}-{c[1]}-{c[2]}-{c[3]}-p{c[4]}-cap{c[5]}-{len(c[6])}")
def test_attention(case, wide):
    base.test_attention(case)


def test_rows_that_see_nothing_and_damaged_pages(wide):
    base.test_rows_that_see_nothing_and_damaged_pages()


def test_queries_of_any_size(wide):
    base.test_queries_of_any_size()


def test_scales_of_very_different_pages(wide):
    base.test_scales_of_very_different_pages()


@pytest.mark.parametrize("rows", [2, 140])
@pytest.mark.parametrize("scale", [0.0, -0.2])
def test_zero_scales_and_signs(rows, scale, wide):
    base.test_zero_scales_and_signs(rows, scale)


def test_cache_past_32_bit_offsets(wide):
    base.test_cache_past_32_bit_offsets()


@pytest.mark.parametrize("dtype,hq,hkv,d,page,rows,kv,bound,cap", [
    ("bf16", 4, 4, 256, 64, 150, 2600, 16384, 30.0),
    ("f16", 8, 4, 128, 32, 130, 1500, 16384, 0.0),
    ("bf16", 4, 4, 64, 16, 260, 4500, 65536, 0.0),
])
def test_split_keys(dtype, hq, hkv, d, page, rows, kv, bound, cap):
    cols = -(-kv // page)
    c = Cache(cols + 1, page, hkv, d, seed=21)
    table = np.full((1, bound // page), -1, dtype=np.int32)
    table[:, :cols] = c.table(1, cols)
    x = queries(rows, hq * d, dtype, f"split{kv}")
    b = q.KvBatch(i32(table), i32([0, rows]), i32([kv]), max_q=rows, max_kv=bound)
    assert q.kv_attention_workspace_bytes(c.cache, b, hq) > 0
    out = q.qlin_kv_attention(x.to(DEV), c.cache, b, hq, softcap=cap)
    torch.cuda.synchronize()
    check(out, x, c, table, [0, rows], [kv], hq, d ** -0.5, cap, None, dtype)
    one = torch.empty_like(out)
    st = q.load().qlin_kv_attention(x.to(DEV).data_ptr(), {"f16": q.QLIN_F16, "bf16": q.QLIN_BF16}[dtype], rows, hq * d, hq,
                                    c.cache._ref, b._ref, d ** -0.5, cap, one.data_ptr(), hq * d, None, 0,
                                    torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == q.QLIN_OK
    check(one, x, c, table, [0, rows], [kv], hq, d ** -0.5, cap, None, dtype)


@pytest.mark.parametrize("rows,bound,size", [(3, 64, 1e30), (3, KEYS, 1e30), (3, 64, 1e9), (3, KEYS, 1e9), (3, KEYS, 1e6)])
def test_scores_past_the_exponents_range(rows, bound, size):
    """Scores so far apart that a query takes one key's value: that value (one
    rounding to fp16 of a weight of at most 1, one of the output)."""
    c = Cache(4, 16, 1, 128)
    table = np.full((1, bound // 16), -1, dtype=np.int32)
    table[:, :4] = c.table(1, 4)
    x = queries(rows, 128, "bf16", "apart") * size
    b = q.KvBatch(i32(table), i32([0, rows]), i32([60]), max_q=ROWS if bound == KEYS else rows, max_kv=bound)
    out = q.qlin_kv_attention(x.to(DEV), c.cache, b, 1)
    torch.cuda.synchronize()
    with np.errstate(over="ignore"):
        ref = base.oracle.kv_attention(base.f64(x), c.host, table, [0, rows], [60], 1, 128 ** -0.5)
    assert np.all(np.abs(base.f64(out) - ref) <= (2.0 ** -8 + 2.0 ** -10) * np.abs(ref))
