"""Forms of the attention call beside those of the general tests, through both
kernels (GPU only): capped scores in fp16 and at 64-wide heads, capped split
keys, and captured calls of the kernel for prompts.  Tolerances as there.
"""

import numpy as np
import pytest
import torch

import bit_ptq_vla_amd as q
import test_gpu_kv_attention as base
from test_gpu_kv_attention import DEV, Cache, check, i32, queries
from test_gpu_kv_attention_prompts import KEYS, ROWS, wide  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu

CAPPED = [
    # dtype, hq, hkv, d, page, cap, (new, cached, prefix or None) of each sequence
    ("f16", 4, 2, 64, 16, 30.0, [(1, 200, None), (1, 15, None), (0, 4, None)]),
    ("f16", 2, 2, 64, 64, 2.0, [(70, 3, 20), (33, 64, 0)]),
    ("bf16", 4, 1, 64, 32, 50.0, [(1, 333, None), (5, 0, None)]),
    ("bf16", 2, 1, 64, 16, 8.0, [(129, 17, 1000), (64, 0, 5)]),
    ("f16", 4, 4, 128, 16, 30.0, [(1, 500, None)]),
    ("f16", 6, 2, 128, 64, 5.0, [(50, 30, 7), (65, 0, 0)]),
    ("f16", 2, 1, 256, 32, 50.0, [(1, 129, None), (1, 0, None)]),
    ("f16", 1, 1, 256, 16, 20.0, [(140, 9, 11)]),
]


def names(c):
    return f"{c[0]}-{c[1]}-{c[2]}-{c[3]}-p{c[4]}-cap{c[5]}-{len(c[6])}"


@pytest.mark.parametrize("case", CAPPED, ids=names)
def test_capped(case):
    base.test_attention(case)


@pytest.mark.parametrize("case", CAPPED, ids=names)
def test_capped_prompts(case, wide):  # noqa: F811
    base.test_attention(case)


@pytest.mark.parametrize("dtype,hq,hkv,d,page,rows,kv,bound,cap", [
    ("f16", 8, 1, 64, 16, 2, 4097, 4112, 20.0), ("f16", 2, 1, 128, 64, 2, 3000, 3008, 30.0),
    ("f16", 1, 1, 256, 32, 1, 2900, 2912, 4.0), ("bf16", 4, 1, 64, 16, 1, 2000, 2000, 50.0),
    ("f16", 4, 4, 64, 16, 260, 4500, 65536, 10.0), ("f16", 4, 4, 256, 64, 150, 2600, 16384, 30.0),
])
def test_capped_split_keys(dtype, hq, hkv, d, page, rows, kv, bound, cap):
    cols = -(-kv // page)
    c = Cache(cols + 1, page, hkv, d, seed=27)
    table = np.full((1, bound // page), -1, dtype=np.int32)
    table[:, :cols] = c.table(1, cols)
    x = queries(rows, hq * d, dtype, f"capsplit{kv}") * 3.0
    b = q.KvBatch(i32(table), i32([0, rows]), i32([kv]), max_q=rows, max_kv=bound)
    assert q.kv_attention_workspace_bytes(c.cache, b, hq) > 0
    out = q.qlin_kv_attention(x.to(DEV), c.cache, b, hq, softcap=cap)
    torch.cuda.synchronize()
    check(out, x, c, table, [0, rows], [kv], hq, d ** -0.5, cap, None, dtype)


@pytest.mark.parametrize("dtype,hq,hkv,d,page,cap", [("bf16", 2, 1, 256, 64, 30.0), ("f16", 4, 2, 128, 32, 0.0),
                                                     ("f16", 2, 2, 64, 16, 0.0)])
def test_captured_prompts(dtype, hq, hkv, d, page, cap):
    """One captured call of the kernel for prompts (its keys split: two launches),
    replayed over other lengths, with eager calls and other work between."""
    cols = 20
    c = Cache(2 * cols + 1, page, hkv, d)
    table = np.full((2, KEYS // page), -1, dtype=np.int32)
    table[:, :cols] = c.table(2, cols)
    rows = 180
    q_start, kv = i32([0, 100, 180]), i32([100, 200])
    b = q.KvBatch(i32(table), q_start, kv, max_q=ROWS, max_kv=KEYS)
    work = q.kv_attention_workspace(c.cache, b, hq)
    assert work is not None
    x = queries(rows, hq * d, dtype, "capture").to(DEV)
    out = torch.empty_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q.qlin_kv_attention(x, c.cache, b, hq, softcap=cap, out=out, workspace=work)
    for t, (starts, lens) in enumerate([([0, 100, 180], [100, 200]), ([0, 1, 180], [317, 179]), ([0, 180, 180], [200, 9]),
                                        ([0, 60, 180], [60, 120])]):
        h = queries(rows, hq * d, dtype, f"capture{t}")
        x.copy_(h)
        q_start.copy_(torch.tensor(starts))
        kv.copy_(torch.tensor(lens))
        g.replay()
        torch.cuda.synchronize()
        check(out, h, c, table, starts, lens, hq, d ** -0.5, cap, None, dtype)
        eager = q.qlin_kv_attention(x, c.cache, b, hq, softcap=cap)
        (eager.float() @ torch.ones((hq * d, 64), device=DEV)).sum()
        torch.cuda.synchronize()
        assert torch.equal(eager.view(torch.int16), out.view(torch.int16))
