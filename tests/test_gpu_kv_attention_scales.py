"""Attention over pages whose scales lie far apart, through both kernels (GPU
only).  The bounds a call states choose the kernel: those of the lengths give
blocks of 16 query rows, far larger ones the kernel for prompts.
"""

import numpy as np
import pytest
import torch

import bit_ptq_vla_amd as q
from test_gpu_kv_attention import DEV, Cache, check, i32, queries

pytestmark = pytest.mark.gpu
ROWS, KEYS = 200, 1 << 18


def batch_of(table, q_start, kv_len, page, wide):
    n = int(np.diff(q_start).max())
    if not wide:
        return q.KvBatch(i32(table), i32(q_start), i32(kv_len), max_q=n, max_kv=table.shape[1] * page)
    bounds = np.full((len(table), KEYS // page), -7, dtype=np.int32)       # no page: never to be read
    bounds[:, :table.shape[1]] = table
    return q.KvBatch(i32(bounds), i32(q_start), i32(kv_len), max_q=max(ROWS, n), max_kv=KEYS)


@pytest.mark.parametrize("wide", [False, True], ids=["rows16", "prompts"])
@pytest.mark.parametrize("dtype,d,page", [("bf16", 128, 16), ("f16", 128, 32), ("f16", 64, 16), ("bf16", 256, 64)])
def test_zero_key_scales_under_a_negative_scale(dtype, d, page, wide):
    """Keys of a zero scale have score 0, every other key a score near -60: a row
    that sees any of the former averages their values.  A prompt, so that the
    causal limit cuts such a page at every place."""
    cols = 4
    c = Cache(cols + 1, page, 1, d)
    g = np.random.default_rng(17)
    c.host["k"][:] = g.integers(30, 51, c.host["k"].shape)                 # every product with a query positive
    c.host["k_scale"][:] = 0.025
    table = c.table(1, cols)
    c.host["k_scale"][table[0, [1, 3]]] = 0.0
    c.upload()
    kv = cols * page - 3
    x = queries(kv, d, dtype, f"negative{d}").abs() * 0.25 + 1.0
    out = q.qlin_kv_attention(x.to(DEV), c.cache, batch_of(table, [0, kv], [kv], page, wide), 1, sm_scale=-64.0 / d)
    torch.cuda.synchronize()
    check(out, x, c, table, [0, kv], [kv], 1, -64.0 / d, 0.0, None, dtype)
