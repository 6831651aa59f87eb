"""Tree attention for many rows, whose work is dealt to the CUs in even shares
(GPU only): shares of a step or less, of several whole blocks of rows, of ends
and beginnings; sequences without tokens, without keys, of one token."""

import numpy as np
import pytest
import torch

import bit_ptq_vla_amd as q
from test_gpu_kv_attention import Cache, i32, queries
from test_gpu_tree import check, make_sees, random_parents, starts

pytestmark = pytest.mark.gpu
DEV = "cuda"

CASES = [
    # dtype, hq, hkv, d, page, cap, max_kv, (nodes, cached) of each sequence
    ("bf16", 4, 2, 128, 64, 0.0, 1 << 16, [(200, 37), (0, 5), (129, 3000), (1, 0), (64, 6000), (17, 0)]),
    ("f16", 4, 2, 128, 16, 30.0, 1 << 16, [(130, 7), (256, 900), (5, 2000)]),
    ("bf16", 8, 8, 64, 32, 0.0, 2048, [(140 - b % 3, 40 + 5 * b) for b in range(40)]),
    ("f16", 4, 1, 256, 32, 0.0, 1 << 16, [(70, 1500), (40, 20), (33, 700)]),
    ("bf16", 6, 2, 256, 64, 50.0, 1 << 16, [(0, 0), (50, 0), (64, 129), (0, 77)]),
]


def build(case):
    dtype, hq, hkv, d, page, cap, max_kv, seqs = case
    g = np.random.default_rng(11)
    start, kv = starts([n for n, _ in seqs]), np.array([n + c for n, c in seqs])
    cols = max(1, -(-int(kv.max()) // page))
    c = Cache(len(seqs) * cols + 2, page, hkv, d)
    table = c.table(len(seqs), cols)
    wide = np.zeros((len(seqs), max_kv // page), dtype=np.int32)
    wide[:, :cols] = table
    parents = np.concatenate([random_parents(n, g) for n, _ in seqs])
    x = queries(int(start[-1]), hq * d, dtype, "shares").to(DEV)
    lengths = i32(kv)
    batch = q.KvBatch(i32(wide), i32(start), lengths, max_q=max(n for n, _ in seqs), max_kv=max_kv)
    return c, table, start, kv, parents, x, batch, lengths


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}-{c[1]}-{c[2]}-{c[3]}-p{c[4]}-cap{c[5]}-{len(c[7])}")
def test_shares(case):
    dtype, hq, hkv, d, page, cap, max_kv, seqs = case
    c, table, start, kv, parents, x, batch, _ = build(case)
    sees = make_sees(parents, start, batch.max_q)
    mask, _ = q.qlin_tree_plan(i32(parents), batch)
    work = q.kv_attention_tree_workspace(c.cache, batch, hq)
    assert work is not None and work.numel() > 256
    for fill in (255, 127):                     # (what the workspace holds does not matter)
        work.fill_(fill)
        out = torch.full_like(x, 5.0)
        q.qlin_kv_attention_tree(x, c.cache, batch, hq, mask, softcap=cap, out=out, workspace=work)
        torch.cuda.synchronize()
        check(out, x, c, table, start, kv, hq, sees, d ** -0.5, cap, dtype)


def test_replays_follow_the_lengths():
    """A captured call reads the lengths anew; a sequence without any gives zeros."""
    case = CASES[0]
    c, table, start, kv, parents, x, batch, lengths = build(case)
    mask, _ = q.qlin_tree_plan(i32(parents), batch)
    work = q.kv_attention_tree_workspace(c.cache, batch, 4)
    out = torch.empty_like(x)
    q.qlin_kv_attention_tree(x, c.cache, batch, 4, mask, out=out, workspace=work)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q.qlin_kv_attention_tree(x, c.cache, batch, 4, mask, out=out, workspace=work)
    for change in ([0] * 6, [0, 0, -2990, 0, -5000, 0], [10 ** 6] * 6, [-10 ** 6] * 6, [-200, 0, 0, 0, -64, 0], [0] * 6):
        lengths.copy_(i32(kv + np.array(change)))
        want = q.qlin_kv_attention_tree(x, c.cache, batch, 4, mask)
        out.fill_(3.0)
        work.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        if change[0] == -10 ** 6:
            assert torch.all(out == 0)
