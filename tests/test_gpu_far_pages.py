"""The same pages at the front of a small cache and behind 2^32 bytes of codes of a
large one give the same bits (GPU only)."""

import numpy as np
import pytest
import torch

import bit_ptq_vla_amd as q
from test_gpu_kv_attention import Cache, i32, queries
from test_gpu_tree import random_parents, starts

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def caches():
    """A cache of 40 pages of 64 KB, and one of 2^16 + 60 whose last 40 hold the same."""
    small = Cache(40, 64, 8, 128).cache
    far = 2 ** 16 + 20
    shapes = [(far + 40, 8, 64, 128), (far + 40, 8, 128, 64)]
    k, v = (torch.empty(s, dtype=torch.int8, device=DEV) for s in shapes)
    ks, vs = (torch.empty(far + 40, 8, device=DEV) for _ in range(2))
    for whole, part in ((k, small.k), (v, small.v), (ks, small.k_scale), (vs, small.v_scale)):
        whole[far:] = part
    return small, q.KvCache(k, ks, v, vs), far


def same(small, large, far):
    torch.cuda.synchronize()
    for name in ("k", "v", "k_scale", "v_scale"):
        assert torch.equal(getattr(small, name), getattr(large, name)[far:]), name


# a wave's blocks, and those for many rows (the bound is long)
@pytest.mark.parametrize("nodes,max_kv", [(9, 768), (100, 1 << 16)])
def test_tree_attention(caches, nodes, max_kv):
    small, large, far = caches
    g = np.random.default_rng(4)
    start, kv = starts([nodes, nodes - 3]), [nodes + 500, nodes + 130]
    table = np.zeros((2, max_kv // 64), dtype=np.int32)
    table[:, :12] = g.permutation(40)[:24].reshape(2, 12)
    x = queries(int(start[-1]), 16 * 128, "bf16", "far").to(DEV)
    out = []
    for cache, base in ((small, 0), (large, far)):
        batch = q.KvBatch(i32(table + base), i32(start), i32(kv), max_q=nodes, max_kv=max_kv)
        parents = np.concatenate([random_parents(n, np.random.default_rng(n)) for n in (nodes, nodes - 3)])
        mask, _ = q.qlin_tree_plan(i32(parents), batch)
        out.append(q.qlin_kv_attention_tree(x, cache, batch, 16, mask))
    torch.cuda.synchronize()
    assert torch.equal(*out)


def test_copies_and_compaction(caches):
    small, large, far = caches
    pairs = np.array([[3, 38], [39, 2], [5, 6]])
    path, count = i32([[0, 3, 4, 9, 20, 41]]), i32([6])
    table = np.array([[7, 30, 1, 12]])
    for cache, base in ((small, 0), (large, far)):
        stack = q.KvStack([cache])
        q.qlin_kv_copy_pages(stack, i32(pairs + base))
        batch = q.KvBatch(i32(table + base), i32([0, 60]), i32([180]), max_q=60, max_kv=256)
        wide = torch.full((1, 60), -1, dtype=torch.int32, device=DEV)
        wide[:, :6] = path
        assert q.qlin_kv_compact(stack, batch, wide, count).tolist() == [126]
    same(small, large, far)


def test_a_shared_page_is_copied_behind_a_large_pool(caches):
    small, large, far = caches
    for cache, base in ((small, 0), (large, far)):
        pool = q.KvPool.empty(cache.pages, DEV)
        taken = torch.arange(cache.pages, device=DEV) < base + 10          # ten pages and what lies before
        pool.refs.copy_(taken.int())
        words = np.packbits((~taken).cpu().numpy(), bitorder="little")
        words = np.concatenate([words, np.zeros(-len(words) % 4, dtype=np.uint8)]).view(np.int32)
        pool.free_bits.copy_(torch.from_numpy(words.copy()).to(DEV))
        table = torch.full((2, 4), -1, dtype=torch.int32, device=DEV)
        stack = q.KvStack([cache])
        lengths = q.qlin_kv_resize(pool, stack, table, i32([0, 0]), i32([100, 0]))
        q.qlin_kv_fork(pool, table, i32([0]), i32([1]), i32([100]), 64)
        moved = torch.empty((2, 2), dtype=torch.int32, device=DEV)
        lengths = q.qlin_kv_resize(pool, stack, table, i32([100, 100]), i32([130, 101]), moved=moved)
        assert lengths.tolist() == [130, 101]
        assert moved.tolist() == [[base + 11, base + 12], [-1, -1]]
        assert table.tolist() == [[base + 10, base + 12, base + 13, -1], [base + 10, base + 11, -1, -1]]
    same(small, large, far)
