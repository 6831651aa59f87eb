"""Pages of the cache against the plain oracle (GPU only): page numbers, lengths,
reference counts, copies, codes and scales are all equal."""

import numpy as np
import pytest
import torch

import bit_ptq_vla_amd as q
import oracle
from test_gpu_kv_attention import Cache, i32

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Pages:
    """A pool with its table and a stack of caches, on both sides."""

    def __init__(self, pages, rows, cols, page, layers=2, heads=2, d=64):
        self.page = page
        self.ref = oracle.Pool(pages, rows, cols, page)
        self.pool = q.KvPool.empty(pages, DEV)
        self.full = torch.full((rows, cols + 3), 55, dtype=torch.int32, device=DEV)
        self.table = self.full[:, :cols]
        self.table.fill_(-1)
        self.layers = [Cache(pages, page, heads, d, seed=i) for i in range(layers)]
        self.stack = q.KvStack([c.cache for c in self.layers])
        self.len = [0] * rows

    def check(self):
        torch.cuda.synchronize()
        assert np.array_equal(self.table.cpu().numpy(), self.ref.table)
        assert torch.all(self.full[:, self.table.shape[1]:] == 55)
        assert np.array_equal(self.pool.refs.cpu().numpy(), self.ref.refs)
        bits = np.unpackbits(self.pool.free_bits.cpu().numpy().view(np.uint8), bitorder="little")
        assert np.array_equal(bits[:len(self.ref.refs)], self.ref.refs == 0) and not bits[len(self.ref.refs):].any()
        for c in self.layers:
            for name in ("k", "v", "k_scale", "v_scale"):
                assert np.array_equal(getattr(c.cache, name).cpu().numpy(), c.host[name]), name

    def resize(self, new, old=None):
        old = self.len if old is None else old
        lengths, moved = self.ref.resize(old, new)
        got_moved = torch.full((len(new), 2), 9, dtype=torch.int32, device=DEV)
        got = q.qlin_kv_resize(self.pool, self.stack, self.table, i32(old), i32(new), moved=got_moved)
        assert got.tolist() == lengths and got_moved.tolist() == [list(m) for m in moved]
        for a, b in moved:
            if a >= 0:
                for c in self.layers:
                    for x in c.host.values():
                        x[b] = x[a]
        self.len = lengths
        self.check()

    def fork(self, src, dst, length):
        self.ref.fork(src, dst, length)
        q.qlin_kv_fork(self.pool, self.table, i32(src), i32(dst), i32(length), self.page)
        for b, n in zip(dst, length):
            if 0 <= b < len(self.len):
                self.len[b] = n
        self.check()


@pytest.mark.parametrize("page", [16, 32, 64])
def test_growth_sharing_and_return(page):
    p = Pages(23, 6, 5, page)
    p.check()
    p.resize([page, 1, 0, 2 * page + 1, 0, 0])
    p.resize([page + 1, page, 0, 2 * page + 1, 3, 0])
    p.fork([3, 3], [2, 5], [2 * page + 1, page])
    p.resize([n + 1 for n in p.len])                   # two of three holders of the last page copy it
    p.resize([n + page for n in p.len])
    p.resize([0, 5, 0, page, 3, 0])
    p.resize([0] * 6)
    assert len(p.ref.free()) == 23


def test_a_pool_that_runs_out():
    p = Pages(7, 5, 6, 16)
    p.resize([30, 16, 0, 1, 0])                        # 4 of 7 pages
    p.resize([30 + 16, 16, 48, 16, 1])                 # 1 more, then 3: too many; growth inside a page; a later one stays
    assert p.len == [46, 16, 0, 16, 0]
    p.fork([0], [4], [46])
    p.resize([47, 16, 48, 16, 46])                     # row 0 copies its shared page; 3 pages are not there
    assert p.len == [47, 16, 0, 16, 46]
    p.resize([0, 0, 48, 0, 47])                        # what is given back is there for the rows that grow
    assert p.len == [0, 0, 48, 0, 47]


def test_a_holder_that_stays_keeps_its_page_to_itself():
    """The first holder's copy does not fit: the second, which would need none
    after it, stays too."""
    p = Pages(3, 4, 4, 16)
    p.resize([5, 0, 0, 32])
    p.fork([0], [1], [5])
    p.resize([6, 7, 0, 32])
    assert p.len == [5, 5, 0, 32]
    p.resize([6, 7, 0, 16])
    assert p.len == [6, 7, 0, 16]


@pytest.mark.parametrize("rows,pages", [(1024, 5000), (64, 100003), (1, 1)])
def test_many_rows_and_pages(rows, pages):
    g = np.random.default_rng(rows)
    cols = 9
    p = Pages(pages, rows, cols, 16, layers=1, heads=1) if pages < 10000 else None
    if p is None:                                      # bookkeeping alone
        ref = oracle.Pool(pages, rows, cols, 16)
        pool = q.KvPool.empty(pages, DEV)
        taken = g.random(pages) < 0.98                 # few free pages, far apart
        ref.refs[taken] = 1
        pool.refs.copy_(torch.from_numpy(taken.astype(np.int32)))
        bits = np.zeros(-(-pages // 32) * 32, dtype=np.uint8)
        bits[:pages] = ~taken
        pool.free_bits.copy_(torch.from_numpy(np.packbits(bits, bitorder="little").view(np.int32)))
        table = torch.full((rows, cols), -1, dtype=torch.int32, device=DEV)
        old, new = np.zeros(rows, dtype=int), g.integers(0, 140, rows)
        for _ in range(3):
            want, moved = ref.resize(old, new)
            got = q.qlin_kv_resize(pool, None, table, i32(old), i32(new), page_size=16)
            assert got.tolist() == want and np.array_equal(table.cpu().numpy(), ref.table)
            assert np.array_equal(pool.refs.cpu().numpy(), ref.refs)
            old, new = np.array(want), g.integers(0, 140, rows)
        return
    for _ in range(3):
        p.resize(g.integers(0, 100, rows).tolist())
        empty = [r for r in range(rows) if p.len[r] == 0]
        src = [r for r in range(rows) if p.len[r] > 0][:len(empty)]
        if src:
            p.fork(src, empty[:len(src)], [p.len[r] for r in src])
            p.resize([n + int(g.integers(0, 5)) for n in p.len])


def test_damaged_tables_and_lengths():
    p = Pages(9, 3, 4, 16)
    p.resize([20, 40, 0])
    for at, value in (((0, 1), -1), ((1, 0), 1 << 20), ((1, 2), -77)):
        p.ref.table[at] = value
        p.table[at] = value
    p.resize([0, 0, -5])                               # those pages stay lost, nothing else changes
    assert p.len == [0, 0, 0]
    p.resize([0, 10 ** 9, 3])                          # cut to the table's columns
    assert p.len[1] == 64
    p.ref.table[2, 0] = p.ref.table[1, 0]              # the same page twice: given back twice, free once
    p.table[2, 0] = p.table[1, 0]
    p.ref.refs[p.ref.table[1, 0]] = 1
    p.resize([0, 0, 0])
    p.fork([0, -1, 7, 1], [1, 2, 2, 9], [16, 16, 16, 16])


def test_copy_pages():
    p = Pages(40, 1, 1, 32, layers=35, heads=3, d=128)   # more layers than a launch takes
    g = np.random.default_rng(5)
    order = g.permutation(40)
    pairs = np.array(list(zip(order[:15], order[15:30])) + [(-1, 33), (3, 40), (1 << 30, 2), (5, -9)])
    q.qlin_kv_copy_pages(p.stack, i32(pairs))
    for a, b in pairs[:15]:
        for c in p.layers:
            for x in c.host.values():
                x[b] = x[a]
    p.check()
    q.qlin_kv_copy_pages(p.stack, torch.zeros((0, 2), dtype=torch.int32, device=DEV))
    many = np.full((3000, 2), -1)                        # most pairs copy nothing, over several gathers
    many[[0, 1023, 1024, 2999]] = [(1, 2), (3, 4), (5, 6), (7, 8)]
    q.qlin_kv_copy_pages(p.stack, i32(many))
    for a, b in ((1, 2), (3, 4), (5, 6), (7, 8)):
        for c in p.layers:
            for x in c.host.values():
                x[b] = x[a]
    p.check()


# ---- compaction

CASES = [
    # heads, d, page, layers, (nodes, cached, path) of each sequence
    (2, 64, 16, 1, [(1, 0, [0])]),
    (2, 128, 16, 2, [(16, 100, [0, 3, 4, 9, 15]), (16, 3, [0, 1, 2]), (16, 13, [0, 5]), (0, 7, []), (5, 0, [])]),
    (1, 256, 64, 2, [(64, 50, [0, 1, 2, 30, 31, 40, 41, 42, 43, 44, 45, 60, 61, 62, 63]), (33, 64, [32]), (7, 10, [0, 6])]),
    (3, 64, 32, 3, [(100, 20, list(range(0, 100, 2))), (90, 0, list(range(1, 90))), (40, 31, list(range(40)))]),
    (2, 128, 64, 34, [(20, 60, [0, 2, 8, 9])]),
    (1, 64, 16, 1, [(200, 9, list(range(0, 20)) + list(range(50, 180, 3)))]),
]


def compact(c, heads, d, page, layers, seqs, paths=None, counts=None, damage=None):
    new = [s[0] for s in seqs]
    kv = np.array([s[0] + s[1] for s in seqs])
    start = np.concatenate([[0], np.cumsum(new)])
    cols = max(1, -(-int(kv.max()) // page))
    caches = [Cache(len(seqs) * cols + 2, page, heads, d, seed=i, spread=3.0) for i in range(layers)]
    table = caches[0].table(len(seqs), cols).copy()
    if damage:
        damage(table, kv)
    mq = max(1, max(new))
    path = np.full((len(seqs), mq + 1), 7)
    for b, s in enumerate(seqs):
        path[b, :len(s[2])] = s[2]
    count = np.array([len(s[2]) for s in seqs]) if counts is None else np.array(counts)
    batch = q.KvBatch(i32(table), i32(start), i32(kv), max_q=mq, max_kv=cols * page)
    got = q.qlin_kv_compact(q.KvStack([x.cache for x in caches]), batch, i32(path), i32(count))
    torch.cuda.synchronize()
    want = oracle.kv_compact([x.host for x in caches], table, start, kv, path, count)
    assert got.tolist() == want
    for x in caches:
        for name in ("k_scale", "v_scale", "k", "v"):
            assert np.array_equal(getattr(x.cache, name).cpu().numpy(), x.host[name]), name


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}x{c[1]}-p{c[2]}-l{c[3]}")
def test_compact(case):
    compact(None, *case)


def test_compact_over_damaged_paths_counts_and_pages():
    seqs = [(16, 20, [0, 3, 3, 5]), (16, 5, [0, 4, 2]), (8, 40, [1, 7, 8]), (6, 30, [0, -2, 4]), (9, 17, [2, 4, 6, 8]), (5, 9, [4])]
    compact(None, 2, 64, 16, 2, seqs)
    compact(None, 2, 64, 16, 1, seqs, counts=[100, -3, 2, 1 << 30, 3, 1])

    def damage(table, kv):
        table[0, 1], table[2, 2], table[4, 1] = -1, 10 ** 7, -5
        kv[5] = 3                                        # more new tokens than its length

    compact(None, 2, 64, 16, 1, seqs, damage=damage)


def test_compact_with_zero_scales_and_captured():
    c = Cache(6, 16, 1, 64)
    c.host["k_scale"][:] = 0
    c.host["v_scale"][2:4] = 0
    c.upload()
    table, start, kv = np.array([[1, 2, 3]]), [0, 20], [45]
    path, count = i32([[0, 2, 9, 12, 13, 14, 19] + [-1] * 13]), i32([7])
    batch = q.KvBatch(i32(table), i32(start), i32(kv), max_q=20, max_kv=48)
    stack = q.KvStack([c.cache])
    out = torch.empty(1, dtype=torch.int32, device=DEV)
    first = [t.clone() for t in (c.cache.k, c.cache.v, c.cache.k_scale, c.cache.v_scale)]
    oracle.kv_compact([c.host], table, start, kv, path.tolist(), [7])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.qlin_kv_compact(stack, batch, path, count, kv_len_out=out)
    for _ in range(3):
        for t, x in zip((c.cache.k, c.cache.v, c.cache.k_scale, c.cache.v_scale), first):
            t.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert out.tolist() == [32]
        for name in ("k_scale", "v_scale", "k", "v"):
            assert np.array_equal(getattr(c.cache, name).cpu().numpy(), c.host[name]), name


@pytest.mark.parametrize("page,cached,nodes,path", [
    (64, 48, 16, [0, 3, 9, 15]), (64, 47, 40, [0, 1, 2, 16, 17, 30, 39]), (32, 16, 8, [3, 7]), (64, 1, 63, [0, 62]),
    (32, 31, 70, list(range(0, 70, 3))), (16, 15, 33, [0, 32])])
@pytest.mark.parametrize("equal", [True, False])
def test_granules_of_kept_tokens(page, cached, nodes, path, equal):
    """Granules of a page whose tokens are all kept: under one scale for all pages, where
    nothing of them changes, and under scales of their own."""
    cols = -(-(cached + nodes) // page)
    c = Cache(cols + 1, page, 2, 64, seed=cached + page, spread=3.0)
    if equal:
        c.host["k_scale"][:] = 0.03
        c.host["v_scale"][:] = 0.02
        c.upload()
    table = c.table(1, cols)
    batch = q.KvBatch(i32(table), i32([0, nodes]), i32([cached + nodes]), max_q=nodes, max_kv=cols * page)
    wide = np.full((1, nodes), -1)
    wide[0, :len(path)] = path
    before = {n: x.copy() for n, x in c.host.items()}
    got = q.qlin_kv_compact(q.KvStack([c.cache]), batch, i32(wide), i32([len(path)]))
    torch.cuda.synchronize()
    assert got.tolist() == oracle.kv_compact([c.host], table, [0, nodes], [cached + nodes], wide, [len(path)])
    for name in ("k_scale", "v_scale", "k", "v"):
        assert np.array_equal(getattr(c.cache, name).cpu().numpy(), c.host[name]), name
    if equal:
        first = table[0, 0]
        kept = min(cached, page)
        assert np.array_equal(c.host["k"][first][:, :kept], before["k"][first][:, :kept])
        assert np.array_equal(c.host["v"][first][:, :, :kept], before["v"][first][:, :, :kept])
