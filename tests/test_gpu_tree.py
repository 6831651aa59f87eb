"""Trees of drafted tokens against the float64 oracle (GPU only): masks, positions
and accepted paths are whole numbers and equal; attention within the tolerance
derived in test_gpu_kv_attention.py (the same kernels' roundings)."""

import numpy as np
import pytest
import torch

import bit_ptq_vla_amd as q
import oracle
from test_gpu_kv_attention import DT, HALF_STEP, Cache, batch_of, f64, i32, queries

pytestmark = pytest.mark.gpu
DEV = "cuda"


def random_parents(n, g, wide=8):
    return np.array([-1 if i == 0 or g.random() < 0.05 else i - 1 - int(g.random() ** 2 * min(i, wide)) for i in range(n)], dtype=np.int64)


def mask_words(sees, words):
    """bool [tokens][n] to int32 [tokens][words]."""
    bits = np.zeros((len(sees), 32 * words), dtype=np.uint8)
    bits[:, :sees.shape[1]] = sees
    return np.packbits(bits, axis=1, bitorder="little").view(np.int32)


def starts(new):
    return np.concatenate([[0], np.cumsum(new)]).astype(np.int64)


def make_sees(parents, q_start, max_q):
    sees = np.zeros((len(parents), max_q), dtype=bool)
    for a, b in zip(q_start[:-1], q_start[1:]):
        sees[a:b, :b - a] = oracle.tree_sees(parents[a:b])
    return sees


@pytest.mark.parametrize("new", [[1], [16], [33, 0, 1, 32, 64, 65, 31], [1024, 5], [0, 0]])
@pytest.mark.parametrize("shape", ["random", "chain", "star", "roots"])
def test_plan_and_accept(new, shape):
    g = np.random.default_rng(len(new) + 7)
    start = starts(new)
    tokens, mq = int(start[-1]), max(max(new), 1)
    local = np.concatenate([np.arange(n) for n in new]).astype(np.int64) if tokens else np.zeros(0, dtype=np.int64)
    parents = {"random": np.concatenate([random_parents(n, g) for n in new] + [np.zeros(0, dtype=np.int64)]),
               "chain": local - 1, "star": np.where(local > 0, 0, -1),
               "roots": local + g.integers(0, 3, tokens)}[shape]      # (no earlier node: itself or a later one)
    kv = np.array(new) + g.integers(0, 50, len(new))
    batch = q.KvBatch(i32(np.zeros((len(new), 80))), i32(start), i32(kv), max_q=mq, max_kv=80 * 16)
    sees = make_sees(parents, start, mq)
    words = -(-mq // 32)
    mask = torch.full((tokens, words + 2), 77, dtype=torch.int32, device=DEV)
    got_mask, got_pos = q.qlin_tree_plan(i32(parents), batch, mask=mask)
    draft = g.integers(0, 3, tokens)
    sampled = g.integers(0, 3, tokens)
    path, count, token = q.qlin_tree_accept(i32(parents), i32(draft), i32(sampled), batch)
    torch.cuda.synchronize()
    assert np.array_equal(got_mask.cpu().numpy()[:, :words], mask_words(sees, words))
    assert np.all(got_mask.cpu().numpy()[:, words:] == 77)
    seq = np.repeat(np.arange(len(new)), new)
    assert np.array_equal(got_pos.cpu().numpy(), (kv - np.array(new))[seq] + sees.sum(1) - 1)
    for b in range(len(new)):
        s = slice(start[b], start[b + 1])
        want, last = oracle.tree_accept(parents[s], draft[s], sampled[s])
        assert path[b].tolist() == want + [-1] * (mq - len(want))
        assert (int(count[b]), int(token[b])) == (len(want), last)


def check(out, x, c, table, q_start, kv_len, hq, sees, scale, cap, dtype):
    d = c.cache.head_dim
    ref = oracle.kv_attention_tree(f64(x), c.host, table, q_start, kv_len, hq, sees, scale, cap)
    a = oracle.kv_attention_tree(f64(x), dict(c.host, v=np.abs(c.host["v"].astype(np.int16))), table, q_start, kv_len, hq,
                                 sees, scale, cap)
    rows = np.arange(q_start[0], q_start[-1])
    n = max(1, int(np.max(kv_len)))
    kmax = 127.0 * float(np.max(c.host["k_scale"]))
    vmax = 127.0 * float(np.max(c.host["v_scale"]))
    b = abs(scale) * kmax * np.abs(f64(x)[rows]).reshape(-1, hq, d).sum(2)
    if cap:
        b = np.minimum(b, cap)
    delta = (d + 8) * 2.0 ** -24 * b + (2.0 ** -21 * cap if cap else 0.0)
    rel = np.repeat(2 * delta + 2.0 ** -11 + (n + 8) * 2.0 ** -24, d, axis=1)
    tiny = 2.0 ** -25 if dtype == "f16" else 0.0
    tol = rel * a[rows] * (1 + 2.0 ** -6) + n * 2.0 ** -25 * vmax + HALF_STEP[dtype] * np.abs(ref[rows]) * (1 + 2.0 ** -6) + tiny
    err = np.abs(f64(out)[rows] - ref[rows])
    assert np.all(err <= tol), f"worst {np.max(err / tol):.3g} of the tolerance, error {np.max(err):.3g}"


CASES = [
    # dtype, hq, hkv, d, page, cap, (nodes, cached) of each sequence
    ("f16", 2, 2, 128, 16, 0.0, [(1, 0)]),
    ("f16", 4, 4, 128, 16, 0.0, [(16, 816)]),
    ("bf16", 8, 2, 128, 32, 0.0, [(16, 100), (1, 31), (9, 64), (0, 9), (0, 0), (16, 0), (7, 33)]),
    ("bf16", 4, 1, 256, 64, 50.0, [(5, 300), (8, 62)]),
    ("f16", 6, 2, 64, 16, 0.0, [(5, 40), (1, 3), (17, 0), (33, 31)]),
    ("bf16", 20, 1, 64, 32, 0.0, [(7, 77), (2, 0)]),
    ("f16", 2, 2, 128, 32, 0.0, [(50, 81), (50, 16)]),
    ("bf16", 2, 2, 256, 64, 30.0, [(70, 0), (33, 5), (64, 64)]),
    ("f16", 8, 1, 64, 64, 0.0, [(40, 0), (64, 129)]),
    ("bf16", 3, 1, 128, 16, 5.0, [(130, 3), (97, 0), (128, 64)]),
    ("f16", 2, 1, 128, 64, 0.0, [(200, 37), (129, 0), (1, 500)]),
    ("f16", 8, 2, 128, 16, 0.0, [(64, 700), (63, 1000)]),
    ("f16", 1, 1, 256, 16, 0.0, [(150, 20)]),
]


def setup(case, seed=3):
    dtype, hq, hkv, d, page, cap, seqs = case
    g = np.random.default_rng(seed)
    new = [n for n, _ in seqs]
    start = starts(new)
    kv = np.array([n + c for n, c in seqs])
    cols = max(1, -(-int(kv.max()) // page))
    c = Cache(len(seqs) * cols + 2, page, hkv, d)
    table = c.table(len(seqs), cols)
    parents = np.concatenate([random_parents(n, g) for n in new])
    x = queries(int(start[-1]), hq * d, dtype, f"tree{seed}").to(DEV)
    return c, table, start, kv, parents, x, batch_of(table, start, kv, page)


@pytest.mark.parametrize("bound", ["exact", "wide"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}-{c[1]}-{c[2]}-{c[3]}-p{c[4]}-cap{c[5]}-{len(c[6])}")
def test_attention(case, bound):
    dtype, hq, hkv, d, page, cap, seqs = case
    c, table, start, kv, parents, x, batch = setup(case)
    if bound == "wide":                               # (the kernel for many rows, and the splits of a long bound)
        wide = np.zeros((len(seqs), 2048 // page + table.shape[1]), dtype=np.int32)
        wide[:, :table.shape[1]] = table
        batch = q.KvBatch(i32(wide), i32(start), i32(kv), max_q=min(1024, batch.max_q * 4), max_kv=wide.shape[1] * page)
    sees = make_sees(parents, start, max(1, batch.max_q))
    mask, _ = q.qlin_tree_plan(i32(parents), batch)
    out = q.qlin_kv_attention_tree(x, c.cache, batch, hq, mask, softcap=cap)
    torch.cuda.synchronize()
    check(out, x, c, table, start, kv, hq, sees, d ** -0.5, cap, dtype)
    one = torch.empty_like(out)
    q._check(q.load().qlin_kv_attention_tree(x.data_ptr(), q._TORCH_TO_QLIN[x.dtype], len(x), x.stride(0), hq,
                                             c.cache._ref, batch._ref, mask.data_ptr(), mask.shape[1], d ** -0.5, cap,
                                             one.data_ptr(), one.stride(0), None, 0, q._stream(x.device)), "unsplit")
    torch.cuda.synchronize()
    check(one, x, c, table, start, kv, hq, sees, d ** -0.5, cap, dtype)


@pytest.mark.parametrize("max_kv", [1 << 16, 1 << 19, 1 << 22])
@pytest.mark.parametrize("case", [CASES[i] for i in (2, 4, 5, 6, 7, 9, 10, 11, 12)],
                         ids=lambda c: f"{c[0]}-{c[1]}-{c[2]}-{c[3]}-p{c[4]}-cap{c[5]}-{len(c[6])}")
def test_attention_under_far_bounds(case, max_kv):
    """The kernels for more rows are chosen by the bound: blocks of 32 and of 256 rows
    on short sequences, with and without split keys."""
    dtype, hq, hkv, d, page, cap, seqs = case
    c, table, start, kv, parents, x, batch = setup(case)
    wide = np.zeros((len(seqs), max_kv // page), dtype=np.int32)
    wide[:, :table.shape[1]] = table
    batch = q.KvBatch(i32(wide), i32(start), i32(kv), max_q=batch.max_q, max_kv=max_kv)
    sees = make_sees(parents, start, max(1, batch.max_q))
    mask, _ = q.qlin_tree_plan(i32(parents), batch)
    for split in (True, False):
        out = torch.full_like(x, 5.0)
        work = q.kv_attention_tree_workspace(c.cache, batch, hq) if split else None
        q._check(q.load().qlin_kv_attention_tree(x.data_ptr(), q._TORCH_TO_QLIN[x.dtype], len(x), x.stride(0), hq,
                                                 c.cache._ref, batch._ref, mask.data_ptr(), mask.shape[1], d ** -0.5, cap,
                                                 out.data_ptr(), out.stride(0), q._ptr(work),
                                                 0 if work is None else work.numel(), q._stream(x.device)), "tree")
        torch.cuda.synchronize()
        check(out, x, c, table, start, kv, hq, sees, d ** -0.5, cap, dtype)


@pytest.mark.parametrize("case", [CASES[2], CASES[6], CASES[9]], ids=["16", "50", "130"])
def test_chain_gives_the_bits_of_causal_attention(case):
    """Where every key behind a query is masked either way, the products are the same."""
    dtype, hq, hkv, d, page, cap, seqs = case
    c, table, start, kv, _, x, batch = setup(case)
    chain = np.concatenate([np.arange(n) - 1 for n, _ in seqs])
    mask, positions = q.qlin_tree_plan(i32(chain), batch)
    tree = q.qlin_kv_attention_tree(x, c.cache, batch, hq, mask, softcap=cap)
    causal = q.qlin_kv_attention(x, c.cache, batch, hq, softcap=cap)
    torch.cuda.synchronize()
    sees = make_sees(chain, start, max(1, batch.max_q))
    check(tree, x, c, table, start, kv, hq, sees, d ** -0.5, cap, dtype)
    assert torch.allclose(tree.float(), causal.float(), rtol=2 * HALF_STEP[dtype], atol=1e-3)
    want = np.concatenate([np.arange(k - n, k) for (n, _), k in zip(seqs, kv)])
    assert np.array_equal(positions.cpu().numpy(), want)


def test_any_mask_empty_rows_and_bits_behind_the_nodes():
    """Masks that no tree has: rows of zeros (with and without cached keys), without
    the own bit, and with bits set behind the sequence's nodes."""
    g = np.random.default_rng(8)
    case = ("f16", 4, 2, 64, 16, 0.0, [(40, 0), (33, 21), (3, 7)])
    c, table, start, kv, _, x, batch = setup(case)
    sees = g.random((int(start[-1]), 64)) < 0.2
    sees[[0, 5, 39, 50]] = False
    mask = mask_words(sees, 2)
    for b, (n, _) in enumerate(case[6]):
        sees[start[b]:start[b + 1], n:] = False
    out = q.qlin_kv_attention_tree(x, c.cache, batch, 4, torch.from_numpy(mask.copy()).to(DEV))
    torch.cuda.synchronize()
    check(out, x, c, table, start, kv, 4, sees, 0.125, 0.0, "f16")
    assert torch.all(out[5] == 0)


def test_strides_rows_behind_and_pages_outside_the_pool():
    case = ("bf16", 4, 2, 128, 16, 0.0, [(5, 40), (12, 100)])
    c, table, start, kv, parents, x, batch = setup(case)
    table = table.copy()
    table[1, 2], table[0, 0] = -1, 10 ** 6
    batch = batch_of(table, start, kv, 16)
    tokens = int(start[-1])
    wide_q = torch.zeros((tokens + 3, 4 * 128 + 64), dtype=x.dtype, device=DEV)
    wide_q[:tokens, :512] = x
    out = torch.full((tokens + 3, 4 * 128 + 8), 9.0, dtype=x.dtype, device=DEV)
    mask = torch.zeros((tokens + 3, 5), dtype=torch.int32, device=DEV)
    sees = make_sees(parents, start, 12)
    mask[:tokens, :1] = torch.from_numpy(mask_words(sees, 1).copy()).to(DEV)
    q.qlin_kv_attention_tree(wide_q[:, :512], c.cache, batch, 4, mask, out=out[:, :512])
    torch.cuda.synchronize()
    check(out[:tokens, :512], x, c, table, start, kv, 4, sees, 128 ** -0.5, 0.0, "bf16")
    assert torch.all(out[tokens:] == 9.0) and torch.all(out[:, 512:] == 9.0)


def test_captured_and_on_another_stream():
    case = ("f16", 8, 2, 128, 16, 0.0, [(16, 500), (9, 1000)])
    c, table, start, kv, parents, x, batch = setup(case)
    p = i32(parents)
    mask, positions = q.qlin_tree_plan(p, batch)
    work = q.kv_attention_tree_workspace(c.cache, batch, 8)
    want = q.qlin_kv_attention_tree(x, c.cache, batch, 8, mask, workspace=work).clone()
    out = torch.empty_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q.qlin_tree_plan(p, batch, mask=mask, positions=positions)
        q.qlin_kv_attention_tree(x, c.cache, batch, 8, mask, out=out, workspace=work)
    for _ in range(3):
        out.zero_()
        mask.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = q.qlin_kv_attention_tree(x, c.cache, batch, 8, mask)
    side.synchronize()
    assert torch.equal(again, want)


@pytest.mark.parametrize("tokens", [0, 3])
def test_steps_without_new_tokens(tokens):
    """A batch none of whose sequences has a new token: nothing is written but counts and lengths."""
    c = Cache(6, 16, 2, 64)
    kv = [20, 0, 33]
    batch = q.KvBatch(i32(c.table(3, 2)), i32([0, 0, 0, 0]), i32(kv), max_q=0, max_kv=32)
    parents = i32(np.zeros(tokens))
    mask, positions = q.qlin_tree_plan(parents, batch, positions=torch.full((tokens,), 7, dtype=torch.int32, device=DEV))
    assert mask.shape == (tokens, 0) and positions.tolist() == [7] * tokens
    x = queries(tokens, 4 * 64, "f16", "none").to(DEV) if tokens else torch.empty((0, 256), dtype=torch.float16, device=DEV)
    out = torch.full_like(x, 5.0)
    q.qlin_kv_attention_tree(x, c.cache, batch, 4, mask, out=out)
    path, count, token = q.qlin_tree_accept(parents, parents, parents, batch)
    assert path.shape == (3, 0) and count.tolist() == [0] * 3 and token.tolist() == [-1] * 3
    assert q.qlin_kv_compact(q.KvStack([c.cache]), batch, path, count).tolist() == [20, 0, 32]
    torch.cuda.synchronize()
    assert torch.all(out == 5.0)
    for name in ("k_scale", "v_scale", "k", "v"):
        assert np.array_equal(getattr(c.cache, name).cpu().numpy(), c.host[name]), name
    # the same with room for one, and no token at all
    if tokens == 0:
        one = q.KvBatch(batch.page_table, batch.q_start, batch.kv_len, max_q=1, max_kv=32)
        mask, _ = q.qlin_tree_plan(parents, one)
        assert q.qlin_kv_attention_tree(x, c.cache, one, 4, mask).shape == (0, 256)


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}-{c[1]}-{c[2]}-{c[3]}-p{c[4]}-cap{c[5]}-{len(c[6])}")
def test_chain_and_causal_attention(case):
    """A chain's mask row is the causal one: where blocks of 16 rows take both calls the products
    and sums come in one order, and the outputs are the same bits; elsewhere both are within the
    derived tolerance of the oracle, and so of each other within its double."""
    dtype, hq, hkv, d, page, cap, seqs = case
    c, table, start, kv, _, x, batch = setup(case)
    chain = np.concatenate([np.arange(n) - 1 for n, _ in seqs])
    mask, _ = q.qlin_tree_plan(i32(chain), batch)
    tree = q.qlin_kv_attention_tree(x, c.cache, batch, hq, mask, softcap=cap)
    causal = q.qlin_kv_attention(x, c.cache, batch, hq, softcap=cap)
    torch.cuda.synchronize()
    if case in CASES[:11]:
        assert torch.equal(tree, causal)
    sees = make_sees(chain, start, max(1, batch.max_q))
    for out in (tree, causal):
        check(out, x, c, table, start, kv, hq, sees, d ** -0.5, cap, dtype)
