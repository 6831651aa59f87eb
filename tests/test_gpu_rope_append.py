"""The rotary append to the paged int8 cache against the float64 oracle (GPU
only).

Scales and codes come from float64 values that are exact (a 16-bit input times
an fp32 cosine) or one rounding of their sum, on both sides the same, and are
compared for equality; so is everything a call must leave alone.  q is turned
in fp32: each product rounds once (2^-24 of it), their sum once, then the
output's half step.
"""

import numpy as np
import pytest
import torch

import bit_ptq_vla_amd as q
import oracle
from bit_ptq_vla_amd import synth

pytestmark = pytest.mark.gpu
DEV = "cuda"
SEED = 977
DT = {"f16": torch.float16, "bf16": torch.bfloat16}
HALF_STEP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


class Pool:
    """A library cache and its NumPy twin, with the same arbitrary start."""

    def __init__(self, pages, page, heads, d, seed=5):
        g = np.random.default_rng(seed)
        self.host = dict(k=g.integers(-127, 128, (pages, heads, page, d), dtype=np.int8),
                         v=g.integers(-127, 128, (pages, heads, d, page), dtype=np.int8),
                         k_scale=g.uniform(0.001, 0.003, (pages, heads)).astype(np.float32),
                         v_scale=g.uniform(0.001, 0.003, (pages, heads)).astype(np.float32))
        dev = {n: torch.from_numpy(a.copy()).to(DEV) for n, a in self.host.items()}
        self.cache = q.KvCache(dev["k"], dev["k_scale"], dev["v"], dev["v_scale"])
        self.order = g.permutation(pages)

    def table(self, batch, cols):
        return self.order[:batch * cols].reshape(batch, cols).astype(np.int32)

    def same(self):
        c = self.cache
        for name, t in (("k_scale", c.k_scale), ("v_scale", c.v_scale), ("k", c.k), ("v", c.v)):
            assert np.array_equal(t.cpu().numpy(), self.host[name]), name


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


def inputs(tokens, cols, dtype, tag):
    x = synth.normal_tensor(SEED, f"append/{tag}/{tokens}", (tokens, cols), dtype=dtype, outliers=max(1, cols // 50),
                            outlier_scale=8.0)
    return x


def check_q(out, want, x, hq, d, dtype, rows):
    got, ref = f64(out)[rows], want[rows]
    # |a cos| + |b sin| <= the two inputs' magnitudes
    mag = np.abs(f64(x)[rows][:, :hq * d]).reshape(-1, hq, d).max(axis=2, keepdims=True).repeat(d, 2).reshape(ref.shape)
    tiny = 2.0 ** -25 if dtype == "f16" else 0.0
    tol = 2.0 ** -24 * (2 * mag + np.abs(ref)) + HALF_STEP[dtype] * np.abs(ref) * (1 + 2.0 ** -12) + tiny
    assert np.all(np.abs(got - ref) <= tol)


def append(pool, x, table, q_start, kv_len, hq, rope, inter, positions=None, max_q=None, max_kv=None, q_out=None):
    n = np.diff(q_start)
    b = q.KvBatch(i32(table), i32(q_start), i32(kv_len), max_q=max_q if max_q is not None else int(n.max()),
                  max_kv=max_kv if max_kv is not None else table.shape[1] * pool.cache.page_size)
    return q.qlin_rope_append_kv(x.to(DEV), pool.cache, b, hq,
                                 None if rope is None else torch.from_numpy(rope).to(DEV), interleaved=inter,
                                 positions=None if positions is None else i32(positions), q_out=q_out)


CASES = [
    # dtype, hq, hkv, d, page, rot, interleaved, (new, cached) of each sequence
    ("f16", 2, 2, 128, 16, 128, False, [(1, 0)]),
    ("f16", 4, 4, 128, 16, 128, False, [(1, 30)]),
    ("bf16", 8, 2, 64, 32, 64, True, [(1, 31), (1, 32), (1, 33), (1, 0), (0, 5), (0, 0)]),
    ("bf16", 2, 1, 256, 64, 256, False, [(70, 0), (1, 100), (64, 64), (129, 3)]),
    ("f16", 3, 1, 64, 16, 32, True, [(17, 0), (16, 16), (15, 17), (33, 15)]),
    ("bf16", 1, 1, 128, 64, 48, False, [(5, 61), (3, 62)]),
    ("f16", 2, 2, 256, 32, 128, True, [(31, 0), (40, 7)]),
    ("bf16", 4, 4, 64, 64, 0, False, [(9, 60), (2, 1)]),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}-{c[1]}-{c[2]}-{c[3]}-p{c[4]}-r{c[5]}-{c[6]}")
def test_append(case):
    dtype, hq, hkv, d, page, rot, inter, seqs = case
    new, ctx = [n for n, _ in seqs], [c for _, c in seqs]
    kv = np.array(new) + np.array(ctx)
    cols = max(1, -(-int(kv.max()) // page))
    pool = Pool(len(seqs) * cols + 2, page, hkv, d)
    table = pool.table(len(seqs), cols)
    q_start = np.concatenate([[0], np.cumsum(new)])
    tokens = int(q_start[-1])
    x = inputs(tokens, (hq + 2 * hkv) * d, dtype, str(case))
    rope = oracle.rope_table(int(kv.max()) + 1, rot) if rot else None
    out = append(pool, x, table, q_start, kv, hq, rope, inter)
    torch.cuda.synchronize()
    want = oracle.rope_append_kv(f64(x), pool.host, table, q_start, kv, hq, rope, rot, inter)
    pool.same()
    check_q(out, want, x, hq, d, dtype, np.arange(tokens))
    # once more: nothing changes
    append(pool, x, table, q_start, kv, hq, rope, inter)
    torch.cuda.synchronize()
    pool.same()


def test_token_by_token_grows_the_scales():
    hq, hkv, d, page = 2, 1, 64, 16
    pool = Pool(6, page, hkv, d)
    table = pool.table(2, 3)
    rope = oracle.rope_table(48, d)
    for t in range(37):
        x = inputs(2, (hq + 2 * hkv) * d, "bf16", f"step{t}") * (1.0 + 0.2 * (t % 16))     # growth inside every page
        kv = np.array([t + 1, max(0, t - 5)])
        q_start = np.array([0, 1, 2 if t >= 6 else 1])
        append(pool, x, table, q_start, kv, hq, rope, False)
        torch.cuda.synchronize()
        oracle.rope_append_kv(f64(x), pool.host, table, q_start, kv, hq, rope, d, False)
        pool.same()


def test_given_positions_and_their_bounds():
    hq, hkv, d, page = 2, 1, 64, 32
    pool = Pool(3, page, hkv, d)
    table = pool.table(1, 2)
    x = inputs(7, (hq + 2 * hkv) * d, "f16", "pos")
    rope = oracle.rope_table(20, 32)
    pos = np.array([3, 0, 19, 20, 1 << 30, -1, -(1 << 31)])            # past either end: the end's row
    out = append(pool, x, table, np.array([0, 7]), np.array([40]), hq, rope, True, positions=pos)
    torch.cuda.synchronize()
    want = oracle.rope_append_kv(f64(x), pool.host, table, [0, 7], [40], hq, rope, 32, True, positions=pos)
    pool.same()
    check_q(out, want, x, hq, d, "f16", np.arange(7))


def test_damaged_metadata_stays_inside_the_pool():
    # index arithmetic of the same cases: test_index_arithmetic_stays_in_bounds
    hq, hkv, d, page = 2, 2, 64, 16
    pool = Pool(9, page, hkv, d)
    table = pool.table(4, 2)
    table[0, 1] = 9            # behind the pool
    table[1, 0] = -1
    table[2, 1] = 1 << 30
    q_start = np.array([0, 20, 24, 44, 50])
    kv = np.array([20, 4, 32, 3])                    # the last: six new tokens, three of them in front of the cache
    x = inputs(50, (hq + 2 * hkv) * d, "bf16", "bad")
    rope = oracle.rope_table(32, 64)
    append(pool, x, table, q_start, kv, hq, rope, False)
    torch.cuda.synchronize()
    oracle.rope_append_kv(f64(x), pool.host, table, q_start, kv, hq, rope, 64, False)
    pool.same()


def test_infinities_and_nans_stay_out_of_the_scale():
    hq, hkv, d, page = 1, 1, 64, 16
    pool = Pool(2, page, hkv, d)
    table = pool.table(1, 2)
    x = inputs(19, 3 * d, "f16", "nan")
    x[2, d + 4] = float("inf")
    x[3, d + 40] = float("nan")
    x[17, 2 * d + 1] = -float("inf")
    x[18, 2 * d + 2] = float("nan")
    rope = oracle.rope_table(19, 32)
    append(pool, x, table, np.array([0, 19]), np.array([19]), hq, rope, False)
    torch.cuda.synchronize()
    with np.errstate(invalid="ignore"):
        oracle.rope_append_kv(f64(x), pool.host, table, [0, 19], [19], hq, rope, 32, False)
    pool.same()
    assert torch.isfinite(pool.cache.k_scale).all() and torch.isfinite(pool.cache.v_scale).all()


def test_pitched_rows_and_rows_of_no_sequence():
    hq, hkv, d, page = 2, 1, 64, 16
    cols = (hq + 2 * hkv) * d
    pool = Pool(4, page, hkv, d)
    table = pool.table(1, 2)
    x = inputs(9, cols, "bf16", "pitch")
    wide = torch.zeros((9, cols + 24), dtype=torch.bfloat16, device=DEV)
    wide[:, :cols] = x.to(DEV)
    out = torch.full((9, hq * d + 8), 5.0, dtype=torch.bfloat16, device=DEV)
    rope = oracle.rope_table(32, 64)
    q_start = np.array([2, 7])                       # rows 0, 1 and 7, 8 belong to nobody
    append(pool, wide[:, :cols], table, q_start, np.array([20]), hq, rope, False, q_out=out[:, :hq * d])
    torch.cuda.synchronize()
    want = oracle.rope_append_kv(f64(x), pool.host, table, q_start, [20], hq, rope, 64, False)
    pool.same()
    check_q(out[:, :hq * d], want, x, hq, d, "bf16", np.arange(2, 7))
    assert torch.all(out[:2] == 5.0) and torch.all(out[7:] == 5.0) and torch.all(out[:, hq * d:] == 5.0)


def test_stream_and_replayed_graph():
    hq, hkv, d, page = 4, 2, 64, 16
    pool = Pool(5, page, hkv, d)
    table = pool.table(2, 2)
    rope = oracle.rope_table(32, 64)
    x = inputs(2, (hq + 2 * hkv) * d, "f16", "graph").to(DEV)
    kv = i32([1, 7])
    b = q.KvBatch(i32(table), i32([0, 1, 2]), kv, max_q=1, max_kv=32)
    rope_d = torch.from_numpy(rope).to(DEV)
    out = torch.empty((2, hq * d), dtype=torch.float16, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        q.qlin_rope_append_kv(x, pool.cache, b, hq, rope_d, q_out=out)
    side.synchronize()
    oracle.rope_append_kv(f64(x), pool.host, table, [0, 1, 2], [1, 7], hq, rope, 64, False)
    pool.same()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q.qlin_rope_append_kv(x, pool.cache, b, hq, rope_d, q_out=out)
    for t in range(4):                               # the graph reads the lengths: later tokens, new contents
        x.copy_(inputs(2, (hq + 2 * hkv) * d, "f16", f"graph{t}"))
        kv.copy_(torch.tensor([2 + 6 * t, 8 + 6 * t]))
        g.replay()
        torch.cuda.synchronize()
        want = oracle.rope_append_kv(f64(x), pool.host, table, [0, 1, 2], kv.cpu().numpy(), hq, rope, 64, False)
        pool.same()
        check_q(out, want, x, hq, d, "f16", np.arange(2))


def test_refused_calls():
    pool = Pool(4, 16, 1, 64)
    table = i32(pool.table(1, 2))
    x = torch.zeros((2, 3 * 64), dtype=torch.float16, device=DEV)
    rope = torch.zeros((32, 64), device=DEV)
    with pytest.raises(ValueError):                  # the table's rows do not hold max_kv
        q.qlin_rope_append_kv(x, pool.cache, q.KvBatch(table, i32([0, 2]), i32([2]), max_q=2, max_kv=33), 1, rope)
    b = q.KvBatch(table, i32([0, 2]), i32([2]), max_q=2, max_kv=32)
    with pytest.raises(ValueError):
        q.qlin_rope_append_kv(x[:, :128], pool.cache, b, 1, rope)
    with pytest.raises(ValueError):
        q.qlin_rope_append_kv(x, pool.cache, b, 1, rope.half())
    with pytest.raises(ValueError):
        q.qlin_rope_append_kv(x, pool.cache, b, 1, rope.cpu())
    with pytest.raises(q.QlinError):
        q.qlin_rope_append_kv(x.float(), pool.cache, b, 1, rope)
    with pytest.raises(q.QlinError):
        q.qlin_rope_append_kv(x, pool.cache, b, 1, torch.zeros((32, 24), device=DEV))
    with pytest.raises(ValueError):
        q.KvBatch(table.long(), i32([0, 2]), i32([2]), max_q=2, max_kv=32)
    with pytest.raises(ValueError):
        q.KvCache(pool.cache.k, pool.cache.k_scale, pool.cache.k, pool.cache.v_scale)


@pytest.mark.parametrize("n,rot,base,stretch", [(1, 2, 10000.0, 1.0), (200, 128, 10000.0, 1.0), (70000, 64, 5e5, 4.0)])
def test_rope_table(n, rot, base, stretch):
    t = q.qlin_rope_table(n, rot, base=base, stretch=stretch)
    torch.cuda.synchronize()
    # float64 angles up to n, whose own rounding is 2^-53 n; then one fp32 rounding each
    assert np.all(np.abs(f64(t) - oracle.rope_table(n, rot, base, stretch).astype(np.float64)) <= 2.0 ** -24 + 2.0 ** -50 * n)


@pytest.mark.parametrize("d,page,held,ratio", [(128, 64, 45, 0.5), (64, 32, 31, 0.25), (256, 16, 15, 0.5), (128, 64, 63, 3 / 254),
                                               (64, 64, 1, -2.0), (128, 32, 17, 0.0), (256, 64, 50, 1e-30)])
def test_held_codes_follow_the_scale(d, page, held, ratio):
    """A page's earlier codes when its scale rises: all of them ties (ratios of
    1/2, 1/4), far below the new scale, and scales no append leaves behind."""
    pool = Pool(3, page, 2, d)
    pool.host["k"][:] = (np.arange(pool.host["k"].size) % 255 - 127).reshape(pool.host["k"].shape)
    pool.host["v"][:] = (np.arange(pool.host["v"].size) % 255 - 127).reshape(pool.host["v"].shape)
    pool.host["k_scale"][:] = pool.host["v_scale"][:] = np.float32(ratio * 2.0 ** -7)
    for n, t in (("k", pool.cache.k), ("v", pool.cache.v), ("k_scale", pool.cache.k_scale), ("v_scale", pool.cache.v_scale)):
        t.copy_(torch.from_numpy(pool.host[n]))
    x = torch.zeros((1, 6 * d), dtype=torch.float16)
    x[0, ::d] = 127 * 2.0 ** -7          # the new scale is 2^-7
    append(pool, x, pool.table(1, 1), np.array([0, 1]), np.array([held + 1]), 2, None, False)
    torch.cuda.synchronize()
    oracle.rope_append_kv(f64(x), pool.host, pool.table(1, 1), np.array([0, 1]), np.array([held + 1]), 2, None, 0, False)
    pool.same()


@pytest.mark.parametrize("size", [2.0 ** -133, 2.0 ** -126, 2.0 ** -110, 2.0 ** 126])
def test_values_at_the_ends_of_the_range(size):
    """bf16 values whose turned products leave fp32's normal range (the oracle is exact there too)."""
    d, page = 64, 16
    pool = Pool(4, page, 1, d)
    x = (inputs(18, 3 * d, "bf16", "ends").to(torch.float64).clamp(-3.5, 3.5) * size).to(torch.bfloat16)
    rope = oracle.rope_table(32, d)
    append(pool, x, pool.table(1, 3), np.array([0, 18]), np.array([25]), 1, rope, False)
    torch.cuda.synchronize()
    with np.errstate(over="ignore"):
        oracle.rope_append_kv(f64(x), pool.host, pool.table(1, 3), np.array([0, 18]), np.array([25]), 1, rope, d, False)
    pool.same()
