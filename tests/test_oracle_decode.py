"""The oracle of decoding with drafted tokens, pinned by hand-worked cases and by
other routes to the same answer."""

import itertools

import numpy as np
import pytest

import oracle


def test_tree_sees_by_powers_of_the_parent_matrix():
    parents = [-1, 0, 0, 1, 1, 2, 9, 5]               # node 6 names no earlier node: a root
    n = len(parents)
    a = np.zeros((n, n), dtype=int)
    for i, p in enumerate(parents):
        if 0 <= p < i:
            a[i, p] = 1
    want = sum(np.linalg.matrix_power(a, k) for k in range(n)) > 0
    assert np.array_equal(oracle.tree_sees(parents), want)


def test_tree_accept_by_hand():
    #        0 -> 1 (7), 2 (8); 2 -> 3 (9), 4 (9); 4 -> 5 (1)
    parents, draft = [-1, 0, 0, 2, 2, 4], [0, 7, 8, 9, 9, 1]
    assert oracle.tree_accept(parents, draft, [8, 0, 9, 5, 1, 2]) == ([0, 2, 3], 5)
    assert oracle.tree_accept(parents, draft, [6, 0, 9, 5, 1, 2]) == ([0], 6)
    assert oracle.tree_accept([], [], []) == ([], -1)


def test_sample_by_hand():
    x = np.log(np.array([1.0, 4.0, 2.0, 1.0]))         # order 1, 2, 0, 3; masses 4, 2, 1, 1 of 8
    got = [oracle.sample(x, u)[0] for u in (0.0, 0.49, 0.51, 0.74, 0.76, 0.87, 0.88, 0.999)]
    assert got == [1, 1, 2, 2, 0, 0, 3, 3]
    assert [oracle.sample(x, u, top_k=2)[0] for u in (0.66, 0.67)] == [1, 2]
    assert [oracle.sample(x, u, top_p=0.6)[0] for u in (0.66, 0.67)] == [1, 2]
    assert [oracle.sample(x, u, top_p=0.45)[0] for u in (0.0, 0.99)] == [1, 1]
    assert [oracle.sample(x, u, min_p=0.4)[0] for u in (0.66, 0.67)] == [1, 2]
    assert oracle.sample(x, 0.9, temperature=0.0)[:2] == (1, 0.0)
    assert oracle.sample(x, 0.3)[1] == pytest.approx(np.log(0.5))
    assert oracle.sample(2 * x, 0.7, temperature=2.0)[0] == 2
    assert oracle.sample([-np.inf, np.nan])[0] == -1
    assert oracle.sample([np.inf, 1.0, np.inf], 0.6)[0] == 2


def test_attention_of_a_chain_is_causal_attention():
    g = np.random.default_rng(1)
    cache = dict(k=g.integers(-127, 128, (6, 1, 16, 64)).astype(np.int8), v=g.integers(-127, 128, (6, 1, 64, 16)).astype(np.int8),
                 k_scale=np.full((6, 1), 0.01, np.float32), v_scale=np.full((6, 1), 0.02, np.float32))
    q = g.standard_normal((9, 128))
    table, start, kv = np.array([[3, 1], [0, 5]]), [0, 4, 9], [20, 5]
    sees = np.zeros((9, 8), dtype=bool)
    for b, n in enumerate((4, 5)):
        sees[start[b]:start[b] + n, :n] = oracle.tree_sees(range(-1, n - 1))
    got = oracle.kv_attention_tree(q, cache, table, start, kv, 2, sees, 0.125)
    assert np.allclose(got, oracle.kv_attention(q, cache, table, start, kv, 2, 0.125), rtol=1e-13, atol=1e-13)


def test_compact_keeps_the_values_that_the_new_scales_can_hold():
    g = np.random.default_rng(2)
    c = dict(k=g.integers(-127, 128, (4, 2, 16, 64)).astype(np.int8), v=g.integers(-127, 128, (4, 2, 64, 16)).astype(np.int8),
             k_scale=(0.01 + 0.01 * g.random((4, 2))).astype(np.float32), v_scale=(0.01 + 0.01 * g.random((4, 2))).astype(np.float32))
    table = [[2, 0, 3]]

    def value(c, pos):
        p = table[0][pos // 16]
        return (c["k"][p, :, pos % 16] * c["k_scale"][p][:, None].astype(float),
                c["v"][p, :, :, pos % 16] * c["v_scale"][p][:, None].astype(float))

    was = {n: a.copy() for n, a in c.items()}
    nodes = [0, 3, 4, 9, 20, 21]
    assert oracle.kv_compact([c], table, [0, 30], [43], [nodes], [6]) == [19]
    for i, a in itertools.chain(enumerate(nodes, 13), ((p, p - 13) for p in range(13))):
        for x, y, s in zip(value(c, i), value(was, 13 + a), (c["k_scale"], c["v_scale"])):
            assert np.all(np.abs(x - y) <= s[table[0][i // 16]][:, None] * 0.5 * (1 + 1e-9))


def test_pool_by_hand():
    p = oracle.Pool(5, 3, 3, 16)
    assert p.resize([0, 0, 0], [20, 0, 0]) == ([20, 0, 0], [(-1, -1)] * 3)
    assert p.table[0].tolist() == [0, 1, -1] and p.refs.tolist() == [1, 1, 0, 0, 0]
    p.fork([0, 0], [1, 2], [20, 20])
    assert p.refs.tolist() == [3, 3, 0, 0, 0]
    # the first two of three growing holders copy the shared last page
    assert p.resize([20] * 3, [21] * 3) == ([21] * 3, [(1, 2), (1, 3), (-1, -1)])
    assert p.refs.tolist() == [3, 1, 1, 1, 0] and p.table.tolist() == [[0, 2, -1], [0, 3, -1], [0, 1, -1]]
    # one page is left: the first growth takes it, later ones stay
    assert p.resize([21, 21, 21], [21, 33, 40]) == ([21, 33, 21], [(-1, -1)] * 3)
    assert p.resize([21, 33, 21], [0, 3, 40])[0] == [0, 3, 40]
    assert p.refs.tolist() == [2, 1, 1, 0, 0] and p.table.tolist() == [[-1] * 3, [0, -1, -1], [0, 1, 2]]
