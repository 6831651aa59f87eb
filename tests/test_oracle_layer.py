"""Pins of the layer oracle (oracle/layer_ref.py): closed forms, invariances
and torch's own float64 routines."""

import numpy as np
import pytest
import torch

import oracle


def rng(seed):
    return np.random.default_rng(seed)


@pytest.mark.parametrize("eps", [0.0, 1e-6, 0.5])
def test_rmsnorm_is_torchs(eps):
    x, w = rng(1).standard_normal((5, 24)), rng(2).standard_normal(24).astype(np.float32)
    r, n = oracle.add_rmsnorm(x, None, w, eps, "f32")
    ref = torch.nn.functional.rms_norm(torch.from_numpy(x), (24,), torch.from_numpy(w).double(), float(np.float32(eps)))
    assert np.array_equal(r, x)
    assert np.allclose(n, ref.numpy(), rtol=1e-14, atol=0)


def test_residual_is_rounded_to_the_type_before_the_norm():
    # 1 + 2^-9 is not a bfloat16 (8 significant bits): it rounds to 1
    r, n = oracle.add_rmsnorm([[1.0, 2.0]], [[2.0 ** -9, 0.0]], np.ones(2, np.float32), 0.0, "bf16")
    assert r.tolist() == [[1.0, 2.0]]
    assert np.allclose(n, np.array([[1.0, 2.0]]) / np.sqrt(2.5), rtol=1e-15)


def test_norm_codes_by_hand():
    # max 6 -> 7 x 3 / 6 = 3.5 is a tie: to even, 4; 7 x 1 / 6 = 1.17 -> 1
    r, codes, scale = oracle.add_rmsnorm_quant([[3.0, -6.0, 1.0, 0.0]], None, np.ones(4, np.float32), 0.0, 0, 4, "f32")
    assert codes.tolist() == [[4, -7, 1, 0]]
    assert scale[0] == np.float32(6.0 / np.sqrt(46.0 / 4) / 7)


def test_norm_codes_ignore_the_rows_scale_and_zero_rows():
    x, w = rng(3).standard_normal((3, 64)), rng(4).standard_normal(64).astype(np.float32)
    _, a, sa = oracle.add_rmsnorm_quant(x, None, w, 0.0, 16, 8, "f32")
    _, b, sb = oracle.add_rmsnorm_quant(x * 8.0, None, w, 0.0, 16, 8, "f32")
    assert np.array_equal(a, b) and np.allclose(sa, sb, rtol=1e-7)
    _, z, sz = oracle.add_rmsnorm_quant(np.zeros((1, 64)), None, w, 0.0, 16, 8, "f32")
    assert not z.any() and sz[0] == 0


def test_norm_quant_is_the_unfused_chain():
    x, w = rng(5).standard_normal((4, 128)), rng(6).standard_normal(128).astype(np.float32)
    _, n = oracle.add_rmsnorm(x, None, w, 1e-5, "f32")
    want, s_want, _ = oracle.rotate_quant_act(n, None, 32, 8)
    _, codes, scale = oracle.add_rmsnorm_quant(x, None, w, 1e-5, 32, 8, "f32")
    assert np.max(np.abs(codes - want)) <= 1 and np.mean(codes != want) < 1e-2   # the chain divides by the rounded scale
    assert np.allclose(scale, s_want, rtol=1e-7)


# ---- rotary positions and the paged cache

@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_is_a_complex_product_and_keeps_distances(interleaved):
    d, rot = 16, 8
    x, y = rng(7).standard_normal(d), rng(8).standard_normal(d)
    t = oracle.rope_table(40, rot)
    row = t[11].astype(np.float64)
    a = np.arange(rot // 2) * 2 if interleaved else np.arange(rot // 2)
    b = a + 1 if interleaved else a + rot // 2
    z = (x[a] + 1j * x[b]) * (row[:rot // 2] + 1j * row[rot // 2:])
    got = oracle.rope(x, t[11], rot, interleaved)
    assert np.allclose(got[a], z.real, rtol=1e-14) and np.allclose(got[b], z.imag, rtol=1e-14)
    assert np.array_equal(got[rot:], x[rot:])
    # scores depend on the distance of two positions only
    s = [oracle.rope(x, t[p + 3], rot, interleaved) @ oracle.rope(y, t[p], rot, interleaved) for p in (0, 9, 30)]
    assert np.allclose(s, s[0], atol=1e-6)


def test_rope_table_is_torchs_and_stretches():
    t = oracle.rope_table(50, 12, base=500.0, stretch=2.0)
    p = torch.arange(50, dtype=torch.float64)[:, None] / 2.0 / 500.0 ** (torch.arange(0, 12, 2, dtype=torch.float64) / 12)
    assert np.allclose(t, torch.cat([p.cos(), p.sin()], 1).numpy(), atol=1e-7)
    assert np.allclose(t[::2], oracle.rope_table(25, 12, base=500.0), atol=1e-7)


def empty_cache(pages, heads, page, d):
    return dict(k=np.full((pages, heads, page, d), 77, np.int8), v=np.full((pages, heads, d, page), 77, np.int8),
                k_scale=np.full((pages, heads), 9.0, np.float32), v_scale=np.full((pages, heads), 9.0, np.float32))


def test_append_by_hand():
    # one head, d = 4, pages of 4 in the order 2, 0; q k v a token
    c = empty_cache(3, 1, 4, 4)
    x = np.zeros((5, 12))
    x[:, 4] = [127.0, 254.0, 1.0, -3.0, 5.0]          # k: the page of the first four has scale 2
    x[:, 8] = 1.27
    q = oracle.rope_append_kv(x, c, [[2, 0]], [0, 5], [5], 1, None, 0, False)
    assert c["k_scale"][2, 0] == 2.0 and c["k"][2, 0, :, 0].tolist() == [64, 127, 0, -2]   # 63.5 and 0.5, -1.5: to even
    assert c["k_scale"][0, 0] == np.float32(5 / 127) and c["k"][0, 0, 0, 0] == 127 and c["k"][0, 0, 1, 0] == 77
    assert c["v"][2, 0, 0].tolist() == [127] * 4 and c["v"][0, 0, 0].tolist() == [127, 77, 77, 77]
    assert c["k_scale"][1, 0] == 9.0 and np.array_equal(q, x[:, :4])
    # one more token, twice as large: the page's scale doubles and its code halves (63.5 -> 64)
    x2 = np.zeros((1, 12))
    x2[0, 4] = 10.0
    oracle.rope_append_kv(x2, c, [[2, 0]], [0, 1], [6], 1, None, 0, False)
    assert c["k_scale"][0, 0] == np.float32(10 / 127) and c["k"][0, 0, :2, 0].tolist() == [64, 127]
    before = {n: a.copy() for n, a in c.items()}
    oracle.rope_append_kv(x2, c, [[2, 0]], [0, 1], [6], 1, None, 0, False)
    assert all(np.array_equal(before[n], c[n]) for n in c)


def test_append_bounds_the_stored_error():
    # a page filled at once: every stored value within half a step of its own
    c = empty_cache(2, 2, 16, 8)
    x = rng(9).standard_normal((16, 6 * 8))
    oracle.rope_append_kv(x, c, [[1]], [0, 16], [16], 2, None, 0, False)
    k = x.reshape(16, 6, 8)[:, 2:4].transpose(1, 0, 2)
    v = x.reshape(16, 6, 8)[:, 4:].transpose(1, 2, 0)
    for codes, scale, ref in ((c["k"][1], c["k_scale"][1], k), (c["v"][1], c["v_scale"][1], v)):
        assert np.all(np.abs(codes * scale[:, None, None] - ref) <= 0.5000001 * scale[:, None, None])


def test_append_keeps_damaged_values_out_of_the_scale():
    c = empty_cache(1, 1, 16, 4)
    x = np.zeros((2, 12))
    x[0, 4:8] = [np.inf, -np.inf, np.nan, 127.0]
    oracle.rope_append_kv(x, c, [[0]], [0, 2], [2], 1, None, 0, False)
    assert c["k_scale"][0, 0] == 1.0 and c["k"][0, 0, 0].tolist() == [127, -127, 0, 127]


# ---- attention over the paged cache

def filled(pages, heads, page, d, seed=3):
    g = np.random.default_rng(seed)
    return dict(k=g.integers(-127, 128, (pages, heads, page, d), dtype=np.int8),
                v=g.integers(-127, 128, (pages, heads, d, page), dtype=np.int8),
                k_scale=g.uniform(0.005, 0.02, (pages, heads)).astype(np.float32),
                v_scale=g.uniform(0.005, 0.02, (pages, heads)).astype(np.float32))


@pytest.mark.parametrize("prefix", [None, 0, 6, 11])
def test_attention_is_torchs(prefix):
    heads, group, d, page, n, kv = 2, 2, 8, 4, 5, 11
    c = filled(5, heads, page, d)
    table = [[3, 0, 4]]
    x = rng(10).standard_normal((n, heads * group * d))
    got = oracle.kv_attention(x, c, table, [0, n], [kv], heads * group, 0.3, 0.0, None if prefix is None else [prefix])
    k = np.concatenate([c["k"][p].astype(float) * c["k_scale"][p][:, None, None] for p in table[0]], 1)[:, :kv]
    v = np.concatenate([(c["v"][p].astype(float) * c["v_scale"][p][:, None, None]).transpose(0, 2, 1) for p in table[0]], 1)[:, :kv]
    mask = torch.ones(n, kv).tril(kv - n).bool()
    mask[:, :prefix or 0] = True
    q = torch.from_numpy(x.reshape(n, heads, group, d)).permute(1, 2, 0, 3)
    ref = torch.nn.functional.scaled_dot_product_attention(
        q, torch.from_numpy(k)[:, None].expand(-1, group, -1, -1), torch.from_numpy(v)[:, None].expand(-1, group, -1, -1),
        attn_mask=mask, scale=0.3)
    assert np.allclose(got, ref.permute(2, 0, 1, 3).reshape(n, -1).numpy(), rtol=1e-12)


def test_attention_corner_rows():
    c = filled(2, 1, 4, 8)
    x = rng(11).standard_normal((3, 8))
    # the first of three queries stands in front of the cache; a page outside the pool hides its keys
    got = oracle.kv_attention(x, c, [[0]], [0, 3], [2], 1, 1.0)
    assert not got[0].any() and np.allclose(got[1], c["v"][0, 0, :, 0] * np.float64(c["v_scale"][0, 0]), rtol=1e-12)
    assert not oracle.kv_attention(x, c, [[9]], [0, 3], [3], 1, 1.0).any()
    # a very small cap makes every score the same: the mean of the values
    got = oracle.kv_attention(x[:1], c, [[1]], [0, 1], [4], 1, 1.0, softcap=1e-12)
    assert np.allclose(got[0], c["v"][1, 0].astype(float).mean(1) * c["v_scale"][1, 0], rtol=1e-9)
