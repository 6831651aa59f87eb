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
