"""Plain float64 forms of what stands between the projections of a layer:
residual addition and RMS norm with the activation quantizer, rotary positions
with the append to a paged int8 cache, and attention over that cache.

TEST INFRASTRUCTURE ONLY.  NumPy, one sequence / page / head at a time; shares
no code with the HIP path.
"""

from __future__ import annotations

import numpy as np

from .qlin_ref import qmax_of, rotate_blocks, round_output


def add_rmsnorm(x, residual, weight, eps: float, dtype: str):
    """r = round_T(x + residual) (x where residual is None) and
    n = r * weight / sqrt(mean(r^2) + eps), both float64."""
    x = np.asarray(x, dtype=np.float64)
    r = x if residual is None else round_output((x + np.asarray(residual, dtype=np.float64)).astype(np.float32), dtype)
    ms = np.mean(r * r, axis=1, keepdims=True) + float(np.float32(eps))
    with np.errstate(divide="ignore", invalid="ignore"):
        n = np.where(ms > 0, r * np.asarray(weight, dtype=np.float32).astype(np.float64) / np.sqrt(ms), 0.0)
    return r, n


def add_rmsnorm_quant(x, residual, weight, eps: float, had_block: int, bits: int, dtype: str):
    """Returns (r, codes int64, scale float32).  The codes are rne(qmax * v / max|v|)
    of the un-normalised row (its rms and 1/sqrt(b) cancel), on the +-1 transform,
    so that ties of exactly representable values stay ties."""
    r, n = add_rmsnorm(x, residual, weight, eps, dtype)
    qmax = qmax_of(bits)
    scale = (np.max(np.abs(rotate_blocks(n, had_block)), axis=1) / qmax).astype(np.float32)
    u = r * np.asarray(weight, dtype=np.float32).astype(np.float64)
    if had_block > 1:
        from .qlin_ref import sylvester_hadamard
        u = (u.reshape(-1, had_block) @ sylvester_hadamard(had_block).astype(np.float64)).reshape(u.shape)
    top = np.max(np.abs(u), axis=1, keepdims=True)
    codes = np.rint(np.where(top > 0, u * qmax / np.where(top > 0, top, 1.0), 0.0)).astype(np.int64)
    return r, codes, scale
