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


def rope_table(positions: int, rot: int, base: float = 10000.0, stretch: float = 1.0) -> np.ndarray:
    """float32 [positions][rot]: cosines then sines of p / stretch * base^(-2 i / rot)."""
    i = np.arange(rot // 2, dtype=np.float64)
    angle = np.arange(positions, dtype=np.float64)[:, None] / stretch * base ** (-2.0 * i / rot)
    return np.concatenate([np.cos(angle), np.sin(angle)], axis=1).astype(np.float32)


def rope(x, row, rot: int, interleaved: bool):
    """One head's vector x [d] turned by a table row (float32 [rot]), float64."""
    y = np.array(x, dtype=np.float64)
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        c, s = float(row[i]), float(row[rot // 2 + i])
        y[a], y[b] = x[a] * c - x[b] * s, x[b] * c + x[a] * s
    return y


def _codes(v, s):
    """rne(v / s) in -127 .. 127; infinities at the ends, NaN and a zero scale as 0."""
    v = np.asarray(v, dtype=np.float64)
    if not s > 0:
        return np.zeros(v.shape, dtype=np.int8)
    return np.clip(np.rint(np.where(np.isnan(v), 0.0, v) / np.float64(s)), -127, 127).astype(np.int8)


def _store(codes, scale, new, held: int):
    """One (page, head), token-major codes [page][d] changed in place: new
    [n][d] behind `held` tokens; returns the new scale (float32)."""
    finite = np.abs(new[np.isfinite(new)])
    fresh = np.float32((finite.max() if finite.size else 0.0) / 127.0)
    old = np.float32(scale) if held else np.float32(0)
    s = max(old, fresh)
    if held and s != old:
        codes[:held] = _codes(codes[:held].astype(np.float64) * np.float64(old), s)
    codes[held:held + len(new)] = _codes(new, s)
    return s


def rope_append_kv(qkv, cache, table, q_start, kv_len, heads_q: int, rope_rows, rot: int, interleaved: bool,
                   positions=None):
    """qkv float64 [tokens][(hq + 2 h) d]; cache = dict(k, v, k_scale, v_scale) of
    NumPy arrays in the library's layout, changed in place.  Returns q float64
    [tokens][hq d] (rows of no sequence NaN)."""
    k, v, ks, vs = cache["k"], cache["v"], cache["k_scale"], cache["v_scale"]
    pages, heads, page, d = k.shape
    x = np.asarray(qkv, dtype=np.float64).reshape(len(qkv), heads_q + 2 * heads, d)
    out = np.full((len(qkv), heads_q, d), np.nan)
    for b in range(len(kv_len)):
        n, kv = int(q_start[b + 1] - q_start[b]), int(kv_len[b])
        first, row0 = kv - n, int(q_start[b])
        turned = {}
        for i in range(n):
            pos = int(positions[row0 + i]) if positions is not None else first + i
            row = rope_rows[min(max(pos, 0), len(rope_rows) - 1)] if rot else None
            y = [rope(x[row0 + i, h], row, rot, interleaved) if rot else x[row0 + i, h] for h in range(heads_q + heads)]
            out[row0 + i] = y[:heads_q]
            turned[first + i] = y[heads_q:]
        j = max(first, 0)
        while j < kv:
            end = min(kv, (j // page + 1) * page)
            at = int(table[b][j // page])
            if 0 <= at < pages:
                for h in range(heads):
                    held = j % page
                    ks[at, h] = _store(k[at, h], ks[at, h], np.array([turned[t][h] for t in range(j, end)]), held)
                    new = np.array([x[row0 + t - first, heads_q + heads + h] for t in range(j, end)])
                    vs[at, h] = _store(v[at, h].T, vs[at, h], new, held)
            j = end
    return out.reshape(len(qkv), heads_q * d)


def kv_attention(q, cache, table, q_start, kv_len, heads_q: int, sm_scale: float, softcap: float = 0.0,
                 prefix_len=None):
    """q float64 [tokens][hq d] over the cache (layout of rope_append_kv's), one
    query at a time.  Returns float64 [tokens][hq d], rows of no sequence NaN."""
    k, v, ks, vs = cache["k"], cache["v"], cache["k_scale"], cache["v_scale"]
    pages, heads, page, d = k.shape
    x = np.asarray(q, dtype=np.float64).reshape(len(q), heads_q, d)
    out = np.full(x.shape, np.nan)
    for b in range(len(kv_len)):
        n, kv = int(q_start[b + 1] - q_start[b]), int(kv_len[b])
        j = np.arange(kv)
        at = np.array([int(table[b][i // page]) for i in j], dtype=np.int64)
        there = (at >= 0) & (at < pages)
        at = np.where(there, at, 0)
        for h in range(heads):
            kh = k[at, h, j % page].astype(np.float64) * ks[at, h].astype(np.float64)[:, None]
            vh = v[at, h, :, j % page].astype(np.float64) * vs[at, h].astype(np.float64)[:, None]
            for i in range(n):
                pos = kv - n + i
                seen = there & ((j <= pos) | (j < (int(prefix_len[b]) if prefix_len is not None else 0)))
                for g in range(heads_q // heads):
                    head = h * (heads_q // heads) + g
                    if not seen.any():
                        out[q_start[b] + i, head] = 0.0
                        continue
                    s = kh[seen] @ x[q_start[b] + i, head] * sm_scale
                    if softcap:
                        s = softcap * np.tanh(s / softcap)
                    w = np.exp(s - s.max())
                    out[q_start[b] + i, head] = w @ vh[seen] / w.sum()
    return out.reshape(len(q), heads_q * d)
