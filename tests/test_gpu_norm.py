"""The residual + RMS norm entry points against the float64 oracle (GPU only).

Codes are rounded quotients of exact values evaluated in float64, so they are
compared for equality.  Scales are one fp32 rounding of a float64 value (the
two sides' float64 values differ by a few 2^-53, which can move that rounding
by one step: 2^-23 relative).  The float output is fl(fl(r inv) w) with
inv = fl(1 / rms): three fp32 roundings (3 x 2^-24, and second-order terms)
before the rounding to its type (half a step).
"""

import numpy as np
import pytest
import torch

import bit_ptq_vla_amd as q
import oracle
from bit_ptq_vla_amd import synth

pytestmark = pytest.mark.gpu
DEV = "cuda"
SEED = 4321
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
HALF_STEP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 0.0}   # relative; f32's last rounding is one of the three


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def ints(t, bits):
    a = t.cpu().numpy()
    return {8: lambda: a.astype(np.int64), 4: lambda: oracle.unpack_int4(a),
            6: lambda: oracle.unpack_e2m3(a).astype(np.int64)}[bits]()


def make(m, k, dtype, tag=""):
    x = synth.normal_tensor(SEED, f"norm/x/{m}/{k}/{tag}", (m, k), dtype=dtype, outliers=max(1, k // 100),
                            outlier_scale=30.0)
    res = synth.normal_tensor(SEED, f"norm/r/{m}/{k}/{tag}", (m, k), dtype=dtype)
    w = 1.0 + synth.normal_tensor(SEED, f"norm/w/{k}/{tag}", (k,), std=0.25, dtype="f32")
    return x, res, w


def check_quant(got, x, res, w, eps, b, bits, dtype):
    xq, xs, r = got
    want_r, codes, scale = oracle.add_rmsnorm_quant(f64(x), None if res is None else f64(res), w.numpy(), eps, b,
                                                    4 if bits == 6 else bits, dtype)   # E2M3: the int4 grid
    if r is not None:
        assert np.array_equal(f64(r), want_r), "residual"
    assert np.array_equal(ints(xq, bits), codes), "codes"
    s = f64(xs)
    assert np.all(np.abs(s - scale) <= 2.0 ** -23 * scale), "scale"
    return codes


CASES = [
    # m, k, b, bits, dtype, residual
    (1, 4096, 0, 8, "f16", True),
    (1, 8, 0, 8, "f16", True),          # the shortest row
    (3, 24, 8, 4, "bf16", False),       # chunks behind the row's end
    (50, 1024, 64, 8, "f16", True),
    (50, 1024, 64, 4, "f16", True),
    (37, 2048, 128, 4, "bf16", True),
    (37, 2048, 128, 6, "bf16", True),
    (130, 2048, 128, 8, "bf16", True),
    (9, 512, 256, 8, "f32", True),
    (300, 256, 16, 6, "f32", False),    # several rows per block, ragged last block
    (5, 11008, 0, 8, "f16", True),      # not a power of two
    (4, 8192, 256, 8, "bf16", True),
    (3, 16384, 128, 8, "bf16", True),
    (2, 32768, 256, 4, "bf16", True),   # the longest row
    (2, 32760, 2, 8, "f16", False),
    (65, 640, 4, 8, "bf16", True),
    (33, 128, 32, 4, "f16", True),
]


@pytest.mark.parametrize("m,k,b,bits,dtype,residual", CASES)
def test_add_rmsnorm_quant(m, k, b, bits, dtype, residual):
    x, res, w = make(m, k, dtype)
    if m > 2:
        x[m // 2] = 0
        res[m // 2] = 0
    xd, rd = x.to(DEV), res.to(DEV) if residual else None
    ro = torch.empty_like(xd)
    got = q.qlin_add_rmsnorm_quant(xd, w.to(DEV), residual=rd, eps=1e-6, had_block=b, bits=bits, residual_out=ro)
    torch.cuda.synchronize()
    check_quant(got, x, res if residual else None, w, 1e-6, b, bits, dtype)
    if m > 2:
        assert got[1][m // 2].item() == 0.0


@pytest.mark.parametrize("m,k,dtype,residual", [(1, 4096, "f16", True), (7, 8, "f32", False), (50, 1024, "bf16", True),
                                                (3, 32768, "f16", True), (260, 2048, "f32", True),
                                                (5, 11008, "bf16", False)])
def test_add_rmsnorm_float(m, k, dtype, residual):
    x, res, w = make(m, k, dtype, "f")
    ro = torch.empty((m, k), dtype=DT[dtype], device=DEV)
    y, r = q.qlin_add_rmsnorm(x.to(DEV), w.to(DEV), residual=res.to(DEV) if residual else None, eps=1e-5,
                              residual_out=ro)
    torch.cuda.synchronize()
    want_r, n = oracle.add_rmsnorm(f64(x), f64(res) if residual else None, w.numpy(), 1e-5, dtype)
    assert np.array_equal(f64(r), want_r)
    tol = 3.01 * 2.0 ** -24 + HALF_STEP[dtype] * (1 + 2.0 ** -20)
    tiny = 2.0 ** -25 if dtype == "f16" else 0.0      # half of the smallest step, below the normal range
    assert np.all(np.abs(f64(y) - n) <= tol * np.abs(n) + tiny)


def test_exact_ties_go_to_even():
    # rows of small integers under a weight of ones: 127 v / max has exact halves
    k = 128
    v = torch.zeros((4, k))
    v[0, :4] = torch.tensor([254.0, 1.0, 3.0, 5.0])           # 0.5, 1.5, 2.5
    v[1, :4] = torch.tensor([-254.0, -1.0, -3.0, -7.0])       # -0.5, -1.5, -3.5
    v[2, :3] = torch.tensor([14.0, 7.0, 1.0])                 # 63.5 at int8, 3.5 at int4
    v[3] = 3.0
    w = torch.ones(k)
    for bits in (8, 4):
        got = q.qlin_add_rmsnorm_quant(v.to(DEV).half(), w.to(DEV), eps=0.0, bits=bits)
        torch.cuda.synchronize()
        codes = check_quant(got, v.half(), None, w, 0.0, 0, bits, "f16")
        if bits == 8:
            assert codes[0, :4].tolist() == [127, 0, 2, 2] and codes[1, :4].tolist() == [-127, 0, -2, -4]


def test_pitched_rows_and_updates_in_place():
    m, k = 19, 512
    x, res, w = make(m, k, "bf16", "pitch")
    xb = torch.zeros((m, k + 40), dtype=torch.bfloat16, device=DEV)
    rb = torch.full((m, k + 8), 7.0, dtype=torch.bfloat16, device=DEV)
    xb[:, :k] = x.to(DEV)
    rb[:, :k] = res.to(DEV)
    got = q.qlin_add_rmsnorm_quant(xb[:, :k], w.to(DEV), residual=rb[:, :k], had_block=64, residual_out=rb[:, :k])
    torch.cuda.synchronize()
    check_quant(got, x, res, w, 1e-6, 64, 8, "bf16")
    assert torch.all(rb[:, k:] == 7.0) and torch.equal(xb[:, :k].cpu(), x)
    # r over x
    xi = x.to(DEV)
    got = q.qlin_add_rmsnorm_quant(xi, w.to(DEV), residual=res.to(DEV), bits=4, residual_out=xi)
    torch.cuda.synchronize()
    check_quant(got, x, res, w, 1e-6, 0, 4, "bf16")


def test_rows_with_infinities_and_nans_leave_the_others_alone():
    m, k = 12, 256                      # eight rows to a block
    x, res, w = make(m, k, "f16", "nan")
    clean = q.qlin_add_rmsnorm_quant(x.to(DEV), w.to(DEV), residual=res.to(DEV), had_block=32)
    bad = x.clone()
    bad[2, 5] = float("inf")
    bad[7, 0] = float("nan")
    got = q.qlin_add_rmsnorm_quant(bad.to(DEV), w.to(DEV), residual=res.to(DEV), had_block=32)
    torch.cuda.synchronize()
    rows = [i for i in range(m) if i not in (2, 7)]
    assert torch.equal(got[0][rows], clean[0][rows]) and torch.equal(got[1][rows], clean[1][rows])
    assert not torch.isfinite(got[1][2]) and not torch.isfinite(got[1][7])


def test_large_values_do_not_overflow():
    x = torch.full((2, 64), 3e38, dtype=torch.float32)        # squares leave fp32's range
    x[1] = 1e-30
    w = torch.ones(64)
    got = q.qlin_add_rmsnorm_quant(x.to(DEV), w.to(DEV), eps=0.0, had_block=16)
    y, _ = q.qlin_add_rmsnorm(x.to(DEV), w.to(DEV), eps=0.0)
    torch.cuda.synchronize()
    check_quant(got, x, None, w, 0.0, 16, 8, "f32")
    assert np.allclose(f64(y), 1.0, rtol=4 * 2.0 ** -24)


def test_empty_and_refused_calls():
    w = torch.ones(64, device=DEV)
    e = torch.empty((0, 64), dtype=torch.float16, device=DEV)
    xq, xs, _ = q.qlin_add_rmsnorm_quant(e, w)
    assert xq.shape == (0, 64) and xs.shape == (0,)
    x = torch.zeros((2, 64), dtype=torch.float16, device=DEV)
    with pytest.raises(ValueError):
        q.qlin_add_rmsnorm_quant(x, w.half())
    with pytest.raises(ValueError):
        q.qlin_add_rmsnorm_quant(x, w, residual=x[:1])
    with pytest.raises(ValueError):
        q.qlin_add_rmsnorm_quant(x, w, residual=x.float())
    with pytest.raises(ValueError):
        q.qlin_add_rmsnorm_quant(x.t(), torch.ones(2, device=DEV))
    with pytest.raises(ValueError):
        q.qlin_add_rmsnorm_quant(x, torch.ones(64))
    with pytest.raises(q.QlinError):
        q.qlin_add_rmsnorm_quant(x.expand(2, 64)[:, :60], torch.ones(60, device=DEV))
    with pytest.raises(q.QlinError):
        q.qlin_add_rmsnorm_quant(x[:1].expand(2, 64), w)      # rows of pitch 0


def test_other_stream_and_replayed_graph():
    m, k = 50, 1024
    x, res, w = make(m, k, "bf16", "graph")
    xd, rd, wd = x.to(DEV), res.to(DEV), w.to(DEV)
    ro, xq = torch.empty_like(xd), torch.empty((m, k), dtype=torch.int8, device=DEV)
    xs = torch.empty(m, dtype=torch.float32, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def call():
        q.qlin_add_rmsnorm_quant(xd, wd, residual=rd, had_block=64, residual_out=ro, out=(xq, xs))

    with torch.cuda.stream(side):
        call()
    side.synchronize()
    check_quant((xq, xs, ro), x, res, w, 1e-6, 64, 8, "bf16")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for i in range(3):
        x2, res2, _ = make(m, k, "bf16", f"graph{i}")
        xd.copy_(x2)
        rd.copy_(res2)
        g.replay()
        torch.cuda.synchronize()
        check_quant((xq, xs, ro), x2, res2, w, 1e-6, 64, 8, "bf16")


@pytest.mark.parametrize("dtype,size", [("f32", 2.0 ** 124), ("f32", 2.0 ** -135), ("bf16", 2.0 ** 122), ("bf16", 2.0 ** -128),
                                        ("f16", 2.0 ** -22), ("f16", 2.0 ** 13)])
def test_float_rows_at_the_ends_of_the_range(dtype, size):
    """1 / rms past or near the ends of fp32's range; eps 0."""
    m, k = 3, 512
    base = synth.normal_tensor(SEED, f"norm/ends/{dtype}/{size}", (m, k), dtype="f32").clamp(-3.5, 3.5)
    x = (base.to(torch.float64) * size).to(DT[dtype])
    w = 1.0 + synth.normal_tensor(SEED, "norm/ends/w", (k,), std=0.25, dtype="f32")
    y, _ = q.qlin_add_rmsnorm(x.to(DEV), w.to(DEV), eps=0.0)
    torch.cuda.synchronize()
    _, want = oracle.add_rmsnorm(f64(x), None, w.numpy(), 0.0, dtype)
    tiny = 2.0 ** -25 if dtype == "f16" else 2.0 ** -133
    assert np.all(np.abs(f64(y) - want) <= (3 * 2.0 ** -24 * (1 + 2.0 ** -20) + HALF_STEP[dtype]) * np.abs(want) + tiny)
