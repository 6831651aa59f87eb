"""A decoder layer over the paged int8 cache (GPU only): its launches one after
the other, over a prompt and single-token steps, every stage against the
float64 oracle on the library's own input of that stage, and a captured step
against the eager one.

Codes and the cache are compared for equality, except the two quantizers of
attention and MLP values (`qlin_rotate_quant_act` has its own tests: here its
codes are within one step).  A GEMM of exact int8 sums dequantizes by two fp32
products (2 x 2^-24) before its half step of the output.
"""

import numpy as np
import pytest
import torch

import bit_ptq_vla_amd as q
import oracle
from bit_ptq_vla_amd import synth
from bit_ptq_vla_amd.workload import DecoderLayer
from test_gpu_kv_attention import Cache, check as check_attention
from test_gpu_rope_append import HALF_STEP, check_q, f64, i32

pytestmark = pytest.mark.gpu
DEV = "cuda"


def pull(cache):
    return dict(k=cache.k.cpu().numpy(), v=cache.v.cpu().numpy(), k_scale=cache.k_scale.cpu().numpy(),
                v_scale=cache.v_scale.cpu().numpy())


def check_gemm(y, codes, w, dtype):
    a, s = codes[0].cpu().numpy().astype(np.int64), f64(codes[1])
    ref = (a @ w[0].cpu().numpy().astype(np.int64).T) * s[:, None] * f64(w[1])[None, :]
    tiny = 2.0 ** -25 if dtype == "f16" else 0.0
    assert np.all(np.abs(f64(y) - ref) <= (HALF_STEP[dtype] * (1 + 2.0 ** -12) + 2.0 ** -23) * np.abs(ref) + tiny)


def check_norm(codes, residual, x, before, gamma, dtype):
    r, want, scale = oracle.add_rmsnorm_quant(f64(x), f64(before), gamma.cpu().numpy(), 1e-6, 0, 8, dtype)
    assert np.array_equal(f64(residual), r)
    assert np.array_equal(codes[0].cpu().numpy(), want)
    assert np.all(np.abs(f64(codes[1]) - scale) <= 2.0 ** -23 * scale)


class Steps:
    """A layer with its batch of sequences in shuffled pages."""

    def __init__(self, hq, hkv, d, page, dtype, batch=3, cols=6):
        self.hq, self.hkv, self.d, self.page, self.dtype = hq, hkv, d, page, dtype
        self.layer = DecoderLayer(torch.device(DEV), 128, batch * cols + 1, page, positions=cols * page, hidden=256,
                                  heads=hq, heads_kv=hkv, head_dim=d, ffn=512, dtype=dtype)
        c = self.layer.cache
        for t in (c.k, c.v):
            t.fill_(77)
        for t in (c.k_scale, c.v_scale):
            t.fill_(float("nan"))      # a page needs no clearing before its first token
        self.table = np.random.default_rng(4).permutation(batch * cols + 1)[:batch * cols].reshape(batch, cols)
        self.kv = np.zeros(batch, dtype=np.int64)

    def batch(self, new, max_q=None):
        self.kv = self.kv + new
        self.q_start = np.concatenate([[0], np.cumsum(new)])
        return q.KvBatch(i32(self.table), i32(self.q_start), i32(self.kv), max_q=max_q or int(max(new)),
                         max_kv=self.table.shape[1] * self.page)

    def inputs(self, m, tag):
        return [synth.normal_tensor(11, f"layer/{tag}/{n}/{m}", (m, 256), dtype=self.dtype).to(DEV) for n in "xr"]


def check_step(s, new, tag):
    L, dtype = s.layer, s.dtype
    m = int(np.sum(new))
    x, res = s.inputs(m, tag)
    before = res.clone()
    was = pull(L.cache)
    batch = s.batch(np.array(new))
    y = L.step(x, res, batch)
    torch.cuda.synchronize()
    cut = lambda c: (c[0][:m], c[1][:m])  # noqa: E731
    a, cq, b, hq = map(cut, (L.a, L.cq, L.b, L.hq))
    # residual after the second norm = r1 + yo: redo the first
    r1, _ = oracle.add_rmsnorm(f64(x), f64(before), L.gamma[0].cpu().numpy(), 1e-6, dtype)
    r1 = torch.from_numpy(r1).to(res.dtype)
    check_norm(a, r1, x, before, L.gamma[0], dtype)
    check_gemm(L.qkv[:m], a, L.w["qkv"], dtype)
    rope = L.rope.cpu().numpy()
    want = oracle.rope_append_kv(f64(L.qkv[:m]), was, s.table, s.q_start, s.kv, s.hq, rope, s.d, False)
    now = pull(L.cache)
    for name in ("k_scale", "v_scale", "k", "v"):
        assert np.array_equal(now[name], was[name], equal_nan=name.endswith("scale")), name
    check_q(L.qr[:m], want, L.qkv[:m], s.hq, s.d, dtype, np.arange(m))
    held = Cache.__new__(Cache)
    held.host, held.cache = now, L.cache
    check_attention(L.ctx[:m], L.qr[:m], held, s.table, s.q_start, s.kv, s.hq, s.d ** -0.5, 0.0, None, dtype)
    want_q, want_s = oracle.quantize_rows(f64(L.ctx[:m]), 8)[:2]
    assert np.max(np.abs(cq[0].cpu().numpy() - want_q)) <= 1
    assert np.allclose(f64(cq[1]), want_s, rtol=1e-6)
    check_gemm(L.yo[:m], cq, L.w["o"], dtype)
    check_norm(b, res, L.yo[:m], r1, L.gamma[1], dtype)
    check_gemm(L.gu[:m], b, L.w["gate_up"], dtype)
    gate, up = f64(L.gu[:m, :L.ffn]), f64(L.gu[:m, L.ffn:])
    want_q, want_s = oracle.quantize_rows(oracle.gelu(gate) * up, 8)[:2]
    assert np.max(np.abs(hq[0].cpu().numpy() - want_q)) <= 1
    assert np.allclose(f64(hq[1]), want_s, rtol=1e-5)
    check_gemm(y, hq, L.w["down"], dtype)


@pytest.mark.parametrize("hq,hkv,d,page,dtype", [(2, 2, 128, 16, "f16"), (4, 1, 64, 32, "bf16"), (1, 1, 256, 16, "bf16")])
def test_prompt_then_tokens(hq, hkv, d, page, dtype):
    s = Steps(hq, hkv, d, page, dtype)
    check_step(s, [70, 1, 17], "prompt")
    for t in range(3):
        check_step(s, [1, 1, 1], f"token{t}")
    check_step(s, [0, 9, 1], "mixed")


def test_captured_step():
    """One captured single-token step, replayed with the lengths moving on,
    against eager steps of a second layer from the same prompt."""
    a, b = Steps(4, 2, 64, 16, "f16"), Steps(4, 2, 64, 16, "f16")
    for s in (a, b):
        x, res = s.inputs(30, "prompt")
        s.layer.step(x, res, s.batch(np.array([10, 15, 5])))
    xa, ra = a.inputs(3, "g")
    batch = a.batch(np.array([1, 1, 1]))
    ws = q.kv_attention_workspace(a.layer.cache, batch, 4)
    a.layer.workspace(3)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ya = a.layer.step(xa, ra, batch, attn_workspace=ws)
    for t in range(4):
        xb, rb = b.inputs(3, f"replay{t}")
        xa.copy_(xb)
        ra.copy_(rb)
        yb = b.layer.step(xb, rb, b.batch(np.array([1, 1, 1])))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(ya, yb) and torch.equal(ra, rb)
        n = a.layer.cache
        for name in ("k", "v"):
            assert torch.equal(getattr(n, name), getattr(b.layer.cache, name))
        batch.kv_len.add_(1)


def test_norm_before_the_weight_only_gemv():
    """Residual + RMS norm in x's type, then qlin_gemv_w4a16."""
    m, k, n = 5, 1024, 512
    x, res = [synth.normal_tensor(12, f"gemv/{t}", (m, k), dtype="f16").to(DEV) for t in "xr"]
    gamma = torch.ones(k, device=DEV)
    w = synth.normal_tensor(12, "gemv/w", (n, k), std=0.03, dtype="f16").to(DEV)
    wq, ws = q.qlin_quantize_weights(w, bits=4, group=128)
    h, r = q.qlin_add_rmsnorm(x, gamma, res, residual_out=torch.empty_like(x))
    y = q.qlin_gemv_w4a16(h, wq, ws)
    torch.cuda.synchronize()
    want_r, want = oracle.add_rmsnorm(f64(x), f64(res), gamma.cpu().numpy(), 1e-6, "f16")
    assert np.array_equal(f64(r), want_r)
    assert np.all(np.abs(f64(h) - want) <= (2.0 ** -11 + 2.0 ** -22) * np.abs(want) + 2.0 ** -25)
    _, ref = oracle.gemv_w4a16(f64(h), oracle.unpack_int4(wq.cpu().numpy()), ws.cpu().numpy(), 128)
    assert oracle.compare_outputs(f64(y), ref).ok
