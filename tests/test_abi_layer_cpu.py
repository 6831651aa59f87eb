"""C-ABI checks, without a GPU, of the entry points between a layer's
projections (fake, never-dereferenced pointers: every call is refused, or is
empty, before any HIP call), and the same checks against the sanitizer build.
"""

import os
import subprocess
import sys

import pytest

import bit_ptq_vla_amd as q
from bit_ptq_vla_amd import build_host_sanitized as hs

HERE = os.path.dirname(os.path.abspath(__file__))

P = 0x10000000
P2 = 0x20000000
P3 = 0x40000000
P4 = 0x60000000
P5 = 0x70000000
W = 0x7F000000
BAD = 0x10000001


@pytest.fixture(scope="module")
def lib():
    return q.load()


# ---- qlin_add_rmsnorm_quant(x, dt, m, k, ldx, res, ldr, w, eps, b, bits, res_out, xq, xs, stream)

def norm_quant(lib, x=P, dt=0, m=4, k=512, ldx=512, res=P2, ldr=512, w=W, eps=1e-6, b=64, bits=8, ro=P3, xq=P4,
               xs=P5):
    return lib.qlin_add_rmsnorm_quant(x, dt, m, k, ldx, res, ldr, w, eps, b, bits, ro, xq, xs, None)


NORM_BAD = [
    (dict(x=None), q.QLIN_ERR_NULL), (dict(w=None), q.QLIN_ERR_NULL),
    (dict(dt=3), q.QLIN_ERR_DTYPE), (dict(dt=-1), q.QLIN_ERR_DTYPE),
    (dict(eps=-1.0), q.QLIN_ERR_UNSUPPORTED), (dict(eps=float("nan")), q.QLIN_ERR_UNSUPPORTED),
    (dict(eps=float("inf")), q.QLIN_ERR_UNSUPPORTED),
    (dict(m=-1), q.QLIN_ERR_SHAPE), (dict(m=1 << 31), q.QLIN_ERR_SHAPE), (dict(k=0), q.QLIN_ERR_SHAPE),
    (dict(k=516, ldx=520), q.QLIN_ERR_SHAPE), (dict(ldx=504), q.QLIN_ERR_SHAPE), (dict(ldx=516), q.QLIN_ERR_SHAPE),
    (dict(ldr=504), q.QLIN_ERR_SHAPE), (dict(res=None, ldr=504), q.QLIN_ERR_SHAPE),
    (dict(k=32776, ldx=32776, ldr=32776), q.QLIN_ERR_SHAPE),
    (dict(x=BAD), q.QLIN_ERR_ALIGN), (dict(res=BAD), q.QLIN_ERR_ALIGN), (dict(w=W + 4), q.QLIN_ERR_ALIGN),
    (dict(ro=P3 + 8), q.QLIN_ERR_ALIGN),
    (dict(ro=P + 16), q.QLIN_ERR_ALIAS),                      # shifted against x
    (dict(ro=P, ldr=520), q.QLIN_ERR_ALIAS),                  # x's place, another pitch
    (dict(ro=P2 + 1024), q.QLIN_ERR_ALIAS),                   # shifted against the residual
    (dict(ro=W - 64), q.QLIN_ERR_ALIAS),                      # over the weight
]


@pytest.mark.parametrize("kw,status", NORM_BAD + [
    (dict(xq=None), q.QLIN_ERR_NULL), (dict(xs=None), q.QLIN_ERR_NULL), (dict(xs=BAD), q.QLIN_ERR_ALIGN),
    (dict(bits=0), q.QLIN_ERR_UNSUPPORTED), (dict(bits=5), q.QLIN_ERR_UNSUPPORTED),
    (dict(b=48), q.QLIN_ERR_UNSUPPORTED), (dict(b=512), q.QLIN_ERR_UNSUPPORTED),
    (dict(k=520, ldx=520, ldr=520), q.QLIN_ERR_SHAPE),        # not a multiple of the block
    (dict(k=576, ldx=576, ldr=576, bits=6), q.QLIN_ERR_SHAPE),  # E2M3 takes k in multiples of 128
    (dict(xq=P + 512), q.QLIN_ERR_ALIAS), (dict(xq=P3 + 16), q.QLIN_ERR_ALIAS), (dict(xs=P4 + 16), q.QLIN_ERR_ALIAS),
])
def test_add_rmsnorm_quant_rejects(lib, kw, status):
    assert norm_quant(lib, **kw) == status


def norm(lib, x=P, dt=0, m=4, k=512, ldx=512, res=P2, ldr=512, w=W, eps=1e-6, ro=P3, y=P4):
    return lib.qlin_add_rmsnorm(x, dt, m, k, ldx, res, ldr, w, eps, ro, y, None)


@pytest.mark.parametrize("kw,status", NORM_BAD + [(dict(y=None), q.QLIN_ERR_NULL), (dict(y=P + 1024), q.QLIN_ERR_ALIAS)])
def test_add_rmsnorm_rejects(lib, kw, status):
    assert norm(lib, **kw) == status


def test_add_rmsnorm_empty_is_ok(lib):
    assert norm_quant(lib, m=0) == q.QLIN_OK
    assert norm_quant(lib, m=0, x=None, res=None, ro=None, ldr=0, xq=None, xs=None) == q.QLIN_OK
    assert norm_quant(lib, m=0, ro=P) == q.QLIN_OK and norm_quant(lib, m=0, ro=P2) == q.QLIN_OK    # in place
    assert norm(lib, m=0) == q.QLIN_OK


def test_more_threads_than_a_launch_holds_are_refused(lib):
    """2^32 threads: 32 to 1024 a row of the norm, 256 a (page, head) and one to
    16 values of q in the append, 512 a block of the attention."""
    big = 1 << 62                           # (any overlap of the fake spans comes later)
    for k, rows in ((64, 1 << 27), (4096, 1 << 23), (4104, 1 << 22), (32768, 1 << 22)):
        assert norm_quant(lib, m=rows, k=k, ldx=k, res=None, ro=None, b=0, x=big) == q.QLIN_ERR_SHAPE
        assert norm(lib, m=rows, k=k, ldx=k, res=None, ro=None, x=big) == q.QLIN_ERR_SHAPE
    wide = cache(heads=32, d=128)
    many = batch(n=1 << 16, max_q=8192, max_kv=64)
    assert append(lib, c=wide, b=many, hq=32, ld=96 * 128, ldq=32 * 128) == q.QLIN_ERR_SHAPE
    deep = batch(n=1 << 18, max_q=16, max_kv=64)
    assert attention(lib, c=wide, b=deep, hq=32, ldq=32 * 128, ldo=32 * 128) == q.QLIN_ERR_SHAPE
    assert lib.qlin_kv_attention_workspace_bytes(32, *refs(wide, deep)) == -1
    huge = batch(n=(1 << 31) - 1, max_q=1 << 20, max_kv=64)
    assert attention(lib, c=wide, b=huge, hq=32, ldq=32 * 128, ldo=32 * 128) == q.QLIN_ERR_SHAPE
    assert append(lib, c=wide, b=huge, hq=32, ld=96 * 128, ldq=32 * 128) == q.QLIN_ERR_SHAPE
    assert lib.qlin_rope_table(R, (1 << 31) - 1, 128, 1e4, 1.0, None) == q.QLIN_ERR_SHAPE


@pytest.mark.parametrize("cap", [-0.5, 1e-7, 4097.0, 1e30, float("inf"), float("nan")])
def test_caps_out_of_range_are_refused(lib, cap):
    assert attention(lib, cap=cap) == q.QLIN_ERR_UNSUPPORTED


def test_batch_bounds_are_32_bit():
    i32 = q.torch.zeros(2, dtype=q.torch.int32)
    for bad in (dict(max_q=1 << 32, max_kv=1), dict(max_q=1, max_kv=(1 << 32) + 1), dict(max_q=-1, max_kv=1)):
        with pytest.raises(ValueError, match="2\\^31"):
            q.KvBatch(i32.reshape(1, 2), i32, i32[:1], **bad)


# ---- paged cache descriptors

I1, I2, I3, I4, R = 0x91000000, 0x92000000, 0x93000000, 0x94000000, 0x95000000   # index arrays, the rope table
C1, C2, C3, C4 = 0x100000000, 0x200000000, 0x300000000, 0x300100000              # k, v, k_scale, v_scale


def cache(k=C1, v=C2, ks=C3, vs=C4, pages=64, page=16, heads=2, d=64):
    return q._KvCacheC(k, v, ks, vs, pages, page, heads, d)


def batch(table=I1, ld=4, q_start=I2, kv_len=I3, prefix=None, n=3, max_q=7, max_kv=64):
    return q._KvBatchC(table, ld, q_start, kv_len, prefix, n, max_q, max_kv)


def refs(c, b):
    return [None if x is None else q.ctypes.addressof(x) for x in (c, b)]


KV_BAD = [
    (dict(c=None), q.QLIN_ERR_NULL), (dict(b=None), q.QLIN_ERR_NULL),
    (dict(c=cache(k=None)), q.QLIN_ERR_NULL), (dict(c=cache(vs=None)), q.QLIN_ERR_NULL),
    (dict(b=batch(table=None)), q.QLIN_ERR_NULL), (dict(b=batch(q_start=None)), q.QLIN_ERR_NULL),
    (dict(b=batch(kv_len=None)), q.QLIN_ERR_NULL),
    (dict(c=cache(page=8)), q.QLIN_ERR_UNSUPPORTED), (dict(c=cache(page=48)), q.QLIN_ERR_UNSUPPORTED),
    (dict(c=cache(d=96)), q.QLIN_ERR_UNSUPPORTED),
    (dict(c=cache(pages=0)), q.QLIN_ERR_SHAPE), (dict(c=cache(heads=0)), q.QLIN_ERR_SHAPE),
    (dict(hq=0), q.QLIN_ERR_SHAPE), (dict(hq=5), q.QLIN_ERR_SHAPE), (dict(tokens=-1), q.QLIN_ERR_SHAPE),
    (dict(b=batch(n=-1)), q.QLIN_ERR_SHAPE), (dict(b=batch(max_q=-1)), q.QLIN_ERR_SHAPE),
    (dict(b=batch(max_kv=-1)), q.QLIN_ERR_SHAPE), (dict(b=batch(ld=3)), q.QLIN_ERR_SHAPE),
    (dict(b=batch(max_kv=65)), q.QLIN_ERR_SHAPE),
    (dict(b=batch(max_kv=(1 << 30) + 1, ld=1 << 30)), q.QLIN_ERR_SHAPE),
    (dict(b=batch(max_q=1 << 30)), q.QLIN_ERR_SHAPE),                  # x 2 query heads of a kv head
    (dict(c=cache(k=C1 + 8)), q.QLIN_ERR_ALIGN), (dict(c=cache(vs=C4 + 4)), q.QLIN_ERR_ALIGN),
    (dict(b=batch(kv_len=I3 + 2)), q.QLIN_ERR_ALIGN), (dict(b=batch(prefix=I4 + 1)), q.QLIN_ERR_ALIGN),
    (dict(dt=2), q.QLIN_ERR_DTYPE), (dict(dt=3), q.QLIN_ERR_DTYPE), (dict(dt=-1), q.QLIN_ERR_DTYPE),
]


def append(lib, qkv=P, dt=1, tokens=20, ld=8 * 64, hq=4, rope=R, rope_len=64, rot=64, inter=0, pos=None, c=cache(),
           b=batch(), out=P2, ldq=4 * 64):
    return lib.qlin_rope_append_kv(qkv, dt, tokens, ld, hq, rope, rope_len, rot, inter, pos, *refs(c, b), out, ldq, None)


@pytest.mark.parametrize("kw,status", KV_BAD + [
    (dict(qkv=None), q.QLIN_ERR_NULL), (dict(out=None), q.QLIN_ERR_NULL), (dict(rope=None), q.QLIN_ERR_NULL),
    (dict(inter=2), q.QLIN_ERR_UNSUPPORTED),
    (dict(rot=-16), q.QLIN_ERR_SHAPE), (dict(rot=24), q.QLIN_ERR_SHAPE), (dict(rot=80), q.QLIN_ERR_SHAPE),
    (dict(rope_len=0), q.QLIN_ERR_SHAPE), (dict(ld=504), q.QLIN_ERR_SHAPE), (dict(ld=516), q.QLIN_ERR_SHAPE),
    (dict(ldq=248), q.QLIN_ERR_SHAPE), (dict(ldq=260), q.QLIN_ERR_SHAPE),
    (dict(b=batch(n=1 << 30, max_q=1000)), q.QLIN_ERR_SHAPE),          # more blocks than a launch holds
    (dict(qkv=P + 2), q.QLIN_ERR_ALIGN), (dict(out=P2 + 4), q.QLIN_ERR_ALIGN), (dict(rope=R + 4), q.QLIN_ERR_ALIGN),
    (dict(pos=I4 + 2), q.QLIN_ERR_ALIGN),
    (dict(out=P), q.QLIN_ERR_ALIAS), (dict(out=C1 + 4096), q.QLIN_ERR_ALIAS), (dict(pos=P2 + 64), q.QLIN_ERR_ALIAS),
    (dict(c=cache(v=C1 + 64)), q.QLIN_ERR_ALIAS), (dict(c=cache(ks=C1)), q.QLIN_ERR_ALIAS),
    (dict(b=batch(kv_len=C3)), q.QLIN_ERR_ALIAS), (dict(b=batch(table=C2 + 1024)), q.QLIN_ERR_ALIAS),
])
def test_rope_append_rejects(lib, kw, status):
    assert append(lib, **kw) == status


def test_rope_append_empty_is_ok(lib):
    assert append(lib, tokens=0, qkv=None, out=None) == q.QLIN_OK
    assert append(lib, b=batch(n=0, table=None, q_start=None, kv_len=None)) == q.QLIN_OK
    assert append(lib, b=batch(max_q=0)) == q.QLIN_OK
    assert append(lib, tokens=0, rot=0, rope=None, rope_len=0) == q.QLIN_OK


def attention(lib, x=P, dt=1, tokens=20, ldq=4 * 64, hq=4, c=cache(), b=batch(), scale=0.125, cap=0.0, out=P2,
              ldo=4 * 64, ws=None, wsb=0):
    return lib.qlin_kv_attention(x, dt, tokens, ldq, hq, *refs(c, b), scale, cap, out, ldo, ws, wsb, None)


LONG = dict(ld=64, max_kv=1024, max_q=1)      # few rows over many keys: takes a split


@pytest.mark.parametrize("kw,status", KV_BAD + [
    (dict(x=None), q.QLIN_ERR_NULL), (dict(out=None), q.QLIN_ERR_NULL), (dict(wsb=64), q.QLIN_ERR_NULL),
    (dict(scale=float("nan")), q.QLIN_ERR_UNSUPPORTED), (dict(scale=float("inf")), q.QLIN_ERR_UNSUPPORTED),
    (dict(cap=-1.0), q.QLIN_ERR_UNSUPPORTED), (dict(cap=float("nan")), q.QLIN_ERR_UNSUPPORTED),
    (dict(ldq=248), q.QLIN_ERR_SHAPE), (dict(ldq=260), q.QLIN_ERR_SHAPE), (dict(ldo=250), q.QLIN_ERR_SHAPE),
    (dict(ws=P4, wsb=-16), q.QLIN_ERR_SHAPE),
    (dict(x=P + 2), q.QLIN_ERR_ALIGN), (dict(out=P2 + 4), q.QLIN_ERR_ALIGN), (dict(ws=P4 + 8, wsb=64), q.QLIN_ERR_ALIGN),
    (dict(b=batch(**LONG), ws=P4, wsb=1024), q.QLIN_ERR_WORKSPACE),
    (dict(out=P), q.QLIN_ERR_ALIAS), (dict(out=C1 + 4096), q.QLIN_ERR_ALIAS), (dict(out=C3), q.QLIN_ERR_ALIAS),
    (dict(b=batch(**LONG), ws=C2, wsb=1 << 24), q.QLIN_ERR_ALIAS),
    (dict(b=batch(**LONG), ws=P2 - 4096, wsb=1 << 24), q.QLIN_ERR_ALIAS),     # over out
    (dict(b=batch(prefix=P2 + 64)), q.QLIN_ERR_ALIAS),
])
def test_kv_attention_rejects(lib, kw, status):
    assert attention(lib, **kw) == status


def test_kv_attention_empty_is_ok_and_workspace_bytes(lib):
    assert attention(lib, tokens=0, x=None, out=None) == q.QLIN_OK
    assert attention(lib, b=batch(n=0, table=None, q_start=None, kv_len=None)) == q.QLIN_OK
    assert attention(lib, b=batch(max_q=0)) == q.QLIN_OK
    def need(hq, c, b):
        return lib.qlin_kv_attention_workspace_bytes(hq, *refs(c, b))

    assert need(4, cache(), batch(**LONG)) > 0 and need(4, cache(), batch(**LONG)) % 16 == 0
    assert need(4, cache(), batch(max_kv=0)) == 0
    assert need(5, cache(), batch()) == -1
    assert need(4, None, None) == -1


@pytest.mark.parametrize("args,status", [
    ((None, 8, 16, 1e4, 1.0), q.QLIN_ERR_NULL), ((R, -1, 16, 1e4, 1.0), q.QLIN_ERR_SHAPE),
    ((R, 8, 15, 1e4, 1.0), q.QLIN_ERR_SHAPE), ((R, 8, 0, 1e4, 1.0), q.QLIN_ERR_SHAPE),
    ((R, 8, 16, 0.0, 1.0), q.QLIN_ERR_UNSUPPORTED), ((R, 8, 16, 1e4, float("nan")), q.QLIN_ERR_UNSUPPORTED),
    ((R, 8, 16, float("inf"), 1.0), q.QLIN_ERR_UNSUPPORTED), ((R, 8, 16, 1e4, -1.0), q.QLIN_ERR_UNSUPPORTED),
    ((R + 8, 8, 16, 1e4, 1.0), q.QLIN_ERR_ALIGN), ((R, 0, 16, 1e4, 1.0), q.QLIN_OK),
])
def test_rope_table_checks(lib, args, status):
    assert lib.qlin_rope_table(*args, None) == status


# ---- the index arithmetic of the kernels, on the host

INDEX_CHECK = r"""
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>
#include "kv_index.h"
using namespace qlin;
static void need(bool ok, const char* what) { if (!ok) { std::printf("broken: %s\n", what); std::exit(1); } }
int main() {
    std::mt19937 r(11);
    auto any = [&](int lo, int hi) { return lo + static_cast<int>(r() % static_cast<unsigned>(hi - lo + 1)); };
    for (int it = 0; it < 20000; ++it) {
        KvIndex x{};
        const bool damaged = it & 1;
        x.page_size = 16 << any(0, 2);
        x.batch = any(1, 5);
        x.max_q = any(0, 90);
        x.max_kv = any(0, 300);
        const int cols = (x.max_kv + x.page_size - 1) / x.page_size;
        x.table_ld = cols + any(0, 2);
        x.pages = any(1, 40);
        // exactly what the kernels may read: an index past it is an error under the sanitizer
        std::vector<int32_t> table((x.batch - 1) * x.table_ld + cols), start(x.batch + 1), kv(x.batch), pre(x.batch);
        int at = 0;
        for (int b = 0; b <= x.batch; ++b) {
            start[b] = at;
            if (b < x.batch) { const int n = any(0, x.max_q < x.max_kv ? x.max_q : x.max_kv); at += n; kv[b] = any(n, x.max_kv); }
        }
        x.tokens = at + any(0, 3);
        for (auto& p : table) p = any(0, static_cast<int>(x.pages) - 1);
        for (auto& p : pre) p = any(-3, x.max_kv + 3);
        if (damaged) {
            const int32_t bad[] = {-1, INT32_MIN, INT32_MAX, 1 << 20, -77};
            for (auto* v : {&table, &start, &kv, &pre})
                for (auto& e : *v) if (any(0, 3) == 0) e = bad[any(0, 4)];
        }
        x.page_table = table.data(); x.q_start = start.data(); x.kv_len = kv.data();
        x.prefix_len = any(0, 1) ? pre.data() : nullptr;
        const int touched = kv_max_touched(x.max_q, x.page_size);
        for (int b = 0; b < x.batch; ++b) {
            const KvSeq s = kv_seq(x, b);
            need(s.n >= 0 && s.n <= x.max_q && s.kv >= 0 && s.kv <= x.max_kv, "lengths");
            need(s.row0 >= 0 && s.row0 + s.n <= x.tokens, "rows");
            int covered = 0;
            for (int i = 0; i < touched + 2; ++i) {
                const KvSpan p = kv_touched(x, s, i);
                if (p.hi <= p.lo || s.n == 0) continue;
                need(i < touched, "pages touched past the grid");
                need(p.idx >= 0 && p.idx < cols, "page column");
                need(p.lo / x.page_size == p.idx && (p.hi - 1) / x.page_size == p.idx, "span in its page");
                for (int j = p.lo; j < p.hi; ++j) need(j >= s.first && j - s.first < s.n, "token of a position");
                const int page = kv_page(x, b, p.idx);
                need(page == kNoPage || (page >= 0 && page < x.pages), "page");
                covered += p.hi - p.lo;
            }
            need(covered == (s.n == 0 ? 0 : s.kv - (s.first < 0 ? 0 : s.first)), "every new token once");
            for (int i = 0; i < s.n; ++i) {
                const int v = kv_visible(x, s, b, s.first + i);
                need(v >= 0 && v <= s.kv, "visible keys");
                if (!damaged && !x.prefix_len) need(v == s.first + i + 1, "causal");
            }
        }
    }
    std::printf("index arithmetic holds\n");
}
"""


def test_index_arithmetic_stays_in_bounds(tmp_path):
    """Token ranges, page columns and page numbers over random and damaged
    metadata, under the host sanitizers."""
    src, exe = tmp_path / "index.cpp", tmp_path / "index"
    src.write_text(INDEX_CHECK)
    r = subprocess.run([hs.compiler(), "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined",
                        "-fno-sanitize-recover=undefined", "-D_GLIBCXX_ASSERTIONS", f"-I{hs.CSRC}", str(src), "-o", str(exe)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    env = {k: v for k, v in os.environ.items() if k != "LD_PRELOAD"}
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300, env=env)
    assert r.returncode == 0 and "holds" in r.stdout, (r.stdout + r.stderr)[-3000:]


# ---- the same calls under AddressSanitizer and UndefinedBehaviorSanitizer

@pytest.mark.skipif("QLIN_LIB_PATH" in os.environ, reason="already the sanitizer build")
def test_layer_validation_under_asan_and_ubsan(tmp_path):
    try:
        asan = hs.runtime("libasan.so")
        lib = hs.build(str(tmp_path / "libqlin_host_sanitized.so"))
    except RuntimeError as e:
        pytest.skip(f"no host sanitizer toolchain: {e}")
    env = dict(os.environ)
    env.update({
        "QLIN_LIB_PATH": lib,
        "LD_PRELOAD": asan,
        "ASAN_OPTIONS": "detect_leaks=0:halt_on_error=1:abort_on_error=1:alloc_dealloc_mismatch=0"
                        ":detect_odr_violation=0",
        "UBSAN_OPTIONS": "halt_on_error=1:print_stacktrace=1",
    })
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", os.path.abspath(__file__)],
                       env=env, capture_output=True, text=True, timeout=600)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-4000:]
    assert " passed" in r.stdout and "ERROR: AddressSanitizer" not in out and "runtime error:" not in out
