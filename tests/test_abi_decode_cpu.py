"""C-ABI checks, without a GPU, of trees, sampling and pages (fake,
never-dereferenced pointers: every call is refused, or is empty, before any HIP
call), the same against the sanitizer build, and what masks give a lane of the
attention kernels, on the host.
"""

import os
import subprocess
import sys

import pytest
import torch

import bit_ptq_vla_amd as q
from bit_ptq_vla_amd import build_host_sanitized as hs
from test_abi_layer_cpu import BAD, C1, C2, C3, C4, I1, I2, I3, I4, P, P2, P3, P4, batch, cache, refs

T1, T2, T3 = 0xA1000000, 0xA2000000, 0xA3000000


@pytest.fixture(scope="module")
def lib():
    return q.load()


def ref(x):
    return None if x is None else q.ctypes.addressof(x)


LENGTHS_BAD = [
    (dict(b=None), q.QLIN_ERR_NULL), (dict(b=batch(q_start=None)), q.QLIN_ERR_NULL),
    (dict(b=batch(kv_len=None)), q.QLIN_ERR_NULL), (dict(tokens=-1), q.QLIN_ERR_SHAPE),
    (dict(tokens=1 << 31), q.QLIN_ERR_SHAPE), (dict(b=batch(n=-1)), q.QLIN_ERR_SHAPE),
    (dict(b=batch(max_q=-1)), q.QLIN_ERR_SHAPE), (dict(b=batch(max_q=1025)), q.QLIN_ERR_SHAPE),
    (dict(b=batch(max_kv=-1)), q.QLIN_ERR_SHAPE), (dict(b=batch(n=(1 << 23) + 1)), q.QLIN_ERR_SHAPE),
    (dict(b=batch(q_start=I2 + 2)), q.QLIN_ERR_ALIGN), (dict(b=batch(kv_len=I3 + 1)), q.QLIN_ERR_ALIGN),
]


def plan(lib, parents=T1, tokens=20, b=batch(), mask=P, ld=1, pos=P2):
    return lib.qlin_tree_plan(parents, tokens, ref(b), mask, ld, pos, None)


@pytest.mark.parametrize("kw,status", LENGTHS_BAD + [
    (dict(parents=None), q.QLIN_ERR_NULL), (dict(mask=None), q.QLIN_ERR_NULL), (dict(pos=None), q.QLIN_ERR_NULL),
    (dict(ld=0), q.QLIN_ERR_SHAPE), (dict(b=batch(max_q=33)), q.QLIN_ERR_SHAPE), (dict(ld=1 << 31), q.QLIN_ERR_SHAPE),
    (dict(parents=T1 + 2), q.QLIN_ERR_ALIGN), (dict(mask=P + 1), q.QLIN_ERR_ALIGN), (dict(pos=P2 + 2), q.QLIN_ERR_ALIGN),
    (dict(mask=T1 + 8), q.QLIN_ERR_ALIAS), (dict(pos=T1), q.QLIN_ERR_ALIAS), (dict(pos=P + 16), q.QLIN_ERR_ALIAS),
    (dict(mask=I3), q.QLIN_ERR_ALIAS), (dict(pos=I2 + 8), q.QLIN_ERR_ALIAS),
])
def test_plan_rejects(lib, kw, status):
    assert plan(lib, **kw) == status


def accept(lib, parents=T1, draft=T2, sampled=T3, tokens=20, b=batch(), path=P, ld=7, count=P2, token=P3):
    return lib.qlin_tree_accept(parents, draft, sampled, tokens, ref(b), path, ld, count, token, None)


@pytest.mark.parametrize("kw,status", LENGTHS_BAD + [
    (dict(parents=None), q.QLIN_ERR_NULL), (dict(draft=None), q.QLIN_ERR_NULL), (dict(sampled=None), q.QLIN_ERR_NULL),
    (dict(path=None), q.QLIN_ERR_NULL), (dict(count=None), q.QLIN_ERR_NULL), (dict(token=None), q.QLIN_ERR_NULL),
    (dict(ld=6), q.QLIN_ERR_SHAPE), (dict(draft=T2 + 1), q.QLIN_ERR_ALIGN), (dict(token=P3 + 2), q.QLIN_ERR_ALIGN),
    (dict(path=T2), q.QLIN_ERR_ALIAS), (dict(count=T3 + 4), q.QLIN_ERR_ALIAS), (dict(token=P2), q.QLIN_ERR_ALIAS),
    (dict(count=P + 40), q.QLIN_ERR_ALIAS),
])
def test_accept_rejects(lib, kw, status):
    assert accept(lib, **kw) == status


def tree(lib, x=P, dt=1, tokens=20, ldq=256, hq=4, c=cache(), b=batch(), mask=T1, ldm=1, scale=0.125, cap=0.0, out=P2,
         ldo=256, ws=None, wsb=0):
    return lib.qlin_kv_attention_tree(x, dt, tokens, ldq, hq, *refs(c, b), mask, ldm, scale, cap, out, ldo, ws, wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(mask=None), q.QLIN_ERR_NULL), (dict(b=None), q.QLIN_ERR_NULL), (dict(c=None), q.QLIN_ERR_NULL),
    (dict(x=None), q.QLIN_ERR_NULL), (dict(b=batch(prefix=I4)), q.QLIN_ERR_UNSUPPORTED),
    (dict(b=batch(max_q=1025)), q.QLIN_ERR_SHAPE), (dict(ldm=0), q.QLIN_ERR_SHAPE), (dict(b=batch(max_q=33)), q.QLIN_ERR_SHAPE),
    (dict(mask=T1 + 2), q.QLIN_ERR_ALIGN), (dict(out=T1), q.QLIN_ERR_ALIAS), (dict(out=C3), q.QLIN_ERR_ALIAS),
    (dict(dt=2), q.QLIN_ERR_DTYPE), (dict(hq=5), q.QLIN_ERR_SHAPE), (dict(cap=-1.0), q.QLIN_ERR_UNSUPPORTED),
    (dict(b=batch(ld=64, max_kv=1024, max_q=1), ws=T1 - 64, wsb=1 << 24), q.QLIN_ERR_ALIAS),
    (dict(b=batch(ld=64, max_kv=1024, max_q=1), ws=P4, wsb=1024), q.QLIN_ERR_WORKSPACE),
])
def test_tree_attention_rejects(lib, kw, status):
    assert tree(lib, **kw) == status


def sample(lib, x=P, dt=0, rows=4, vocab=1000, ld=1000, u=T1, t=T2, k=None, p=T3, m=None, token=P2, lp=P3, ws=None, wsb=0):
    return lib.qlin_sample(x, dt, rows, vocab, ld, u, t, k, p, m, token, lp, ws, wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), q.QLIN_ERR_NULL), (dict(u=None), q.QLIN_ERR_NULL), (dict(token=None), q.QLIN_ERR_NULL),
    (dict(wsb=64), q.QLIN_ERR_NULL), (dict(dt=3), q.QLIN_ERR_DTYPE), (dict(dt=-1), q.QLIN_ERR_DTYPE),
    (dict(rows=-1), q.QLIN_ERR_SHAPE), (dict(rows=(1 << 21) + 1), q.QLIN_ERR_SHAPE), (dict(vocab=0), q.QLIN_ERR_SHAPE),
    (dict(vocab=(1 << 18) + 1, ld=1 << 19), q.QLIN_ERR_SHAPE), (dict(ld=992), q.QLIN_ERR_SHAPE),
    (dict(ld=1004), q.QLIN_ERR_SHAPE), (dict(dt=2, ld=1002), q.QLIN_ERR_SHAPE), (dict(ld=1 << 31), q.QLIN_ERR_SHAPE),
    (dict(ws=P4, wsb=-1), q.QLIN_ERR_SHAPE),
    (dict(x=BAD), q.QLIN_ERR_ALIGN), (dict(u=T1 + 2), q.QLIN_ERR_ALIGN), (dict(k=T2 + 1), q.QLIN_ERR_ALIGN),
    (dict(token=P2 + 2), q.QLIN_ERR_ALIGN), (dict(ws=P4 + 8, wsb=1 << 24), q.QLIN_ERR_ALIGN),
    (dict(token=P + 64), q.QLIN_ERR_ALIAS), (dict(lp=T1 + 4), q.QLIN_ERR_ALIAS), (dict(lp=P2 + 8), q.QLIN_ERR_ALIAS),
    (dict(ws=P - 16, wsb=1 << 24), q.QLIN_ERR_ALIAS), (dict(m=P2), q.QLIN_ERR_ALIAS),
])
def test_sample_rejects(lib, kw, status):
    assert sample(lib, **kw) == status


def test_empty_calls_are_ok(lib):
    assert plan(lib, tokens=0, parents=None, mask=None, pos=None) == q.QLIN_OK
    assert plan(lib, b=batch(n=0, q_start=None, kv_len=None)) == q.QLIN_OK
    assert accept(lib, b=batch(n=0, q_start=None, kv_len=None), path=None, count=None, token=None) == q.QLIN_OK
    assert tree(lib, tokens=0, x=None, out=None) == q.QLIN_OK
    assert sample(lib, rows=0, x=None, u=None, token=None) == q.QLIN_OK
    assert resize(lib, rows=0, table=None, old=None, new=None, out=None, moved=None) == q.QLIN_OK
    assert fork(lib, n=0, src=None, dst=None, length=None) == q.QLIN_OK
    assert copies(lib, n=0, pairs=None) == q.QLIN_OK
    assert compact(lib, b=batch(n=0, table=None, q_start=None, kv_len=None), path=None, count=None) == q.QLIN_OK


def test_workspace_sizes(lib):
    assert lib.qlin_sample_workspace_bytes(-1, 10) == -1 and lib.qlin_sample_workspace_bytes(1, 0) == -1
    assert lib.qlin_sample_workspace_bytes(1, (1 << 18) + 1) == -1
    assert lib.qlin_sample_workspace_bytes((1 << 21) + 1, 1) == -1
    for rows in (0, 1, 7, 64, 1024, 1 << 21):
        for vocab in (1, 1000, 32000, 1 << 18):
            n = lib.qlin_sample_workspace_bytes(rows, vocab)
            assert n >= 0 and n % 16 == 0 and n < 1 << 30
    need = lib.qlin_kv_attention_tree_workspace_bytes
    long = batch(ld=64, max_kv=1024, max_q=1)
    assert need(4, *refs(cache(), long)) > 0
    assert need(4, *refs(cache(), batch(prefix=I4))) == -1 and need(4, None, None) == -1
    assert need(4, *refs(cache(), batch(max_q=1025))) == -1


# ---- pages

def pool(r=T1, f=T2, pages=64):
    return q._KvPoolC(r, f, pages)


POOL_BAD = [
    (dict(p=None), q.QLIN_ERR_NULL), (dict(p=pool(r=None)), q.QLIN_ERR_NULL), (dict(p=pool(f=None)), q.QLIN_ERR_NULL),
    (dict(p=pool(pages=0)), q.QLIN_ERR_SHAPE), (dict(p=pool(pages=1 << 31)), q.QLIN_ERR_SHAPE),
    (dict(p=pool(r=T1 + 4)), q.QLIN_ERR_ALIGN), (dict(p=pool(f=T2 + 8)), q.QLIN_ERR_ALIGN),
    (dict(table=None), q.QLIN_ERR_NULL), (dict(page=8), q.QLIN_ERR_UNSUPPORTED), (dict(rows=-1), q.QLIN_ERR_SHAPE),
    (dict(cols=-1), q.QLIN_ERR_SHAPE), (dict(ld=3), q.QLIN_ERR_SHAPE), (dict(cols=(1 << 24) + 1, ld=1 << 25), q.QLIN_ERR_SHAPE),
    (dict(table=P + 2), q.QLIN_ERR_ALIGN),
]


@pytest.mark.parametrize("kw,status", [(k, s) for k, s in POOL_BAD if "p" in k] + [(dict(p=pool(f=T1 + 16)), q.QLIN_ERR_ALIAS)])
def test_pool_init_rejects(lib, kw, status):
    assert lib.qlin_kv_pool_init(ref(kw["p"]), None) == status


def stack(*caches):
    return (q._KvCacheC * len(caches))(*caches)


ONE = cache()
TWO = cache(k=C1 + (1 << 28), v=C2 + (1 << 28), ks=C3 + (1 << 28), vs=C4 + (1 << 28))
STACK_BAD = [
    (dict(c=stack(ONE, cache(k=None))), q.QLIN_ERR_NULL), (dict(c=stack(ONE, cache(d=128))), q.QLIN_ERR_SHAPE),
    (dict(c=stack(ONE, cache(pages=65))), q.QLIN_ERR_SHAPE), (dict(c=stack(cache(page=8))), q.QLIN_ERR_UNSUPPORTED),
    (dict(c=stack(cache(heads=0))), q.QLIN_ERR_SHAPE), (dict(c=stack(cache(v=C2 + 4))), q.QLIN_ERR_ALIGN),
    (dict(c=stack(ONE, TWO, ONE)), q.QLIN_ERR_ALIAS),
]


def resize(lib, p=pool(), c=stack(ONE, TWO), layers=None, page=16, table=P, ld=4, cols=4, rows=3, old=I1, new=I2, out=I3, moved=I4):
    return lib.qlin_kv_resize(ref(p), ref(c), (0 if c is None else len(c)) if layers is None else layers, page, table, ld, cols,
                              rows, old, new, out, moved, None)


@pytest.mark.parametrize("kw,status", POOL_BAD + STACK_BAD + [
    (dict(layers=-1), q.QLIN_ERR_SHAPE), (dict(c=None, layers=2), q.QLIN_ERR_NULL), (dict(rows=1025), q.QLIN_ERR_SHAPE),
    (dict(page=32), q.QLIN_ERR_SHAPE), (dict(p=pool(pages=63)), q.QLIN_ERR_SHAPE),
    (dict(old=None), q.QLIN_ERR_NULL), (dict(new=None), q.QLIN_ERR_NULL), (dict(out=None), q.QLIN_ERR_NULL),
    (dict(moved=None), q.QLIN_ERR_NULL), (dict(moved=I4 + 2), q.QLIN_ERR_ALIGN),
    (dict(out=I1), q.QLIN_ERR_ALIAS), (dict(out=I4 + 16), q.QLIN_ERR_ALIAS), (dict(moved=P + 16), q.QLIN_ERR_ALIAS),
    (dict(table=T1 + 16), q.QLIN_ERR_ALIAS), (dict(old=T2), q.QLIN_ERR_ALIAS), (dict(new=C1 + 64), q.QLIN_ERR_ALIAS),
    (dict(table=C2 + (1 << 28)), q.QLIN_ERR_ALIAS),
])
def test_resize_rejects(lib, kw, status):
    assert resize(lib, **kw) == status


def fork(lib, p=pool(), page=16, table=P, ld=4, cols=4, rows=3, src=I1, dst=I2, length=I3, n=2):
    return lib.qlin_kv_fork(ref(p), page, table, ld, cols, rows, src, dst, length, n, None)


@pytest.mark.parametrize("kw,status", POOL_BAD + [
    (dict(n=-1), q.QLIN_ERR_SHAPE), (dict(n=(1 << 20) + 1), q.QLIN_ERR_SHAPE), (dict(src=None), q.QLIN_ERR_NULL),
    (dict(length=None), q.QLIN_ERR_NULL), (dict(dst=I2 + 1), q.QLIN_ERR_ALIGN), (dict(dst=P + 4), q.QLIN_ERR_ALIAS),
    (dict(src=T1), q.QLIN_ERR_ALIAS),
])
def test_fork_rejects(lib, kw, status):
    assert fork(lib, **kw) == status


def copies(lib, c=stack(ONE, TWO), pairs=I1, n=3):
    return lib.qlin_kv_copy_pages(ref(c), 0 if c is None else len(c), pairs, n, None)


@pytest.mark.parametrize("kw,status", STACK_BAD + [
    (dict(c=None), q.QLIN_ERR_NULL), (dict(pairs=None), q.QLIN_ERR_NULL), (dict(n=-1), q.QLIN_ERR_SHAPE),
    (dict(n=(1 << 24) + 1), q.QLIN_ERR_SHAPE), (dict(pairs=I1 + 2), q.QLIN_ERR_ALIGN), (dict(pairs=C4), q.QLIN_ERR_ALIAS),
])
def test_copy_pages_rejects(lib, kw, status):
    assert copies(lib, **kw) == status


def compact(lib, c=stack(ONE, TWO), b=batch(), path=P, ld=7, count=P2, out=P3):
    return lib.qlin_kv_compact(ref(c), 0 if c is None else len(c), ref(b), path, ld, count, out, None)


@pytest.mark.parametrize("kw,status", STACK_BAD + [
    (dict(c=None), q.QLIN_ERR_NULL), (dict(b=None), q.QLIN_ERR_NULL), (dict(path=None), q.QLIN_ERR_NULL),
    (dict(count=None), q.QLIN_ERR_NULL), (dict(ld=6), q.QLIN_ERR_SHAPE), (dict(b=batch(max_q=1025), ld=1025), q.QLIN_ERR_SHAPE),
    (dict(b=batch(ld=3)), q.QLIN_ERR_SHAPE), (dict(b=batch(n=1 << 22), c=stack(ONE)), q.QLIN_ERR_SHAPE),
    (dict(path=P + 2), q.QLIN_ERR_ALIGN), (dict(out=P3 + 1), q.QLIN_ERR_ALIGN), (dict(out=P2), q.QLIN_ERR_ALIAS),
    (dict(out=I3), q.QLIN_ERR_ALIAS), (dict(path=C1), q.QLIN_ERR_ALIAS), (dict(out=C3 + (1 << 28)), q.QLIN_ERR_ALIAS),
    (dict(b=batch(table=C2)), q.QLIN_ERR_ALIAS),
])
def test_compact_rejects(lib, kw, status):
    assert compact(lib, **kw) == status


# ---- the binding

def test_binding_refuses_host_tensors_and_wrong_shapes():
    i32 = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="device tensor"):
        q.KvPool(i32, i32[:1])
    with pytest.raises(ValueError, match="device tensor"):
        q.qlin_sample(torch.zeros((2, 8)), torch.zeros(2))
    with pytest.raises(ValueError, match="row-major"):
        q.qlin_sample(torch.zeros((8, 2)).t(), torch.zeros(2))
    with pytest.raises(ValueError, match="at least"):
        q.KvStack([])
    with pytest.raises(ValueError, match="contiguous int32"):
        q._index(i32[::2], "x", 2, i32.device)
    with pytest.raises(ValueError, match="row-major int32"):
        q._index_rows(torch.zeros((3, 2), dtype=torch.int32), "x", 3, 4, i32.device)


# ---- the bits a lane of the attention kernels sees, on the host

BITS_CHECK = r"""
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>
#include "kv_index.h"
using namespace qlin;
int main() {
    std::mt19937 r(5);
    for (int it = 0; it < 40000; ++it) {
        KvSeq s{0, static_cast<int32_t>(r() % 140), 0, static_cast<int32_t>(r() % 120) - 20};
        s.kv = s.first + s.n;
        // exactly the words that hold the nodes: a read past them is an error under the sanitizer
        std::vector<uint32_t> row((s.n + 31) / 32);
        for (auto& w : row) w = r();
        for (int j0 = 0; j0 < 300; j0 += 8) {
            const uint32_t bits = kv_tree_bits(row.data(), s, j0);
            for (int i = 0; i < 32; ++i) {
                const int j = j0 + i, node = j - s.first;
                const bool want = j < s.first || (node >= 0 && node < s.n && (row[node / 32] >> (node % 32) & 1));
                if (want != static_cast<bool>(bits >> i & 1)) {
                    std::printf("n %d first %d key %d\n", s.n, s.first, j);
                    return 1;
                }
            }
        }
    }
    std::printf("bits hold\n");
}
"""


def test_mask_bits_stay_in_bounds(tmp_path):
    src, exe = tmp_path / "bits.cpp", tmp_path / "bits"
    src.write_text(BITS_CHECK)
    r = subprocess.run([hs.compiler(), "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined",
                        "-fno-sanitize-recover=undefined", "-D_GLIBCXX_ASSERTIONS", f"-I{hs.CSRC}", str(src), "-o", str(exe)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    env = {k: v for k, v in os.environ.items() if k != "LD_PRELOAD"}
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300, env=env)
    assert r.returncode == 0 and "hold" in r.stdout, (r.stdout + r.stderr)[-3000:]


@pytest.mark.skipif("QLIN_LIB_PATH" in os.environ, reason="already the sanitizer build")
def test_decode_validation_under_asan_and_ubsan(tmp_path):
    try:
        asan = hs.runtime("libasan.so")
        lib = hs.build(str(tmp_path / "libqlin_host_sanitized.so"))
    except RuntimeError as e:
        pytest.skip(f"no host sanitizer toolchain: {e}")
    env = dict(os.environ)
    env.update({"QLIN_LIB_PATH": lib, "LD_PRELOAD": asan,
                "ASAN_OPTIONS": "detect_leaks=0:halt_on_error=1:abort_on_error=1:alloc_dealloc_mismatch=0:detect_odr_violation=0",
                "UBSAN_OPTIONS": "halt_on_error=1:print_stacktrace=1"})
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", os.path.abspath(__file__)],
                       env=env, capture_output=True, text=True, timeout=600)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-4000:]
    assert " passed" in r.stdout and "ERROR: AddressSanitizer" not in out and "runtime error:" not in out


# ---- calls in which no sequence has a new token: arrays that hold nothing may be null

def test_calls_without_new_tokens_take_empty_arrays(lib):
    none = batch(max_q=0)
    assert tree(lib, tokens=0, x=None, out=None, mask=None) == q.QLIN_OK
    assert tree(lib, tokens=0, x=None, out=None, mask=None, b=none, ldm=0) == q.QLIN_OK
    assert tree(lib, b=none, mask=None, ldm=0) == q.QLIN_OK
    assert plan(lib, b=none, mask=None, ld=0) == q.QLIN_OK
    # what would be read or written is still asked for
    assert tree(lib, mask=None) == plan(lib, mask=None) == accept(lib, path=None) == compact(lib, path=None) == q.QLIN_ERR_NULL
    assert tree(lib, b=none, mask=None, ldm=-1) == plan(lib, b=none, mask=None, ld=-1) == q.QLIN_ERR_SHAPE


def test_short_rows_of_logits_take_no_workspace(lib):
    size = lib.qlin_sample_workspace_bytes
    assert all(size(rows, vocab) == 0 for rows in (1, 16, 128) for vocab in (1, 32000, 49152))
    assert size(1, 49153) > 0 and size(64, 49153) > 0 and size(65, 49153) == 0
    assert size(85, 81919) == 0 and size(85, 81920) > 0
    assert size(128, (1 << 17) - 1) == 0 and size(128, 1 << 17) > 0 and size(129, 1 << 18) == 0
    for rows in range(1, 129):
        for vocab in (49153, 65536, 65537, 81920, 98304, 98305, 131071, 131072, 200000, 1 << 18):
            part = 16 + 2048 * 12
            parts = size(rows, vocab) // rows // part
            assert size(rows, vocab) == rows * parts * part and parts * rows <= 256 and parts <= 16 and parts != 1
