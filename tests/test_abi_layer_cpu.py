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
