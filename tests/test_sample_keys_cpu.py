"""Ranges of logits' keys on the host: the elements that lie in a range by their keys
are those that do by comparisons of floats, for every part that sampling narrows a
range to.  (A zero counted in a part that ends below it has a place before the part's
first.)"""

import os
import subprocess

from bit_ptq_vla_amd import build_host_sanitized as hs

CHECK = r"""
#include <cmath>
#include <cstdio>
#include <random>
#include <vector>
#include "sample_keys.h"
using namespace qlin;

static const float kFar[] = {0.f, -0.f, 1.f, -1.f, 0x1p-149f, -0x1p-149f, 0x1p-126f, -0x1p-126f, 3.402823466e38f,
                             -3.402823466e38f, INFINITY};

// what a wave does: a comparison with both limits, then the place among the parts
static bool check(KeyRange r, int shift, float v) {
    const uint32_t k = key_of(v);
    const bool in = logit_of(r.lo) <= v && v <= logit_of(r.hi);
    if (in != (r.lo <= k && k <= r.hi) || (in && (r.hi - k) >> shift > 2047)) {
        std::printf("range %08x .. %08x, logit %a (key %08x)\n", r.lo, r.hi, v, k);
        return false;
    }
    return true;
}

// narrows as sampling does, to the part that holds each of the values
static bool narrow(KeyRange r, const std::vector<float>& values) {
    for (float v : values) {
        KeyRange x = r;
        while (x.lo < x.hi) {
            const uint32_t width = x.hi - x.lo;
            const int shift = width < 2048 ? 0 : 21 - __builtin_clz(width);
            for (float w : values)
                if (!check(x, shift, w)) return false;
            const uint32_t k = key_of(v);
            if (k < x.lo || k > x.hi) break;
            x = part_of_range(x, shift, (x.hi - k) >> shift);
        }
        for (float w : values)
            if (!check(x, 31, w)) return false;
    }
    return true;
}

int main() {
    std::mt19937 g(3);
    std::vector<float> values(kFar, kFar + sizeof(kFar) / sizeof(kFar[0]));
    for (int i = 1; i < 300; i += 7) {
        values.push_back(i * 0x1p-149f);
        values.push_back(i * -0x1p-149f);
    }
    // a row whose largest is 255 denormal steps: parts of 2^19 keys, then of 2^8, the second of
    // which ends right below the zeros
    for (uint32_t steps = 1; steps < 5000; ++steps)
        if (!narrow({kKeyNone + 1, 0x80000000u + steps}, values)) return 1;
    for (int it = 0; it < 3000; ++it) {
        uint32_t lo = g() % 0xFF000000u, hi = g() % 0xFF800001u;
        if (it % 3 == 0) hi = 0x80000000u + g() % (1u << g() % 31);
        if (it % 2 == 0) lo = 0x80000000u - g() % (1u << g() % 31);
        if (hi > 0xFF800000u) hi = 0xFF800000u;
        if (lo <= kKeyNone) lo = kKeyNone + 1;
        if (hi < lo || hi == kKeyMinusZero) continue;
        if (!narrow({lo, hi}, values)) return 1;
    }
    std::printf("ranges hold\n");
}
"""


def test_ranges_hold_by_keys_and_by_floats(tmp_path):
    src, exe = tmp_path / "keys.cpp", tmp_path / "keys"
    src.write_text(CHECK)
    r = subprocess.run([hs.compiler(), "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined",
                        "-fno-sanitize-recover=undefined", f"-I{hs.CSRC}", str(src), "-o", str(exe)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    env = {k: v for k, v in os.environ.items() if k != "LD_PRELOAD"}
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300, env=env)
    assert r.returncode == 0 and "hold" in r.stdout, (r.stdout + r.stderr)[-3000:]
