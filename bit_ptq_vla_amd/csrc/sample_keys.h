// Logits as ordered integers: the keys that sampling searches and narrows, and the
// limits that stand for a range of them in comparisons of floats.  Plain C++ (no HIP
// types), so that a host build can run it over any range.
#pragma once

#include <stdint.h>
#include <string.h>

#ifdef __HIPCC__
#define QLIN_KEY_HD __host__ __device__ __forceinline__
#else
#define QLIN_KEY_HD inline
#endif

namespace qlin {

// Equal logits (the zeros too) have equal keys.  NaN is -infinity: neither is ever taken.
constexpr uint32_t kKeyNone = 0x007FFFFFu;      // of -infinity
// The one between the largest negative number's and that of the zeros, which no logit
// has: read as a float it is -0, which compares equal to the zeros above it.
constexpr uint32_t kKeyMinusZero = 0x7FFFFFFFu;

QLIN_KEY_HD uint32_t float_bits(float v) {
    uint32_t b;
    memcpy(&b, &v, 4);
    return b;
}
QLIN_KEY_HD uint32_t key_of(float v) {
    if (v != v) return kKeyNone;
    const uint32_t b = float_bits(v + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
QLIN_KEY_HD float logit_of(uint32_t key) {
    const uint32_t b = key & 0x80000000u ? key & 0x7FFFFFFFu : ~key;
    float v;
    memcpy(&v, &b, 4);
    return v;
}

// Keys lo to hi.  An element lies in the range where logit_of(lo) <= its logit <=
// logit_of(hi): hi is not kKeyMinusZero, nor is that all of the range.
struct KeyRange {
    uint32_t lo, hi;
};

// The part b of a range that is cut, from its end down, into parts of 2^shift keys (a
// part in which some element lies).
QLIN_KEY_HD KeyRange part_of_range(KeyRange range, int shift, uint32_t b) {
    const uint32_t hi = range.hi - (b << shift), part = (1u << shift) - 1, lo = hi - range.lo > part ? hi - part : range.lo;
    return {lo, hi == kKeyMinusZero && lo < hi ? hi - 1 : hi};
}

}  // namespace qlin
