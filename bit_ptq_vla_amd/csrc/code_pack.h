// Storage of quantizer codes: int8, packed int4 and FP6 E2M3 fields.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qlin {

// Packs eight codes held as the low bytes of words (magic-biased floats or doubles,
// or integers):
// int8 -> two dwords of bytes, int4 -> one dword of nibbles (element 2j in the
// low nibble of byte j).  v_perm_b32 gathers byte 0 of its two sources.
__device__ __forceinline__ uint2 pack8_i8(const uint32_t cb[8]) {
    const uint32_t a = __builtin_amdgcn_perm(cb[1], cb[0], 0x0C0C0400u);
    const uint32_t b = __builtin_amdgcn_perm(cb[3], cb[2], 0x04000C0Cu);
    const uint32_t c = __builtin_amdgcn_perm(cb[5], cb[4], 0x0C0C0400u);
    const uint32_t d = __builtin_amdgcn_perm(cb[7], cb[6], 0x04000C0Cu);
    return make_uint2(a | b, c | d);
}

__device__ __forceinline__ uint32_t pack8_i4(const uint32_t cb[8]) {
    // even elements -> bytes of E, odd elements -> bytes of O, then nibbles
    const uint32_t e = __builtin_amdgcn_perm(cb[2], cb[0], 0x0C0C0400u) |
                       __builtin_amdgcn_perm(cb[6], cb[4], 0x04000C0Cu);
    const uint32_t o = __builtin_amdgcn_perm(cb[3], cb[1], 0x0C0C0400u) |
                       __builtin_amdgcn_perm(cb[7], cb[5], 0x04000C0Cu);
    return (e & 0x0F0F0F0Fu) | ((o << 4) & 0xF0F0F0F0u);
}

// E2M3 fields (FP6: sign, 2 exponent bits with bias 1, 3 mantissa bits) of
// the int4-grid codes 0 .. 7, and of n - 16 for the two's complement nibbles
// n = 9 .. 15, by byte (n = 8, the code -8, never occurs: the grid is
// symmetric).  1 = 1.0 x 2^0 is 0b001000, 3 = 1.5 x 2^1 is 0b010100,
// 7 = 1.75 x 2^2 is 0b011110; negative codes set bit 5.
constexpr uint32_t kE2m3PosLo = 0x14100800u, kE2m3PosHi = 0x1E1C1A18u;
constexpr uint32_t kE2m3NegLo = 0x3A3C3E00u, kE2m3NegHi = 0x28303438u;

// Eight codes held as the low bytes of words -> 48 bits of
// E2M3 fields, code j at bits 6j .. 6j+5 (w.x bits 0..31, then w.y bits 0..15).
// Per byte: the field of the low three bits from the positive or the negative
// table (v_perm_b32 byte lookups), chosen by the byte's sign, which v_perm
// selectors 8 .. 11 replicate (the sign bits of bytes 1 and 3 of each source:
// x << 8 supplies bytes 0 and 2 there).
__device__ __forceinline__ uint2 pack8_e2m3(const uint32_t cb[8]) {
    const uint2 bytes = pack8_i8(cb);
    uint32_t f24[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t x = h ? bytes.y : bytes.x;
        const uint32_t sel = x & 0x07070707u;
        const uint32_t pos = __builtin_amdgcn_perm(kE2m3PosHi, kE2m3PosLo, sel);
        const uint32_t neg = __builtin_amdgcn_perm(kE2m3NegHi, kE2m3NegLo, sel);
        const uint32_t negm = __builtin_amdgcn_perm(x << 8, x, 0x090B080Au);
        const uint32_t c = (neg & negm) | (pos & ~negm);
        // four 6-bit fields from four bytes: pairs to 12 bits, then 24
        const uint32_t t = (c & 0x003F003Fu) | ((c >> 2) & 0x0FC00FC0u);
        f24[h] = (t & 0xFFFu) | ((t >> 4) & 0x00FFF000u);
    }
    return make_uint2(f24[0] | (f24[1] << 24), f24[1] >> 8);
}

// E2M3 store of a lane's eight codes at columns col .. col+7 of a row whose
// codes start at row_out (3 bytes per 4 codes).  The lanes 2j and 2j+1 hold
// consecutive chunks of the same row (their columns are 8 apart), so the pair
// forms 12 bytes at a 4-byte aligned offset and the even lane stores them.
// Both lanes of a pair must be active (same row, same column validity).
__device__ __forceinline__ void store8_e2m3(const uint32_t cb[8], uint8_t* row_out, int64_t col, int lane) {
    const uint2 w = pack8_e2m3(cb);
    // quad_perm [1, 0, 3, 2]: the partner lane's 48 bits
    const uint32_t o0 = static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(w.x), 0xB1, 0xF, 0xF, false));
    const uint32_t o1 = static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(w.y), 0xB1, 0xF, 0xF, false));
    if ((lane & 1) == 0) {
        uint32_t* out = reinterpret_cast<uint32_t*>(row_out + (col >> 3) * 6);
        out[0] = w.x;
        out[1] = (w.y & 0xFFFFu) | (o0 << 16);
        out[2] = (o0 >> 16) | (o1 << 16);
    }
}

// Codes of one chunk (the low bytes of eight words) to their storage: int8, packed
// int4 (two per byte) or E2M3 (see store8_e2m3).
__device__ __forceinline__ void store8_codes(int bits, const uint32_t cb[8], void* q, int64_t row, int64_t k,
                                             int64_t col, int lane) {
    if (bits == 8) {
        int8_t* out = static_cast<int8_t*>(q) + row * k + col;
        *reinterpret_cast<uint2*>(out) = pack8_i8(cb);
    } else if (bits == 4) {
        uint8_t* out = static_cast<uint8_t*>(q) + row * (k / 2) + col / 2;
        *reinterpret_cast<uint32_t*>(out) = pack8_i4(cb);
    } else {
        store8_e2m3(cb, static_cast<uint8_t*>(q) + row * (k / 4 * 3), col, lane);
    }
}

}  // namespace qlin
