// Residual addition -> RMS norm -> block Hadamard -> per-token quantization,
// for gfx950: what stands between a layer's residual stream and its next
// low-bit projection.
//
//   r = rne_T(x + res),   n_j = r_j w_j / sqrt(mean(r^2) + eps),
//   v = n @ blockdiag(H_b / sqrt b),   x_scale = fp32(max|v| / qmax),
//   code_j = rne(qmax v_j / max|v|)
//
// The codes do not depend on the row's norm or on 1/sqrt b: both cancel in
// v_j / max|v|.  So one pass over the row serves: u = (r w) @ H (the +-1
// transform) with its maximum and the sum of squares reduced together, codes
// from u, and x_scale = max|u| / (qmax sqrt b rms).
//
// u is held in float64.  A 16-bit r times an fp32 w is exact there and the
// transform's sums are off by a few 2^-53, so the codes are those of exact
// arithmetic (ties to even) and equal a float64 reference's; the vector
// float64 rate of this chip is its unpacked fp32 rate.  The sum of squares is
// float64 too, so no fp32 row can overflow it.
//
// A row is held by g lanes (a power of two), lane t holding the 8 values from
// 8 (c g + t) for chunk c: one chunk up to 8192 values.  (At 52224 x 2048 bf16,
// Hadamard 128, one, two and four chunks a lane take 168, 161 and 171 us.)
//
// Bound by vector issue at the backbone's widths: 53 instructions per 64 values
// with a Hadamard of 128, 151 us of the 168 us that 52224 x 2048 bf16 rows take
// (749 MB: 4.5 TB/s; a copy moves 5.1).  Without a transform 156, to int4 codes
// 167, to E2M3 177, the float output 146, fp32 rows 241.

#include <cmath>

#include "code_pack.h"
#include "device_common.h"
#include "qlin_internal.h"

namespace qlin {

namespace {

struct NormParams {
    const void* x;
    const void* res;     // or nullptr
    void* res_out;       // r, or nullptr
    const float* w;      // [k]
    int64_t m, k, ldx, ldr;
    float eps;
    int g;               // lanes per row
    int had_block;       // 0/1: none
    int bits;            // 8, 4 or 6; 0: float output
    double unscale;      // 1 / (qmax sqrt b)
    void* q;             // codes, or y
    float* scale;
};

// Lane (lane ^ D)'s double: its two halves by DPP where a pattern exists
// (D = 1, 2, 8), else through the LDS crossbar.
template <int D>
__device__ __forceinline__ int lane_xor_i(int v) {
    if constexpr (D == 1) return __builtin_amdgcn_mov_dpp(v, 0xB1, 0xF, 0xF, false);
    else if constexpr (D == 2) return __builtin_amdgcn_mov_dpp(v, 0x4E, 0xF, 0xF, false);
    else if constexpr (D == 8) return __builtin_amdgcn_mov_dpp(v, 0x128, 0xF, 0xF, false);   // row_ror:8
    else if constexpr (D == 32) return __shfl_xor(v, 32, 64);
    else return __builtin_amdgcn_ds_swizzle(v, (D << 10) | 0x1F);
}
template <int D>
__device__ __forceinline__ double lane_xor_d(double v) {
    return __hiloint2double(lane_xor_i<D>(__double2hiint(v)), lane_xor_i<D>(__double2loint(v)));
}

// The double a DPP pattern brings (the reductions' steps: the two quad swaps,
// then the half-row and row mirrors, which meet the other half's result).
template <int CTRL>
__device__ __forceinline__ double across(double v) {
    return __hiloint2double(__builtin_amdgcn_mov_dpp(__double2hiint(v), CTRL, 0xF, 0xF, false),
                            __builtin_amdgcn_mov_dpp(__double2loint(v), CTRL, 0xF, 0xF, false));
}

template <int D, int NCH>
__device__ __forceinline__ void xlane_stage_d(double (&v)[NCH][8], int lane) {
    const double sgn = (lane & D) ? -1.0 : 1.0;
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[c][e] = fma(v[c][e], sgn, lane_xor_d<D>(v[c][e]));
}

template <int DT>
__device__ __forceinline__ float round_to(float f) {
    if constexpr (DT == BF16) return bf16_to_f32(f32_to_bf16_rne(f));
    else if constexpr (DT == F16) return f16_bits_to_f32(f32_to_f16_bits(f));
    else return f;
}

// max(m, |a|) in one instruction (fmax first quiets operands the compiler does
// not know to be canonical; a NaN operand is ignored either way).
__device__ __forceinline__ double max_abs(double m, double a) {
    double r;
    asm("v_max_f64 %0, %1, |%2|" : "=v"(r) : "v"(m), "v"(a));
    return r;
}

// HB: the Hadamard block at compile time (1: none), or 0 to take it from the
// arguments.  A known block leaves the transform without branches, whose joins
// cost a move a value and stage.
template <int DT, int NCH, int TPB, bool QUANT, int HB>
__global__ __launch_bounds__(TPB) void add_rmsnorm_kernel(NormParams p) {
    constexpr int ES = DT == F32 ? 4 : 2;
    constexpr int NW = TPB / 64;
    __shared__ double red[2][NW];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int g = p.g, t = tid & (g - 1);
    const int b = HB > 0 ? HB : p.had_block > 1 ? p.had_block : 1;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (TPB / g) + tid / g;
    const bool row_ok = row < p.m;
    const int64_t rr = row_ok ? row : p.m - 1;
    const char* xrow = static_cast<const char*>(p.x) + rr * p.ldx * ES;
    const char* rrow = static_cast<const char*>(p.res) + rr * p.ldr * ES;
    char* orow = static_cast<char*>(p.res_out) + rr * p.ldr * ES;

    bool ok[NCH];
    int64_t col[NCH];
    float r[NCH][8];
    double ss = 0.0;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
        col[c] = (static_cast<int64_t>(c) * g + t) * 8;
        ok[c] = col[c] < p.k;
        if (!ok[c]) col[c] = 0;
        load8<DT>(xrow + col[c] * ES, r[c]);
        if (p.res) {
            float a[8];
            load8<DT>(rrow + col[c] * ES, a);
#pragma unroll
            for (int e = 0; e < 8; ++e) r[c][e] = round_to<DT>(r[c][e] + a[e]);
        }
        if (!ok[c]) {
#pragma unroll
            for (int e = 0; e < 8; ++e) r[c][e] = 0.f;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fma(static_cast<double>(r[c][e]), static_cast<double>(r[c][e]), ss);
    }
    if (p.res_out && row_ok) {
#pragma unroll
        for (int c = 0; c < NCH; ++c)
            if (ok[c]) store8<DT>(orow + col[c] * ES, r[c]);
    }

    double v[QUANT ? NCH : 1][8];
    double top = 0.0;
    if constexpr (QUANT) {
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            float w[8];
            load8<F32>(p.w + col[c], w);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[c][e] = static_cast<double>(r[c][e]) * static_cast<double>(w[e]);
#pragma unroll
            for (int h = 1; h < 8; h <<= 1) {
                if (h < b) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        if ((e & h) == 0) {
                            const double a0 = v[c][e], a1 = v[c][e + h];
                            v[c][e] = a0 + a1;
                            v[c][e + h] = a0 - a1;
                        }
                    }
                }
            }
        }
        if (b > 8) xlane_stage_d<1, NCH>(v, lane);
        if (b > 16) xlane_stage_d<2, NCH>(v, lane);
        if (b > 32) xlane_stage_d<4, NCH>(v, lane);
        if (b > 64) xlane_stage_d<8, NCH>(v, lane);
        if (b > 128) xlane_stage_d<16, NCH>(v, lane);
#pragma unroll
        for (int c = 0; c < NCH; ++c)
#pragma unroll
            for (int e = 0; e < 8; ++e) top = max_abs(top, v[c][e]);
    }

    // the row's sum of squares and maximum: lanes (g >= 32), then waves
    ss += across<0xB1>(ss);
    ss += across<0x4E>(ss);
    ss += across<0x141>(ss);
    ss += across<0x140>(ss);
    ss += lane_xor_d<16>(ss);
    if (g > 32) ss += lane_xor_d<32>(ss);
    if constexpr (QUANT) {
        top = max_abs(top, across<0xB1>(top));
        top = max_abs(top, across<0x4E>(top));
        top = max_abs(top, across<0x141>(top));
        top = max_abs(top, across<0x140>(top));
        top = max_abs(top, lane_xor_d<16>(top));
        if (g > 32) top = max_abs(top, lane_xor_d<32>(top));
    }
    if (g > 64) {
        if (lane == 0) {
            red[0][wave] = ss;
            red[1][wave] = top;
        }
        __syncthreads();
        const int wpr = g >> 6, first = (wave / wpr) * wpr;
        ss = red[0][first];
        top = red[1][first];
        for (int i = 1; i < wpr; ++i) {
            ss += red[0][first + i];
            top = fmax(top, red[1][first + i]);
        }
    }
    if (!row_ok) return;

    if constexpr (QUANT) {
        const double qmax = p.bits == 8 ? 127.0 : 7.0;
        if (t == 0) {
            const double rms = sqrt(ss / static_cast<double>(p.k) + static_cast<double>(p.eps));
            // a row of zeros has scale 0 (also at eps = 0)
            p.scale[row] = ss == 0.0 ? 0.f : static_cast<float>(top * p.unscale / rms);
        }
        // qmax / top to a few 2^-52: the reciprocal's 2^-20 or better, squared twice
        // (a subnormal or zero top, or one whose reciprocal is, takes the quotients)
        double inv = 0.0;
        const bool fast = top > 1e-290 && top < 1e290;
        if (fast) {
            inv = __builtin_amdgcn_rcp(top);
            inv = fma(fma(-top, inv, 1.0), inv, inv);
            inv = fma(fma(-top, inv, 1.0), inv, inv) * qmax;
        }
        // fma(v, inv, M) with M = 1.5 * 2^52 rounds the product to an integer
        // once, half to even, and leaves it in the low mantissa bits; |v| <= top
        // keeps it on the grid.  The product is off by 2^-43 at most
        // for codes up to 127: a residual that close to a half (the window is
        // far wider) is decided by the quotient itself.
        constexpr double M = 6755399441055744.0;
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            uint32_t cb[8];
            double worst = 0.0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const double qb = fma(v[c][e], inv, M);
                worst = max_abs(worst, fma(v[c][e], inv, M - qb));
                cb[e] = static_cast<uint32_t>(__double2loint(qb));
            }
            if (worst >= 0.5 - 1e-9 || !fast) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    cb[e] = static_cast<uint32_t>(
                        __double2loint((top > 0.0 ? rint(v[c][e] * qmax / top) : 0.0) + M));
            }
            if (ok[c]) store8_codes(p.bits, cb, p.q, row, p.k, col[c], lane);
        }
    } else {
        const double rms = sqrt(ss / static_cast<double>(p.k) + static_cast<double>(p.eps));
        const double inv64 = ss == 0.0 ? 0.0 : 1.0 / rms;
        const float inv = static_cast<float>(inv64);
        // a reciprocal near the ends of fp32's range multiplies in float64
        const bool plain = inv64 < 0x1p126 && (inv64 > 0x1p-126 || ss == 0.0);
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            float w[8];
            load8<F32>(p.w + col[c], w);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                r[c][e] = (plain ? r[c][e] * inv : static_cast<float>(r[c][e] * inv64)) * w[e];
            if (ok[c]) store8<DT>(static_cast<char*>(p.q) + (row * p.k + col[c]) * ES, r[c]);
        }
    }
}

template <int DT, int NCH, int TPB>
hipError_t launch_tpb(const NormParams& p, hipStream_t st) {
    const int64_t rpb = TPB / p.g;
    const dim3 grid(static_cast<unsigned>((p.m + rpb - 1) / rpb));
    // The blocks 1, 64 and 128 are compiled in for 16-bit rows of up to 8192 values,
    // those of the quantized layers: 52224 x 2048 bf16 take 164 us with 64 (175 with
    // the block from the arguments) and 168 with 128 (182).  The others take it from
    // the arguments: 32 takes 169 us, 256 190.  Above 8192 values a lane holds several
    // chunks: as many values in rows of 16384 take 189 us without a transform and 244
    // with 128, in rows of 32768 282 and 301 (32 registers spill).
    constexpr bool known = DT != F32 && NCH == 1;
    if (!p.bits)
        add_rmsnorm_kernel<DT, NCH, TPB, false, 1><<<grid, TPB, 0, st>>>(p);
    else if (known && p.had_block <= 1)
        add_rmsnorm_kernel<DT, NCH, TPB, true, known ? 1 : 0><<<grid, TPB, 0, st>>>(p);
    else if (known && p.had_block == 64)
        add_rmsnorm_kernel<DT, NCH, TPB, true, known ? 64 : 0><<<grid, TPB, 0, st>>>(p);
    else if (known && p.had_block == 128)
        add_rmsnorm_kernel<DT, NCH, TPB, true, known ? 128 : 0><<<grid, TPB, 0, st>>>(p);
    else
        add_rmsnorm_kernel<DT, NCH, TPB, true, 0><<<grid, TPB, 0, st>>>(p);
    return hipGetLastError();
}

template <int DT>
hipError_t launch_dt(NormParams p, hipStream_t st) {
    int g = 32;
    while (g < 1024 && g * 8 < p.k) g <<= 1;
    p.g = g;
    if (g <= 256) return launch_tpb<DT, 1, 256>(p, st);
    if (g == 512) return launch_tpb<DT, 1, 512>(p, st);
    if (p.k <= 8192) return launch_tpb<DT, 1, 1024>(p, st);
    if (p.k <= 16384) return launch_tpb<DT, 2, 1024>(p, st);
    return launch_tpb<DT, 4, 1024>(p, st);
}

}  // namespace

hipError_t launch_add_rmsnorm(const void* x, int dtype, int64_t m, int64_t k, int64_t ldx, const void* res,
                              int64_t ldr, const float* w, float eps, int had_block, int bits, void* res_out,
                              void* q, float* scale, hipStream_t st) {
    const double unscale = 1.0 / ((bits == 8 ? 127.0 : 7.0) * std::sqrt(had_block > 1 ? had_block : 1));
    NormParams p{x, res, res_out, w, m, k, ldx, ldr, eps, 0, had_block, bits, unscale, q, scale};
    switch (dtype) {
        case F16: return launch_dt<F16>(p, st);
        case BF16: return launch_dt<BF16>(p, st);
        default: return launch_dt<F32>(p, st);
    }
}

}  // namespace qlin
