// What the attention kernels over the paged int8 cache share: their arguments, the
// arithmetic of scores, weights and scales, the kernel for many query rows, and the
// join of split keys.
//
// TREE: the new tokens are the nodes of a tree, and which of them a query sees
// stands in its mask row.  Only the steps that reach behind the cached keys read
// masks, 8 or 16 keys to a lane as bits of one shifted word; a block reads the
// keys to the sequence's end, whatever its rows.
#pragma once

#include "device_common.h"
#include "kv_index.h"
#include "qlin_internal.h"

namespace qlin {

namespace {

typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));

struct AttnParams {
    KvIndex ix;
    const void* q;
    int64_t ldq;
    const int8_t* k;
    const int8_t* v;
    const float* ks;
    const float* vs;
    void* out;
    int64_t ldo;
    int heads_q, heads, group;
    float sm_scale, cap;
    int row_tiles, splits, split_keys;
    float* part_o;     // [splits][batch * max_q][heads_q][D]; with even: [2 even][rows of a block][D]
    float* part_ml;    // [splits][batch * max_q][heads_q][2]
    const uint32_t* mask;   // [tokens][mask_ld] of a tree, or nullptr
    int64_t mask_ld;
    uint32_t even;          // blocks that share a tree's steps evenly, or 0
    uint32_t* shares;       // [64] running sums of the sequences' steps
};

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNegInf = -__builtin_inff();
// Octaves below vr at which a page's v scale stops: what its keys weigh in the sum
// (2^80 to 2^88 each, where a key of the largest scale weighs 1 to 2^8) stays
// inside fp32.  A row whose sum passes 2^79 saw none but such pages, up to the
// number of its keys: those count as zeros.  (A sum past the top is such a row's.)
constexpr float kFloor = 80.f, kOnlyZeros = 0x1p79f, kSumTop = 0x1p112f;

// log2(vs / vr) down to the floor (NaN, both zero, becomes it too).
__device__ __forceinline__ float scale_log(float vs, float vr) {
    return fmaxf(__builtin_amdgcn_logf(vs) - __builtin_amdgcn_logf(vr), -kFloor);
}

// The largest v scale rises from vr to vn and the exponents seen have a new
// maximum top: a row's reference m, its sum l, and the factor of its products.
// In units of vn a row's earlier exponents are lower, and so is its reference
// (past 2^20, where exponents are rounded by more than 2^-5, it stays).
__device__ __forceinline__ float follow(float& m, float& l, float& vr, float vn, float top) {
    const float rise = vr > 0.f && fabsf(m) < 0x1p20f ? -scale_log(vr, vn) : 0.f;
    const float mn = fmaxf(m - rise, top);
    const float r = m > kNegInf ? __builtin_amdgcn_exp2f(m - mn) : 1.f;
    const float ro = vr > 0.f ? r * (vr / vn) : 0.f;      // (products of zero scales count nothing)
    l = fminf(l * r, kSumTop);
    m = mn;
    vr = vn;
    return ro;
}

// Eight codes (two words) as fp16.
__device__ __forceinline__ h8 codes_f16(uint32_t w0, uint32_t w1) {
    const h2 off = {static_cast<_Float16>(-1152.f), static_cast<_Float16>(-1152.f)};
    const uint32_t a = w0 ^ 0x80808080u, b = w1 ^ 0x80808080u;
    const h2 r0 = __builtin_bit_cast(h2, __builtin_amdgcn_perm(0x64646464u, a, 0x04010400u)) + off;
    const h2 r1 = __builtin_bit_cast(h2, __builtin_amdgcn_perm(0x64646464u, a, 0x04030402u)) + off;
    const h2 r2 = __builtin_bit_cast(h2, __builtin_amdgcn_perm(0x64646464u, b, 0x04010400u)) + off;
    const h2 r3 = __builtin_bit_cast(h2, __builtin_amdgcn_perm(0x64646464u, b, 0x04030402u)) + off;
    return h8{r0[0], r0[1], r1[0], r1[1], r2[0], r2[1], r3[0], r3[1]};
}

// Maximum / sum over the four lane groups that share a query (lane ^ 16, ^ 32).
__device__ __forceinline__ float groups_max(float v) {
    v = fmaxf(v, lane_xor<16>(v));
    return fmaxf(v, lane_xor<32>(v));
}
__device__ __forceinline__ float groups_sum(float v) {
    v += lane_xor<16>(v);
    return v + lane_xor<32>(v);
}

// A score in base-2 units from the raw product, capped where CAP, plus add.
template <bool CAP>
__device__ __forceinline__ float score(float raw, float mul, float cap_out, float add) {
    if constexpr (CAP) {
        // c tanh(x / c) = c (1 - 2 / (1 + exp(2 x / c))): mul holds 2 / c * log2 e, cap_out c log2 e
        const float e = __builtin_amdgcn_exp2f(raw * mul);
        return cap_out + add - 2.f * cap_out * __builtin_amdgcn_rcpf(1.f + e);
    } else {
        return fmaf(raw, mul, add);
    }
}

// One query row of a block: column c holds row r0 + c of the (token, head of the group) rows.
struct Row {
    bool ok;
    int64_t token;      // row of q and out
    int64_t slot;       // row of the partials
    int head;
    int vis;            // keys it sees
};

template <bool TREE>
__device__ __forceinline__ Row row_of(const AttnParams& p, const KvSeq& s, int b, int h, int r) {
    Row x;
    const int i = r / p.group;
    x.ok = i < s.n;
    const int ii = x.ok ? i : 0;
    x.token = s.row0 + ii;
    x.slot = static_cast<int64_t>(b) * p.ix.max_q + ii;
    x.head = h * p.group + r % p.group;
    x.vis = !x.ok ? 0 : TREE ? s.kv : kv_visible(p.ix, s, b, s.first + i);
    return x;
}

// ---- many query rows ---------------------------------------------------------

// Byte offset of 16-byte chunk `c` of K row `row` in LDS: D fp16 a row.  LDS has
// 64 banks and serves a 16-byte access sixteen lanes at a time: the xor makes the
// sixteen lanes that read one chunk of sixteen rows, or write every other chunk
// of one or more rows, cover all 256 bytes.
template <int D>
__device__ __forceinline__ int k_off(int row, int c) {
    const int x = D == 64 ? (row >> 1) & 7 : (row & 15) ^ (c >> 4);
    return row * D * 2 + ((c ^ x) << 4);
}
// The same for V: 64 keys (8 chunks) a dimension.
__device__ __forceinline__ int v_off(int d, int c) { return d * 128 + ((c ^ ((d >> 1) & 7)) << 4); }

// The LDS row of key j (0..63) of a step.  The 32x32 product leaves lane half h
// with rows 8 (i / 4) + 4 h + i % 4 in element i; with this order elements
// 8 u .. 8 u + 7 of a lane are keys 16 u + 8 h + (0..7): B operand u of P^T as
// it stands, against V in its stored order.
__device__ __forceinline__ int key_row(int j) {
    return (j & 48) | ((j & 4) << 1) | ((j & 8) >> 1) | (j & 3);
}

// 32 query rows to a wave, eight waves to a block; HV waves share 32 rows of a
// 256-wide head and keep D / HV dimensions of their output each.  The waves run
// in two groups, four (one to a SIMD) each, half a step apart: while one group
// feeds the matrix units (the last step's P V, then this step's K Q) the other
// does its softmax, so the two kinds of work overlap on every SIMD:
//   phase      2t            2t + 1      2t + 2
//   group 0    PV(t-1) QK(t) softmax(t)  PV(t) QK(t+1)
//   group 1    softmax(t-1)  PV(t-1) QK(t)  softmax(t)
// Each group stages its half of K(t + 1) and V(t) between the products of PV(t-1)
// and QK(t): after the last use of K(t - 1) and V(t - 2), before the next of both.
//
// Bound by the matrix units and the softmax's issue beside them: 8192 causal
// tokens (32 heads over 8, 128 wide, 549 GFLOP) take 622 us, 882 TFLOP/s, 63% of
// a large fp16 product's rate (1.4 PFLOP/s on the same card); four waves that did
// both kinds of work in turn took 643 where these took 620.  256-wide heads
// compute K Q, the softmax and the cap in both waves of a pair, and one block fits
// a CU: prompts of up to 816 tokens, 8 x 8 capped heads, are two uneven rounds of
// blocks, 28.6 GFLOP in 110 us with neither unit busy half of the time.
//
// One block's rows r0 .. of a (sequence, kv head) against the keys k0 .. k1 - 1 (k0 a
// multiple of 64); part(row, number) is where a row's partial result goes, -1: the
// result is whole.
template <int D>
constexpr int kPhaseRows = D == 256 ? 128 : 256;

template <int DT, int D, bool CAP, bool TREE, typename F>
__device__ __forceinline__ void phase_unit(const AttnParams& p, char* lds, const KvSeq& s, int b, int h, int r0, int k0,
                                           int k1, F part_of) {
    constexpr int TPB = 512;
    constexpr int HV = D == 256 ? 2 : 1;
    constexpr int ROWS = kPhaseRows<D>;
    constexpr int NS = D / 16;            // k steps of S
    constexpr int ND = D / 32 / HV;       // 32-dimension tiles of the wave's output
    constexpr int NC = D * 4 / TPB > 0 ? D * 4 / TPB : 1;   // 16-byte pieces of k (and of v) a thread stages
    constexpr int AHEAD = D == 256 ? 3 : 6;
    constexpr bool PART = D * 4 < TPB;    // only the first D * 4 threads stage
    constexpr int KB = 64 * D * 2;        // bytes of one operand of a step in LDS
    typedef float f16v __attribute__((ext_vector_type(16)));

    const int rows = s.n * p.group;
    const int last = (r0 + ROWS < rows ? r0 + ROWS : rows) - 1;
    const int steps = k1 > k0 ? (k1 - k0 + 63) >> 6 : 0;

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int grp = wave >> 2, half = HV == 2 ? wave & 1 : 0;
    const int c = lane & 31, hf = lane >> 5;
    const int rw = r0 + 32 * (wave / HV);                // the wave's first row
    const Row row = row_of<TREE>(p, s, b, h, rw + c < rows ? rw + c : last);
    const int vis = rw + c < rows ? row.vis : 0;
    // the wave's rows see at least these keys
    const int wave_lo = rw + 31 >= rows ? 0 : TREE ? s.first : row_of<TREE>(p, s, b, h, rw).vis;
    const uint32_t* mask = TREE ? p.mask + row.token * p.mask_ld : nullptr;
    const int ps = p.ix.page_size, psl = 31 - __builtin_clz(ps);
    const int last_idx = s.kv > 0 ? (s.kv - 1) >> psl : 0;

    // Lane x of each four holds what belongs to granule x of a step: its page,
    // scales and whether it has keys; a piece of v lies in the granule of its own
    // lane, a piece of k in one that the whole wave shares.
    const int x4 = lane & 3;
    const int32_t* table = p.ix.page_table + static_cast<int64_t>(b) * p.ix.table_ld;
    const int64_t page_bytes = static_cast<int64_t>(ps) * D, pool_step = page_bytes * p.heads;
    const int8_t* kh = p.k + h * page_bytes;
    const int8_t* vh = p.v + h * page_bytes;
    const float* ksh = p.ks + h;
    const float* vsh = p.vs + h;
    // entry of the page table for the lane's granule of step t, and the page it
    // stands for (asked for only when it is used: nothing waits for the load)
    auto entry_of = [&](int t) {
        const int idx = (k0 + 64 * t + 16 * x4) >> psl;
        return table[idx < last_idx ? idx : last_idx];
    };
    const uint32_t pool = static_cast<uint32_t>(p.ix.pages);
    auto page_of = [&](int entry, int t) {
        const bool in = static_cast<uint32_t>(entry) < pool, short_of = k0 + 64 * t + 16 * x4 < k1;
        return (in & short_of) ? entry : kNoPage;
    };
    int en0 = 0, en1 = 0, en2 = 0;           // entries of steps t, t + 1, t + 2
    if (steps > 0) {
        en0 = entry_of(0);
        en1 = entry_of(1);
        en2 = entry_of(2);
    }
    u4 kw[NC], vw[NC];
    const bool stages = !PART || tid < D * 4;
    auto fetch_k = [&](int page) {
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            const int i = tid + n * TPB, key = i / (D / 16), kc = i % (D / 16);
            const int pk = __builtin_amdgcn_readlane(page, __builtin_amdgcn_readfirstlane(key >> 4) & 3);
            if (stages)
                kw[n] = *reinterpret_cast<const u4*>(kh + (pk < 0 ? 0 : pk) * pool_step + (key & (ps - 1)) * D + 16 * kc);
        }
    };
    auto fetch_v = [&](int page) {
        const int8_t* vp = vh + (page < 0 ? 0 : page) * pool_step + ((16 * x4) & (ps - 1));
#pragma unroll
        for (int n = 0; n < NC; ++n)
            if (stages) vw[n] = *reinterpret_cast<const u4*>(vp + ((tid + n * TPB) >> 2) * ps);
    };
    // part i of staging: half (8 codes) of piece i / 2 of k, then of v
    auto stage_part = [&](int i, int tk, int tv) {
        const int n = (i >> 1) % NC, e = (i & 1) * 2, at = tid + n * TPB;
        if (i < 2 * NC) {
            const h8 w = codes_f16(kw[n][e], kw[n][e + 1]);
            char* dst = lds + (tk & 1) * KB + k_off<D>(key_row(at / (D / 16)), 2 * (at % (D / 16)) + (i & 1));
            if (stages) *reinterpret_cast<h8*>(dst) = w;
        } else {
            const h8 w = codes_f16(vw[n][e], vw[n][e + 1]);
            char* dst = lds + 2 * KB + (tv & 1) * KB + v_off(at >> 2, 2 * x4 + (i & 1));
            if (stages) *reinterpret_cast<h8*>(dst) = w;
        }
    };
    if (steps > 0) fetch_k(page_of(en0, 0));

    // queries: dimensions 16 j + 8 hf .. + 7 of row c, with sm_scale's sign: what
    // is left of the scale is not negative, so a granule's largest score is that
    // of its largest product
    h8 qf[NS];
    const float sign = p.sm_scale < 0.f ? -1.f : 1.f;
    float qmul = fabsf(p.sm_scale);
    {
        const char* src = static_cast<const char*>(p.q) + (row.token * p.ldq + static_cast<int64_t>(row.head) * D) * 2;
        int e = 0;
        if constexpr (DT == BF16) {
            float top = 0.f;
#pragma unroll
            for (int j = 0; j < NS; ++j) {
                float f[8];
                load8<DT>(src + (16 * j + 8 * hf) * 2, f);
#pragma unroll
                for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(f[i]));
            }
            top = fmaxf(top, lane_xor<32>(top));
            if (top > 0.f && top < __builtin_inff()) e = 14 - __builtin_amdgcn_frexp_expf(top);
            e = e > 120 ? 120 : e < -120 ? -120 : e;
            qmul = __builtin_amdgcn_ldexpf(qmul, -e);
        }
#pragma unroll
        for (int j = 0; j < NS; ++j) {
            float f[8];
            load8<DT>(src + (16 * j + 8 * hf) * 2, f);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                qf[j][i] = static_cast<_Float16>(sign * (DT == BF16 ? __builtin_amdgcn_ldexpf(f[i], e) : f[i]));
        }
    }
    qmul *= CAP ? 2.f * kLog2e / p.cap : kLog2e;
    const float cap_out = CAP ? p.cap * kLog2e : 0.f;

    f16v o[ND];
#pragma unroll
    for (int t = 0; t < ND; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[t][i] = 0.f;
    float m = kNegInf, l = 0.f, vr = 0.f;
    float x[32];
    h8 pf[4];
    float ks_t = 0.f, vs_t = 0.f;            // scales of the lane's granule of step t
    float sc[4], vlog[4], vinv[4], unit = 0.f;
    int dead_t = 0;

    // The products of PV(t - 1), then of QK(t): A operands are read AHEAD products
    // before their use.  A matrix instruction that waits for its unit keeps the
    // other group's vector instructions from issuing, so each is followed by about
    // as much other issue as it runs: its read, and staging or a pause (measured
    // with one wave of each kind on a SIMD: 32.6 cycles a product and nothing
    // beside it without the pause; 34.5, and the other wave at 4/5 of its rate, with).
    constexpr int NP = 4 * ND + 2 * NS;
    auto products = [&](int t, bool second) {
        const char* vl = lds + 2 * KB + ((t - 1) & 1) * KB;
        const char* kl = lds + (t & 1) * KB;
        auto operand = [&](int i) {
            if (i < 4 * ND)
                return *reinterpret_cast<const h8*>(vl + v_off(32 * (half * ND + i / 4) + c, 2 * (i % 4) + hf));
            const int j = i - 4 * ND;
            return *reinterpret_cast<const h8*>(kl + k_off<D>(32 * (j & 1) + c, 2 * (j >> 1) + hf));
        };
        f16v a0, a1;
#pragma unroll
        for (int i = 0; i < 16; ++i) a0[i] = a1[i] = 0.f;
        const int to = second ? NP : 4 * ND;
        h8 fr[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) fr[i] = operand(i);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < to; ++i) {
            const h8 w = fr[i % AHEAD];
            if (i < 4 * ND) o[i / 4] = __builtin_amdgcn_mfma_f32_32x32x16_f16(w, pf[i % 4], o[i / 4], 0, 0, 0);
            else if ((i - 4 * ND) & 1) a1 = __builtin_amdgcn_mfma_f32_32x32x16_f16(w, qf[(i - 4 * ND) >> 1], a1, 0, 0, 0);
            else a0 = __builtin_amdgcn_mfma_f32_32x32x16_f16(w, qf[(i - 4 * ND) >> 1], a0, 0, 0, 0);
            if (i + AHEAD < to) fr[i % AHEAD] = operand(i + AHEAD);
            const int part = second && i >= 4 && (i & 1) == 0 ? (i - 4) / 2 : 4 * NC;
            if (part < 4 * NC) stage_part(part, t + 1, t);
            else asm volatile("s_nop 4");
            __builtin_amdgcn_sched_barrier(0);
        }
        if (second) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                x[i] = a0[i];
                x[16 + i] = a1[i];
            }
        }
    };
    // step t's scales, uniform over the wave
    auto scales = [&](int t) {
        const bool none = page_of(en0, t) == kNoPage;
        dead_t = static_cast<int>(__ballot(none)) & 15;
        const float ks = none ? 0.f : ks_t, vs = none ? 0.f : vs_t;
        float vtop = fmaxf(vs, dpp_mov<0xB1>(vs));
        vtop = fmaxf(vtop, dpp_mov<0x4E>(vtop));
        unit = fmaxf(vr, vtop);
        const float lg = scale_log(vs, unit);
        const float li = __builtin_amdgcn_exp2f(-lg);
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            sc[g] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(ks), g));
            vlog[g] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(lg), g));
            vinv[g] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(li), g));
        }
    };
    // x -> pf, with the row statistics
    auto softmax = [&](int t) {
        const int t0 = k0 + 64 * t;
        float sc_[4];
#pragma unroll
        for (int g = 0; g < 4; ++g) sc_[g] = qmul * sc[g];
        if (CAP) {
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = score<CAP>(x[i], sc_[i >> 3], cap_out, 0.f);
#pragma unroll
            for (int g = 0; g < 4; ++g) sc_[g] = 1.f;
        }
        // element 8 g + e is key 16 g + 8 hf + e of the step
        if (!(t0 + 64 <= wave_lo && dead_t == 0)) {
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int lim = (dead_t >> g & 1) ? 0 : vis - (t0 + 16 * g + 8 * hf);
                // (a zero scale: the scores seen are 0, and a masked one stays -inf)
                const bool zero = sc_[g] == 0.f;
                const uint32_t bits = TREE && lim > 0 ? kv_tree_bits(mask, s, t0 + 16 * g + 8 * hf) : 0;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    x[8 * g + e] = (TREE ? bits >> e & 1 : e < lim) ? (zero ? 0.f : x[8 * g + e]) : kNegInf;
                if (zero) sc_[g] = 1.f;
            }
        }
        float top = kNegInf;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            float hi = x[8 * g];
#pragma unroll
            for (int e = 1; e < 8; ++e) hi = fmaxf(hi, x[8 * g + e]);
            top = fmaxf(top, fmaf(hi, sc_[g], vlog[g]));
        }
        top = fmaxf(top, lane_xor<32>(top));
        // The weights below take x sc unrounded, off the rounded exponent by 2^-24 of
        // it: nothing up to 2^20, past the range of the exponent at the far end.
        // There they take the exponent that the maximum saw.
        float vl[4];
#pragma unroll
        for (int g = 0; g < 4; ++g) vl[g] = vlog[g];
        if (!CAP && __any(fabsf(top) > 0x1p20f && top > kNegInf)) {
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = fmaf(x[i], sc_[i >> 3], vlog[i >> 3]);
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                sc_[g] = 1.f;
                vl[g] = 0.f;
            }
        }
        // the reference follows the maximum once that is 2^8 past it: weights stay
        // below 2^8, far inside fp16, and most steps rescale nothing
        if (__any(top > m + 8.f || unit != vr)) {
            const float ro = follow(m, l, vr, unit, top);
#pragma unroll
            for (int d = 0; d < ND; ++d)
#pragma unroll
                for (int i = 0; i < 16; ++i) o[d][i] *= ro;
        }
        const float base = m > kNegInf ? m : 0.f;        // nothing seen yet: all weights 0
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const float off = vl[g] - base;
            float sum = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float w = __builtin_amdgcn_exp2f(fmaf(x[8 * g + e], sc_[g], off));
                sum += w;
                pf[g][e] = static_cast<_Float16>(w);
            }
            l = fmaf(sum, vinv[g], l);
        }
    };
    // what step t + 1's phases need, on its way during softmax(t)
    // (past the last step: some page's codes, staged and never read)
    auto ahead = [&](int t) {
        fetch_k(page_of(en2, t + 2));
        const int page = page_of(en1, t + 1);
        fetch_v(page);
        const int64_t at = static_cast<int64_t>(page < 0 ? 0 : page) * p.heads;
        ks_t = ksh[at];
        vs_t = vsh[at];
        en0 = en1;
        en1 = en2;
        en2 = entry_of(t + 3);
    };

    if (steps > 0) {
#pragma unroll
        for (int i = 0; i < 2 * NC; ++i) stage_part(i, 0, 0);
        // the first product with V meets weights of 0: its buffer must hold numbers
#pragma unroll
        for (int n = 0; n < (4 * D + TPB - 1) / TPB * 2; ++n)
            if (tid + n * TPB < 8 * D)
                *reinterpret_cast<u4*>(lds + 3 * KB + 16 * (tid + n * TPB)) = u4{0, 0, 0, 0};
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int i = 0; i < 8; ++i) pf[g][i] = static_cast<_Float16>(0.f);
        en2 = en1;
        en1 = en0;
        ahead(-1);
    }
    __syncthreads();
    if (grp) __syncthreads();
    for (int t = 0; t < steps; ++t) {
        products(t, true);
        scales(t);
        __syncthreads();
        ahead(t);
        softmax(t);
        __syncthreads();
    }
    if (steps > 0) products(steps, false);
    if (!grp) __syncthreads();

    l += lane_xor<32>(l);
    const float vo = l < kOnlyZeros ? vr : 0.f;
    if (rw + c >= rows) return;
    // element i of tile d is dimension 32 (half ND + d) + 8 (i / 4) + 4 hf + i % 4 of query c
    const int d0 = 32 * ND * half + 4 * hf;
    const int64_t at = part_of(row, rw + c - r0);
    if (at < 0) {
        const float inv = l > 0.f ? vo / l : 0.f;
        char* dst = static_cast<char*>(p.out) + (row.token * p.ldo + static_cast<int64_t>(row.head) * D + d0) * 2;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
                uint2 w;
                if constexpr (DT == BF16) {
                    w.x = pk_bf16(o[d][i] * inv, o[d][i + 1] * inv);
                    w.y = pk_bf16(o[d][i + 2] * inv, o[d][i + 3] * inv);
                } else {
                    w.x = f32_to_f16_bits(o[d][i] * inv) | static_cast<uint32_t>(f32_to_f16_bits(o[d][i + 1] * inv)) << 16;
                    w.y = f32_to_f16_bits(o[d][i + 2] * inv) | static_cast<uint32_t>(f32_to_f16_bits(o[d][i + 3] * inv)) << 16;
                }
                *reinterpret_cast<uint2*>(dst + (32 * d + 2 * i) * 2) = w;
            }
    } else {
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int i = 0; i < 16; i += 4)
                *reinterpret_cast<float4*>(p.part_o + at * D + 32 * d + 2 * i + d0) =
                    make_float4(o[d][i] * vo, o[d][i + 1] * vo, o[d][i + 2] * vo, o[d][i + 3] * vo);
        if (hf == 0 && half == 0) {
            p.part_ml[2 * at] = m;
            p.part_ml[2 * at + 1] = l;
        }
    }
}

template <int DT, int D, bool CAP>
__global__ __launch_bounds__(512, 2) void kv_attn_phase_kernel(AttnParams p) {
    extern __shared__ __attribute__((aligned(16))) char lds[];
    int64_t u = blockIdx.x;
    const int h = static_cast<int>(u % p.heads);
    u /= p.heads;
    const int sp = static_cast<int>(u % p.splits);
    u /= p.splits;
    const int b = static_cast<int>(u % p.ix.batch);
    const int rt = p.row_tiles - 1 - static_cast<int>(u / p.ix.batch);   // the longest first
    const KvSeq s = kv_seq(p.ix, b);
    const int rows = s.n * p.group, r0 = rt * kPhaseRows<D>;
    if (r0 >= rows) return;
    const int last = (r0 + kPhaseRows<D> < rows ? r0 + kPhaseRows<D> : rows) - 1;
    const int vis_hi = row_of<false>(p, s, b, h, last).vis;
    const int k0 = sp * p.split_keys;
    if (sp > 0 && k0 >= vis_hi) return;
    const int k1 = k0 + p.split_keys < vis_hi ? k0 + p.split_keys : vis_hi;
    phase_unit<DT, D, CAP, false>(p, lds, s, b, h, r0, k0, k1, [&](const Row& row, int) -> int64_t {
        if (p.splits == 1) return -1;
        return (static_cast<int64_t>(sp) * p.ix.batch * p.ix.max_q + row.slot) * p.heads_q + row.head;
    });
}

// Joins the splits of each (token, head).  GROUPS == 1: D / 8 lanes to each, the
// splits in turn (few of them: their loads go out together).  Else a block to
// each, its lanes in GROUPS groups that share the splits and meet in LDS (64
// splits of one token's 32 heads: 5.5 us, one group 23 us; 4 splits: 5.6 and 3.4).
template <int DT, int D, int GROUPS>
__global__ __launch_bounds__(256) void kv_attn_join_kernel(AttnParams p) {
    constexpr int LANES = D / 8;
    __shared__ float lo[GROUPS][D + 8], lm[GROUPS], ll[GROUPS];
    const int64_t u = GROUPS > 1 ? blockIdx.x : (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) / LANES;
    const int64_t slot = u / p.heads_q;
    const int head = static_cast<int>(u % p.heads_q);
    const int b = static_cast<int>(slot / p.ix.max_q), i = static_cast<int>(slot % p.ix.max_q);
    if (b >= p.ix.batch) return;
    const KvSeq s = kv_seq(p.ix, b);
    if (i >= s.n) return;
    const int vis = p.mask ? s.kv : kv_visible(p.ix, s, b, s.first + i);
    const int grp = GROUPS > 1 ? threadIdx.x / LANES : 0, d = threadIdx.x % LANES * 8;
    const int used = vis > 0 ? (vis - 1) / p.split_keys + 1 : 0;
    float m = kNegInf, sum = 0.f, f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    auto add = [&](float ms, float ls, const float* v) {
        const float mn = fmaxf(m, ms), base = mn > kNegInf ? mn : 0.f;
        const float a = __builtin_amdgcn_exp2f(m - base), c = __builtin_amdgcn_exp2f(ms - base);
        sum = sum * a + ls * c;
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = f[e] * a + v[e] * c;
        m = mn;
    };
#pragma unroll 4
    for (int sp = grp; sp < used; sp += GROUPS) {
        const int64_t at = (static_cast<int64_t>(sp) * p.ix.batch * p.ix.max_q + slot) * p.heads_q + head;
        const float ms = p.part_ml[2 * at], ls = p.part_ml[2 * at + 1];
        float v[8];
        load8<F32>(p.part_o + at * D + d, v);
        add(ms, ls, v);
    }
    if (GROUPS > 1) {                         // groups past `used` hold nothing
        store8<F32>(&lo[grp][d], f);
        if (d == 0) {
            lm[grp] = m;
            ll[grp] = sum;
        }
        __syncthreads();
        if (grp > 0) return;
        const int groups = used < GROUPS ? used : GROUPS;
        for (int g = 1; g < groups; ++g) {
            float v[8];
            load8<F32>(&lo[g][d], v);
            add(lm[g], ll[g], v);
        }
    }
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] *= inv;
    store8<DT>(static_cast<char*>(p.out) + ((s.row0 + i) * p.ldo + static_cast<int64_t>(head) * D + d) * 2, f);
}

// The arguments of a call with its plan.
inline AttnParams attn_params(const KvAttnPlan& plan, const void* q, int64_t ldq, int heads_q, const KvIndex& ix,
                              const int8_t* k, const int8_t* v, const float* ks, const float* vs, int heads, int d,
                              float sm_scale, float cap, const uint32_t* mask, int64_t mask_ld, void* out, int64_t ldo,
                              void* ws) {
    AttnParams p{ix, q, ldq, k, v, ks, vs, out, ldo, heads_q, heads, heads_q / heads, sm_scale, cap, plan.row_tiles,
                 plan.splits, plan.split_keys, nullptr, nullptr, mask, mask_ld, 0, nullptr};
    if (plan.splits > 1) {
        p.part_o = static_cast<float*>(ws);
        p.part_ml = p.part_o + static_cast<int64_t>(plan.splits) * ix.batch * ix.max_q * heads_q * d;
    }
    return p;
}

inline hipError_t launch_lds(void (*kernel)(AttnParams), int64_t blocks, int threads, int lds, const AttnParams& p,
                      hipStream_t st) {
    if (lds > 65536) {   // a launch's default limit
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, lds);
        if (e != hipSuccess) return e;
    }
    kernel<<<dim3(static_cast<unsigned>(blocks)), threads, lds, st>>>(p);
    return hipGetLastError();
}

template <int DT, int D>
hipError_t launch_join(const AttnParams& p, hipStream_t st) {
    if (p.splits == 1) return hipSuccess;
    const int64_t rows = static_cast<int64_t>(p.ix.batch) * p.ix.max_q * p.heads_q;
    if (p.splits > 8)
        kv_attn_join_kernel<DT, D, 2048 / D><<<dim3(static_cast<unsigned>(rows)), 256, 0, st>>>(p);
    else
        kv_attn_join_kernel<DT, D, 1><<<dim3(static_cast<unsigned>((rows * (D / 8) + 255) / 256)), 256, 0, st>>>(p);
    return hipGetLastError();
}

}  // namespace

}  // namespace qlin
