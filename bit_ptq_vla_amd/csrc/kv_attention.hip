// Attention over a paged int8 key/value cache with a scale per page and head,
// for gfx950.
//
//   s_ij = sm_scale q_i . (ks_j ck_j)   (capped: c tanh(s / c)),
//   out_i = sum_j exp(s_ij - m_i) vs_j cv_j / sum_j exp(s_ij - m_i)
//
// over the keys the query sees, in one pass with the running maximum m and sum.
// Everything is computed transposed, so that no value ever changes lanes:
//   S^T = K Q^T  (v_mfma_f32_16x16x32_f16: rows keys, columns queries) leaves a
//   lane with scores of ONE query, and the same registers, rounded to fp16, are
//   the B operand of O^T += V^T P^T, whose rows are head dimensions.  A lane's
//   softmax statistics, rescaling and mask limit are its own scalars.
// A step takes 64 keys, four granules of 16: lane group g = lane / 16 ends up
// with the scores of granule g (key 16 g + 4 t + i in element i of tile t).
// Rows of the K operand are permuted to make that so, and V, stored keys-first
// in its page, is then one 16-byte load per lane and 16 dimensions.  A granule
// lies in one page, so a lane needs one k scale and one v scale a step.
//
// Codes become fp16 exactly (|code| <= 127): byte + 128 under the exponent of
// 1024, minus 1152.  bf16 queries become fp16 under a power of two per row that
// brings the row's maximum to 2^13..2^14: exact but for elements 2^-27 below
// that maximum.  Scores, statistics and sums are fp32.  The weights are rounded
// to fp16 after multiplication by vs_j / vr, vr the largest v scale met so far
// (in the exponent; no page overflows them): 2^-11 each at most.

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
    float* part_o;     // [splits][batch * max_q][heads_q][D]
    float* part_ml;    // [splits][batch * max_q][heads_q][2]
};

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNegInf = -__builtin_inff();

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

// A score in base-2 units from the raw product: capped where CAP.
template <bool CAP>
__device__ __forceinline__ float score(float raw, float mul, float cap_in, float cap_out) {
    if constexpr (CAP) {
        // c tanh(x / c) = c (1 - 2 / (1 + exp(2 x / c))): mul holds 2 / c * log2 e, cap_out c log2 e
        const float e = __builtin_amdgcn_exp2f(raw * mul);
        return cap_out - 2.f * cap_out * __builtin_amdgcn_rcpf(1.f + e);
    } else {
        return raw * mul;
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

__device__ __forceinline__ Row row_of(const AttnParams& p, const KvSeq& s, int b, int h, int r) {
    Row x;
    const int i = r / p.group;
    x.ok = i < s.n;
    const int ii = x.ok ? i : 0;
    x.token = s.row0 + ii;
    x.slot = static_cast<int64_t>(b) * p.ix.max_q + ii;
    x.head = h * p.group + r % p.group;
    x.vis = x.ok ? kv_visible(p.ix, s, b, s.first + i) : 0;
    return x;
}

// Up to 16 query rows of one (sequence, kv head) against a range of its keys:
// four waves take the range's 64-key steps in turn and join through LDS.
template <int DT, int D, bool CAP>
__global__ __launch_bounds__(256) void kv_attn_rows16_kernel(AttnParams p) {
    constexpr int NL = D / 64;     // 16-byte K loads per key row and lane
    constexpr int ND = D / 16;     // 16-dimension tiles of the output
    __shared__ float lo[4][16][D + 4];
    __shared__ float lm[4][16], ll[4][16];
    int64_t u = blockIdx.x;
    const int sp = static_cast<int>(u % p.splits);
    u /= p.splits;
    const int rt = static_cast<int>(u % p.row_tiles);
    u /= p.row_tiles;
    const int h = static_cast<int>(u % p.heads);
    const int b = static_cast<int>(u / p.heads);
    const KvSeq s = kv_seq(p.ix, b);
    const int rows = s.n * p.group, r0 = rt * 16;
    if (r0 >= rows) return;
    const int last = (r0 + 16 < rows ? r0 + 16 : rows) - 1;
    const int vis_hi = row_of(p, s, b, h, last).vis, vis_lo = row_of(p, s, b, h, r0).vis;
    const int k0 = sp * p.split_keys;
    if (sp > 0 && k0 >= vis_hi) return;      // the join reads only the splits below the row's limit
    const int k1 = k0 + p.split_keys < vis_hi ? k0 + p.split_keys : vis_hi;

    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = lane & 15, g = lane >> 4;
    const Row row = row_of(p, s, b, h, r0 + c < rows ? r0 + c : last);
    const int vis = r0 + c < rows ? row.vis : 0;
    const int ps = p.ix.page_size;

    // the lane's part of its query: dimensions 64 j + 16 g .. + 15
    h8 qf[2 * NL];
    float qmul = p.sm_scale;
    {
        const char* src = static_cast<const char*>(p.q) + (row.token * p.ldq + static_cast<int64_t>(row.head) * D) * 2;
        float f[2 * NL][8];
        float top = 0.f;
#pragma unroll
        for (int j = 0; j < NL; ++j) {
            load8<DT>(src + (64 * j + 16 * g) * 2, f[2 * j]);
            load8<DT>(src + (64 * j + 16 * g + 8) * 2, f[2 * j + 1]);
        }
        int e = 0;
        if constexpr (DT == BF16) {
#pragma unroll
            for (int j = 0; j < 2 * NL; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(f[j][i]));
            top = groups_max(top);
            if (top > 0.f && top < __builtin_inff()) e = 14 - __builtin_amdgcn_frexp_expf(top);
            e = e > 120 ? 120 : e < -120 ? -120 : e;
            qmul = __builtin_amdgcn_ldexpf(p.sm_scale, -e);
        }
#pragma unroll
        for (int j = 0; j < 2 * NL; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                qf[j][i] = static_cast<_Float16>(DT == BF16 ? __builtin_amdgcn_ldexpf(f[j][i], e) : f[j][i]);
    }
    qmul *= CAP ? 2.f * kLog2e / p.cap : kLog2e;
    const float cap_out = CAP ? p.cap * kLog2e : 0.f;

    f4 o[ND];
#pragma unroll
    for (int t = 0; t < ND; ++t) o[t] = f4{0.f, 0.f, 0.f, 0.f};
    float m = kNegInf, l = 0.f, vr = 0.f;
    const int psl = 31 - __builtin_clz(ps);
    const int last_idx = s.kv > 0 ? (s.kv - 1) >> psl : 0;
    const int gk = c >> 2;                   // granule of the lane's K rows
    const int32_t* table = p.ix.page_table + static_cast<int64_t>(b) * p.ix.table_ld;
    const int64_t page_bytes = static_cast<int64_t>(ps) * D, pool_step = page_bytes * p.heads;
    // t0 is a multiple of 64: a granule's place in its page does not depend on it
    const int8_t* kh = p.k + h * page_bytes + (((16 * gk) & (ps - 1)) + (c & 3)) * D + 16 * g;
    const int8_t* vh = p.v + h * page_bytes + c * ps + ((16 * g) & (ps - 1));
    auto page_ahead = [&](int t0, int gran) {
        const int idx = (t0 + 16 * gran) >> psl;
        return table[idx < last_idx ? idx : last_idx];
    };
    // granules past the cache read its last page (their keys are masked)
    int nk = 0, nv = 0;
    if (k0 + 64 * wave < k1) {
        nk = page_ahead(k0 + 64 * wave, gk);
        nv = page_ahead(k0 + 64 * wave, g);
    }

    for (int t0 = k0 + 64 * wave; t0 < k1; t0 += 256) {
        const bool live = nv >= 0 && nv < p.ix.pages && t0 + 16 * g < s.kv;
        const int pk = nk >= 0 && nk < p.ix.pages ? nk : 0, pv = live ? nv : 0;
        const int8_t* kb = kh + pk * pool_step;
        const int8_t* vb = vh + pv * pool_step;
        u4 kw[4][NL], vw[ND];
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int j = 0; j < NL; ++j) kw[t][j] = *reinterpret_cast<const u4*>(kb + 4 * t * D + 64 * j);
        const int64_t sv = static_cast<int64_t>(pv) * p.heads + h;
        float ksc = p.ks[sv], vsc = p.vs[sv];
#pragma unroll
        for (int t = 0; t < ND; ++t) vw[t] = *reinterpret_cast<const u4*>(vb + 16 * t * ps);
        nk = page_ahead(t0 + 256, gk);
        nv = page_ahead(t0 + 256, g);
        if (!live) ksc = vsc = 0.f;

        float x[16];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            f4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < NL; ++j) {
                const u4 w = kw[t][j];
                acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(codes_f16(w[0], w[1]), qf[2 * j], acc, 0, 0, 0);
                acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(codes_f16(w[2], w[3]), qf[2 * j + 1], acc, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) x[4 * t + i] = acc[i];
        }
        const float mul = qmul * ksc;
        const int lim = live ? vis - (t0 + 16 * g) : 0;      // keys of the granule that the query sees
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = i < lim ? score<CAP>(x[i], mul, 0.f, cap_out) : kNegInf;

        float top = x[0];
#pragma unroll
        for (int i = 1; i < 16; ++i) top = fmaxf(top, x[i]);
        top = groups_max(top);
        const float vn = fmaxf(vr, groups_max(vsc));
        // the reference follows the maximum once that is 2^8 past it (weights stay
        // far inside fp16): most steps rescale nothing
        if (__any(top > m + 8.f || vn != vr)) {
            const float mn = fmaxf(m, top);
            const float r = m > kNegInf ? __builtin_amdgcn_exp2f(m - mn) : 1.f;
            const float ro = r * (vr > 0.f ? vr / vn : 1.f);
#pragma unroll
            for (int t = 0; t < ND; ++t) o[t] *= ro;
            l *= r;
            m = mn;
            vr = vn;
        }
        // weights times the page's v scale over the largest (at least 2^-30 of it:
        // below, they leave fp16 anyway); the sum takes that out again
        const float base = m > kNegInf ? m : 0.f;            // nothing seen yet: all weights 0
        const float vlog = fmaxf(__builtin_amdgcn_logf(vsc) - __builtin_amdgcn_logf(vr), -30.f);
        const float off = vlog - base;
        h8 pf[2];
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float w = __builtin_amdgcn_exp2f(x[i] + off);
            sum += w;
            pf[i >> 3][i & 7] = static_cast<_Float16>(w);
        }
        l = fmaf(sum, __builtin_amdgcn_exp2f(-vlog), l);
#pragma unroll
        for (int t = 0; t < ND; ++t) {
            const u4 w = vw[t];
            o[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(codes_f16(w[0], w[1]), pf[0], o[t], 0, 0, 0);
            o[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(codes_f16(w[2], w[3]), pf[1], o[t], 0, 0, 0);
        }
    }

    // join the waves: element i of tile t is dimension 16 t + 4 g + i of query c
    l = groups_sum(l);
#pragma unroll
    for (int t = 0; t < ND; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) lo[wave][c][16 * t + 4 * g + i] = o[t][i] * vr;
    if (g == 0) {
        lm[wave][c] = m;
        ll[wave][c] = l;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < 16 * (D / 8); e += 256) {
        const int r = e / (D / 8), d = e % (D / 8) * 8;
        if (r0 + r >= rows) continue;
        const Row x = row_of(p, s, b, h, r0 + r);
        float mt = lm[0][r];
#pragma unroll
        for (int w = 1; w < 4; ++w) mt = fmaxf(mt, lm[w][r]);
        const float base = mt > kNegInf ? mt : 0.f;
        float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, sum = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float a = __builtin_amdgcn_exp2f(lm[w][r] - base);
            sum += a * ll[w][r];
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] += a * lo[w][r][d + i];
        }
        if (p.splits == 1) {
            const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] *= inv;
            store8<DT>(static_cast<char*>(p.out) + (x.token * p.ldo + static_cast<int64_t>(x.head) * D + d) * 2, f);
        } else {
            const int64_t at = ((static_cast<int64_t>(sp) * p.ix.batch * p.ix.max_q + x.slot) * p.heads_q + x.head);
            store8<F32>(p.part_o + at * D + d, f);
            if (d == 0) {
                p.part_ml[2 * at] = mt;
                p.part_ml[2 * at + 1] = sum;
            }
        }
    }
}

// ---- many query rows ---------------------------------------------------------

// Byte offset of 16-byte chunk `c` of K row `row` in LDS: D fp16 a row, chunks
// xor-swizzled so that eight lanes reading one chunk of eight rows meet eight
// different bank groups.
template <int D>
__device__ __forceinline__ int k_off(int row, int c) {
    constexpr int M = D / 8 < 16 ? D / 8 - 1 : 15;
    return row * D * 2 + ((c ^ (row & M)) << 4);
}
// The same for V: 64 keys (8 chunks) a dimension.
__device__ __forceinline__ int v_off(int d, int c) { return d * 128 + ((c ^ (d & 7)) << 4); }

// The LDS row of key j (0..63) of a step.  The 32x32 product leaves lane half h
// with rows 8 (i / 4) + 4 h + i % 4 in element i; with this order elements
// 8 u .. 8 u + 7 of a lane are keys 16 u + 8 h + (0..7): B operand u of P^T as
// it stands, against V in its stored order.
__device__ __forceinline__ int key_row(int j) {
    return (j & 48) | ((j & 4) << 1) | ((j & 8) >> 1) | (j & 3);
}

// 32 * NW query rows of one (sequence, kv head), 32 to a wave, against a range
// of its keys.  The block turns each step's 64 keys into fp16 in LDS once (v
// times its page's scale over the largest met) and every wave multiplies
// v_mfma_f32_32x32x16_f16 tiles from there; the next step's codes are in
// flight meanwhile, and two LDS buffers leave one barrier a step.
template <int DT, int D, bool CAP, int NW>
__global__ __launch_bounds__(64 * NW, D == 256 ? 1 : 2) void kv_attn_tile_kernel(AttnParams p) {
    constexpr int TPB = 64 * NW;
    constexpr int NS = D / 16;            // k steps of S
    constexpr int ND = D / 32;            // 32-dimension tiles of the output
    constexpr int NC = D * 4 / TPB;       // 16-byte pieces of k (and of v) a thread stages per step
    constexpr int KB = 64 * D * 2;        // bytes of one operand of a step in LDS
    extern __shared__ __attribute__((aligned(16))) char lds[];
    typedef float f16v __attribute__((ext_vector_type(16)));

    int64_t u = blockIdx.x;
    const int h = static_cast<int>(u % p.heads);
    u /= p.heads;
    const int sp = static_cast<int>(u % p.splits);
    u /= p.splits;
    const int b = static_cast<int>(u % p.ix.batch);
    const int rt = p.row_tiles - 1 - static_cast<int>(u / p.ix.batch);   // the longest first
    const KvSeq s = kv_seq(p.ix, b);
    const int rows = s.n * p.group, r0 = rt * 32 * NW;
    if (r0 >= rows) return;
    const int last = (r0 + 32 * NW < rows ? r0 + 32 * NW : rows) - 1;
    const int vis_hi = row_of(p, s, b, h, last).vis;
    const int k0 = sp * p.split_keys;
    if (sp > 0 && k0 >= vis_hi) return;
    const int k1 = k0 + p.split_keys < vis_hi ? k0 + p.split_keys : vis_hi;

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int c = lane & 31, hf = lane >> 5;
    const int rw = r0 + 32 * wave;                       // the wave's first row
    const Row row = row_of(p, s, b, h, rw + c < rows ? rw + c : last);
    const int vis = rw + c < rows ? row.vis : 0;
    // the wave's rows see at least / at most these keys
    const int wave_lo = rw + 31 < rows ? row_of(p, s, b, h, rw).vis : 0;
    const int wave_hi = rw < rows ? row_of(p, s, b, h, rw + 31 < rows ? rw + 31 : last).vis : 0;
    const int ps = p.ix.page_size, psl = 31 - __builtin_clz(ps);
    const int last_idx = s.kv > 0 ? (s.kv - 1) >> psl : 0;

    // queries: dimensions 16 s + 8 hf .. + 7 of row c
    h8 qf[NS];
    float qmul = p.sm_scale;
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
            qmul = __builtin_amdgcn_ldexpf(p.sm_scale, -e);
        }
#pragma unroll
        for (int j = 0; j < NS; ++j) {
            float f[8];
            load8<DT>(src + (16 * j + 8 * hf) * 2, f);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                qf[j][i] = static_cast<_Float16>(DT == BF16 ? __builtin_amdgcn_ldexpf(f[i], e) : f[i]);
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

    // A step's codes on their way.  Lane x of each four holds what belongs to the
    // step's granule x: its page (read one step ahead of the codes), scales and
    // whether it has keys; a piece of v lies in the granule of its own lane, a
    // piece of k in one that the whole wave shares.
    u4 kw[NC], vw[NC];
    const int x4 = lane & 3;
    const int32_t* table = p.ix.page_table + static_cast<int64_t>(b) * p.ix.table_ld;
    const int64_t page_bytes = static_cast<int64_t>(ps) * D, pool_step = page_bytes * p.heads;
    const int8_t* kh = p.k + h * page_bytes;
    const int8_t* vh = p.v + h * page_bytes;
    int kat[NC], vat[NC], kg[NC], krow[NC];
#pragma unroll
    for (int n = 0; n < NC; ++n) {
        const int i = tid + n * TPB, key = i / (D / 16), kc = i % (D / 16), vd = i >> 2;
        kat[n] = (key & (ps - 1)) * D + 16 * kc;
        vat[n] = vd * ps + ((16 * x4) & (ps - 1));
        kg[n] = __builtin_amdgcn_readfirstlane(key >> 4);
        krow[n] = key_row(key);
    }
    auto page_ahead = [&](int t0) {
        const int idx = (t0 + 16 * x4) >> psl;
        return table[idx < last_idx ? idx : last_idx];
    };
    int ahead = 0, dead_next = 0;
    float ks_next = 0.f, vs_next = 0.f;
    auto fetch = [&](int t0) {
        const bool live = ahead >= 0 && ahead < p.ix.pages && t0 + 16 * x4 < s.kv;
        const int page = live ? ahead : 0;
        dead_next = static_cast<int>(__ballot(!live)) & 15;
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            const int64_t pk = __builtin_amdgcn_readlane(page, kg[n]);
            kw[n] = *reinterpret_cast<const u4*>(kh + pk * pool_step + kat[n]);
        }
        const int8_t* vp = vh + page * pool_step;
#pragma unroll
        for (int n = 0; n < NC; ++n) vw[n] = *reinterpret_cast<const u4*>(vp + vat[n]);
        const int64_t at = static_cast<int64_t>(page) * p.heads + h;
        ks_next = p.ks[at];
        vs_next = p.vs[at];
        if (!live) ks_next = vs_next = 0.f;
        ahead = page_ahead(t0 + 64);
    };
    // the fetched step into buffer `buf`, and its granules' scales and flags
    float mul[4], unit = 0.f, vlog[4], vinv[4];
    int dead = 0;
    auto stage = [&](int buf) {
        char* kl = lds + buf * 2 * KB;
        char* vl = kl + KB;
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            const int i = tid + n * TPB;
            const int kc = i % (D / 16), vd = i >> 2;
            *reinterpret_cast<h8*>(kl + k_off<D>(krow[n], 2 * kc)) = codes_f16(kw[n][0], kw[n][1]);
            *reinterpret_cast<h8*>(kl + k_off<D>(krow[n], 2 * kc + 1)) = codes_f16(kw[n][2], kw[n][3]);
            *reinterpret_cast<h8*>(vl + v_off(vd, 2 * x4)) = codes_f16(vw[n][0], vw[n][1]);
            *reinterpret_cast<h8*>(vl + v_off(vd, 2 * x4 + 1)) = codes_f16(vw[n][2], vw[n][3]);
        }
        float top = fmaxf(vs_next, dpp_mov<0xB1>(vs_next));
        top = fmaxf(top, dpp_mov<0x4E>(top));
        unit = fmaxf(unit, top);
        // a page 2^-30 below the largest keeps that ratio: its weights leave fp16
        // there anyway (and a NaN, all scales 0, becomes it too)
        const float lg = fmaxf(__builtin_amdgcn_logf(vs_next) - __builtin_amdgcn_logf(unit), -30.f);
        const float li = __builtin_amdgcn_exp2f(-lg);
        dead = dead_next;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            mul[x] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(ks_next), x));
            vlog[x] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(lg), x));
            vinv[x] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(li), x));
        }
        unit = __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(unit)));
    };

    int buf = 0;
    if (k0 < k1) {
        ahead = page_ahead(k0);
        fetch(k0);
        stage(0);
    }
    __syncthreads();
    for (int t0 = k0; t0 < k1; t0 += 64, buf ^= 1) {
        const bool more = t0 + 64 < k1;
        if (more) fetch(t0 + 64);
        if (t0 < wave_hi) {
            const char* kl = lds + buf * 2 * KB;
            const char* vl = kl + KB;
            float x[32];
#pragma unroll
            for (int T = 0; T < 2; ++T) {
                f16v acc;
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[i] = 0.f;
#pragma unroll
                for (int j = 0; j < NS; ++j)
                    acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(
                        *reinterpret_cast<const h8*>(kl + k_off<D>(32 * T + c, 2 * j + hf)), qf[j], acc, 0, 0, 0);
#pragma unroll
                for (int i = 0; i < 16; ++i) x[16 * T + i] = acc[i];
            }
            // element 8 g + e is key 16 g + 8 hf + e of the step
            if (CAP) {
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = score<CAP>(x[i], qmul * mul[i >> 3], 0.f, cap_out);
            }
            const bool whole = t0 + 64 <= wave_lo && dead == 0;
            float top = kNegInf;
            float sc[4];
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                sc[g] = CAP ? 1.f : qmul * mul[g];
                if (!whole) {
                    const int lim = (dead >> g & 1) ? 0 : vis - (t0 + 16 * g + 8 * hf);
                    // masked scores leave as the value that scales to -inf (a zero scale: all scores 0)
                    const float out = sc[g] < 0.f ? -kNegInf : kNegInf;
                    const bool zero = sc[g] == 0.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[8 * g + e] = e < lim ? (zero ? 0.f : x[8 * g + e]) : out;
                    if (zero) sc[g] = 1.f;
                }
                float hi = x[8 * g];
                if (!CAP && p.sm_scale < 0.f) {
#pragma unroll
                    for (int e = 1; e < 8; ++e) hi = fminf(hi, x[8 * g + e]);
                } else {
#pragma unroll
                    for (int e = 1; e < 8; ++e) hi = fmaxf(hi, x[8 * g + e]);
                }
                top = fmaxf(top, hi * sc[g]);
            }
            top = fmaxf(top, lane_xor<32>(top));
            // the reference follows the maximum once that is 2^8 past it: weights stay
            // below 2^8, far inside fp16, and most steps rescale nothing
            if (__any(top > m + 8.f || unit != vr)) {
                const float mn = fmaxf(m, top);
                const float r = m > kNegInf ? __builtin_amdgcn_exp2f(m - mn) : 1.f;
                const float ro = r * (vr > 0.f ? vr / unit : 1.f);
#pragma unroll
                for (int t = 0; t < ND; ++t)
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[t][i] *= ro;
                l *= r;
                m = mn;
                vr = unit;
            }
            const float base = m > kNegInf ? m : 0.f;        // nothing seen yet: all weights 0
            h8 pf[4];
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                // weights times the page's v scale over the unit; the sum takes that out again
                const float off = vlog[g] - base;
                float sum = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float w = __builtin_amdgcn_exp2f(fmaf(x[8 * g + e], sc[g], off));
                    sum += w;
                    pf[g][e] = static_cast<_Float16>(w);
                }
                l = fmaf(sum, vinv[g], l);
            }
#pragma unroll
            for (int t = 0; t < ND; ++t)
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    o[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
                        *reinterpret_cast<const h8*>(vl + v_off(32 * t + c, 2 * g + hf)), pf[g], o[t], 0, 0, 0);
        }
        if (more) stage(buf ^ 1);
        __syncthreads();
    }

    l += lane_xor<32>(l);
    if (rw + c >= rows) return;
    // element i of tile t is dimension 32 t + 8 (i / 4) + 4 hf + i % 4 of query c
    if (p.splits == 1) {
        const float inv = l > 0.f ? vr / l : 0.f;
        char* dst = static_cast<char*>(p.out) + (row.token * p.ldo + static_cast<int64_t>(row.head) * D + 4 * hf) * 2;
#pragma unroll
        for (int t = 0; t < ND; ++t)
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
                uint2 w;
                if constexpr (DT == BF16) {
                    w.x = pk_bf16(o[t][i] * inv, o[t][i + 1] * inv);
                    w.y = pk_bf16(o[t][i + 2] * inv, o[t][i + 3] * inv);
                } else {
                    w.x = f32_to_f16_bits(o[t][i] * inv) | static_cast<uint32_t>(f32_to_f16_bits(o[t][i + 1] * inv)) << 16;
                    w.y = f32_to_f16_bits(o[t][i + 2] * inv) | static_cast<uint32_t>(f32_to_f16_bits(o[t][i + 3] * inv)) << 16;
                }
                *reinterpret_cast<uint2*>(dst + (32 * t + 2 * i) * 2) = w;
            }
    } else {
        const int64_t at = ((static_cast<int64_t>(sp) * p.ix.batch * p.ix.max_q + row.slot) * p.heads_q + row.head);
#pragma unroll
        for (int t = 0; t < ND; ++t)
#pragma unroll
            for (int i = 0; i < 16; i += 4)
                *reinterpret_cast<float4*>(p.part_o + at * D + 32 * t + 2 * i + 4 * hf) =
                    make_float4(o[t][i] * vr, o[t][i + 1] * vr, o[t][i + 2] * vr, o[t][i + 3] * vr);
        if (hf == 0) {
            p.part_ml[2 * at] = m;
            p.part_ml[2 * at + 1] = l;
        }
    }
}

// Joins the splits of every (token, head): D / 8 lanes each.
template <int DT, int D>
__global__ __launch_bounds__(256) void kv_attn_join_kernel(AttnParams p) {
    const int64_t u = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) / (D / 8);
    const int d = threadIdx.x % (D / 8) * 8;
    const int64_t slot = u / p.heads_q;
    const int head = static_cast<int>(u % p.heads_q);
    const int b = static_cast<int>(slot / p.ix.max_q), i = static_cast<int>(slot % p.ix.max_q);
    if (b >= p.ix.batch) return;
    const KvSeq s = kv_seq(p.ix, b);
    if (i >= s.n) return;
    const int vis = kv_visible(p.ix, s, b, s.first + i);
    float m = kNegInf, sum = 0.f, f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int sp = 0; sp < p.splits && sp * p.split_keys < vis; ++sp) {
        const int64_t at = (static_cast<int64_t>(sp) * p.ix.batch * p.ix.max_q + slot) * p.heads_q + head;
        const float ms = p.part_ml[2 * at], ls = p.part_ml[2 * at + 1];
        float v[8];
        load8<F32>(p.part_o + at * D + d, v);
        const float mn = fmaxf(m, ms), base = mn > kNegInf ? mn : 0.f;
        const float a = __builtin_amdgcn_exp2f(m - base), c = __builtin_amdgcn_exp2f(ms - base);
        sum = sum * a + ls * c;
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = f[e] * a + v[e] * c;
        m = mn;
    }
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] *= inv;
    store8<DT>(static_cast<char*>(p.out) + ((s.row0 + i) * p.ldo + static_cast<int64_t>(head) * D + d) * 2, f);
}

template <int DT, int D>
hipError_t launch_d(const AttnParams& p, bool tile, hipStream_t st) {
    const int64_t blocks = static_cast<int64_t>(p.ix.batch) * p.heads * p.row_tiles * p.splits;
    if (tile) {
        constexpr int bytes = 2 * 2 * 64 * D * 2;
        auto kernel = p.cap > 0.f ? kv_attn_tile_kernel<DT, D, true, 4> : kv_attn_tile_kernel<DT, D, false, 4>;
        if (bytes > 65536) {
            const hipError_t a = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                                     hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
            if (a != hipSuccess) return a;
        }
        kernel<<<dim3(static_cast<unsigned>(blocks)), 256, bytes, st>>>(p);
    } else if (p.cap > 0.f)
        kv_attn_rows16_kernel<DT, D, true><<<dim3(static_cast<unsigned>(blocks)), 256, 0, st>>>(p);
    else
        kv_attn_rows16_kernel<DT, D, false><<<dim3(static_cast<unsigned>(blocks)), 256, 0, st>>>(p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.splits == 1) return e;
    const int64_t lanes = static_cast<int64_t>(p.ix.batch) * p.ix.max_q * p.heads_q * (D / 8);
    kv_attn_join_kernel<DT, D><<<dim3(static_cast<unsigned>((lanes + 255) / 256)), 256, 0, st>>>(p);
    return hipGetLastError();
}

template <int DT>
hipError_t launch_dt(const AttnParams& p, int d, bool tile, hipStream_t st) {
    if (d == 64) return launch_d<DT, 64>(p, tile, st);
    if (d == 128) return launch_d<DT, 128>(p, tile, st);
    return launch_d<DT, 256>(p, tile, st);
}

}  // namespace

hipError_t launch_kv_attention(const KvAttnPlan& plan, const void* q, int dtype, int64_t ldq, int heads_q,
                               const KvIndex& ix, const int8_t* k, const int8_t* v, const float* ks, const float* vs,
                               int heads, int d, float sm_scale, float cap, void* out, int64_t ldo, void* ws,
                               hipStream_t st) {
    AttnParams p{ix, q, ldq, k, v, ks, vs, out, ldo, heads_q, heads, heads_q / heads, sm_scale, cap, plan.row_tiles,
                 plan.splits, plan.split_keys, nullptr, nullptr};
    if (plan.splits > 1) {
        p.part_o = static_cast<float*>(ws);
        p.part_ml = p.part_o + static_cast<int64_t>(plan.splits) * ix.batch * ix.max_q * heads_q * d;
    }
    return dtype == F16 ? launch_dt<F16>(p, d, plan.tile, st) : launch_dt<BF16>(p, d, plan.tile, st);
}

}  // namespace qlin
