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
// that maximum.  Scores, statistics and sums are fp32.
// A weight is rounded to fp16 after multiplication by its page's v scale over vr,
// the largest met so far (in the exponent, as s_ij + log2(vs_j / vr)), and the
// maximum m is that of these exponents: the largest contribution to a row has a
// weight of 1 whatever the pages' scales, so each is rounded by 2^-11 of itself
// or 2^-25 of the largest.  The sum of the weights takes the scale out again.

#include "kv_attn.h"

namespace qlin {

namespace {

// Up to 16 query rows of one (sequence, kv head) against a range of its keys:
// four waves take the range's 64-key steps in turn, codes straight from memory
// (the next step's are on their way as soon as this one's are used), and join
// through LDS, [wave][row][D + 4] sums and then the statistics.
//
// For single tokens, bound by the cache's bytes: 64 requests of up to 4096 keys
// (32 heads over 8, 128 wide, 411 MB) take 82 us, 5.0 TB/s, the rate of a large
// copy; one request of 131101 keys (268 MB) 50 us, and 5 to join its splits.
// A short request is bound by latency (817 keys, 32 heads: 7 us and 3.5), and so
// are tens of rows: 8 x 50 rows of 8 heads over 866 keys 15 us, each 16-row block
// reading and expanding its head's keys anew (60 MB fetched for 16).
template <int DT, int D, bool CAP>
__global__ __launch_bounds__(256) void kv_attn_rows16_kernel(AttnParams p) {
    constexpr int NWV = 4;
    constexpr int NL = D / 64;     // 16-byte K loads per key row and lane
    constexpr int ND = D / 16;     // 16-dimension tiles of the output
    extern __shared__ __attribute__((aligned(16))) char lds[];
    const int rmax = p.ix.max_q * p.group < 16 ? p.ix.max_q * p.group : 16;
    float* lo = reinterpret_cast<float*>(lds);
    float* lm = lo + NWV * rmax * (D + 4);
    float* ll = lm + NWV * rmax;
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
    const int vis_hi = row_of<false>(p, s, b, h, last).vis;
    const int k0 = sp * p.split_keys;
    if (sp > 0 && k0 >= vis_hi) return;      // the join reads only the splits below the row's limit
    const int k1 = k0 + p.split_keys < vis_hi ? k0 + p.split_keys : vis_hi;

    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = lane & 15, g = lane >> 4;
    const Row row = row_of<false>(p, s, b, h, r0 + c < rows ? r0 + c : last);
    const int vis = r0 + c < rows ? row.vis : 0;
    const int ps = p.ix.page_size;

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
    // granules past the keys that the block's rows see read some page (theirs are masked)
    const uint32_t pool = static_cast<uint32_t>(p.ix.pages);
    u4 kw[4][NL], vw[ND];
    float ksc = 0.f, vsc = 0.f;
    int nk = 0, nv = 0;                      // table entries of the next step
    bool live = false, live_next = false;
    auto load_k = [&]() {
        const int8_t* kb = kh + (static_cast<uint32_t>(nk) < pool ? nk : 0) * pool_step;
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int j = 0; j < NL; ++j) kw[t][j] = *reinterpret_cast<const u4*>(kb + 4 * t * D + 64 * j);
    };
    auto load_v = [&](int t0) {
        live_next = (static_cast<uint32_t>(nv) < pool) & (t0 + 16 * g < k1);
        const int pv = live_next ? nv : 0;
        const int8_t* vb = vh + pv * pool_step;
        const int64_t sv = static_cast<int64_t>(pv) * p.heads + h;
        ksc = p.ks[sv];
        vsc = p.vs[sv];
#pragma unroll
        for (int t = 0; t < ND; ++t) vw[t] = *reinterpret_cast<const u4*>(vb + 16 * t * ps);
    };
    const int first = k0 + 64 * wave;
    if (first < k1) {
        nk = page_ahead(first, gk);
        nv = page_ahead(first, g);
        load_k();
        load_v(first);
        nk = page_ahead(first + 64 * NWV, gk);
        nv = page_ahead(first + 64 * NWV, g);
    }

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
    for (int t0 = first; t0 < k1; t0 += 64 * NWV) {
        live = live_next;
        const float ks_t = live ? ksc : 0.f, vs_t = live ? vsc : 0.f;
        const bool more = t0 + 64 * NWV < k1;

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
        if (more) load_k();
        const float mul = qmul * ks_t;
        const float vn = fmaxf(vr, groups_max(vs_t)), vlog = scale_log(vs_t, vn);
        const int lim = live ? vis - (t0 + 16 * g) : 0;      // keys of the granule that the query sees
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = i < lim ? score<CAP>(x[i], mul, cap_out, vlog) : kNegInf;

        float top = x[0];
#pragma unroll
        for (int i = 1; i < 16; ++i) top = fmaxf(top, x[i]);
        top = groups_max(top);
        // the reference follows the maximum once that is 2^8 past it (weights stay
        // far inside fp16): most steps rescale nothing
        if (__any(top > m + 8.f || vn != vr)) {
            const float ro = follow(m, l, vr, vn, top);
#pragma unroll
            for (int t = 0; t < ND; ++t) o[t] *= ro;
        }
        const float base = m > kNegInf ? m : 0.f;            // nothing seen yet: all weights 0
        h8 pf[2];
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float w = __builtin_amdgcn_exp2f(x[i] - base);
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
        if (more) {
            load_v(t0 + 64 * NWV);
            nk = page_ahead(t0 + 128 * NWV, gk);
            nv = page_ahead(t0 + 128 * NWV, g);
        }
    }

    // join the waves: element i of tile t is dimension 16 t + 4 g + i of query c
    l = groups_sum(l);
    const float vo = l < kOnlyZeros ? vr : 0.f;
    if (c < rmax) {
#pragma unroll
        for (int t = 0; t < ND; ++t)
            *reinterpret_cast<float4*>(lo + (wave * rmax + c) * (D + 4) + 16 * t + 4 * g) =
                make_float4(o[t][0] * vo, o[t][1] * vo, o[t][2] * vo, o[t][3] * vo);
        if (g == 0) {
            lm[wave * rmax + c] = m;
            ll[wave * rmax + c] = l;
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < rmax * (D / 8); e += 64 * NWV) {
        const int r = e / (D / 8), d = e % (D / 8) * 8;
        if (r0 + r >= rows) continue;
        const Row x = row_of<false>(p, s, b, h, r0 + r);
        float mt = lm[r];
#pragma unroll
        for (int w = 1; w < NWV; ++w) mt = fmaxf(mt, lm[w * rmax + r]);
        const float base = mt > kNegInf ? mt : 0.f;
        float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, sum = 0.f;
#pragma unroll
        for (int w = 0; w < NWV; ++w) {
            const float a = __builtin_amdgcn_exp2f(lm[w * rmax + r] - base);
            sum += a * ll[w * rmax + r];
            float v[8];
            load8<F32>(lo + (w * rmax + r) * (D + 4) + d, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] += a * v[i];
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

template <int DT, int D, bool CAP>
hipError_t launch_cap(const AttnParams& p, const KvAttnPlan& plan, hipStream_t st) {
    const hipError_t e =
        plan.many ? launch_lds(kv_attn_phase_kernel<DT, D, CAP>, plan.blocks, 512, 2 * 2 * 64 * D * 2, p, st)
                  : launch_lds(kv_attn_rows16_kernel<DT, D, CAP>, plan.blocks, 256, plan.lds_bytes, p, st);
    return e != hipSuccess ? e : launch_join<DT, D>(p, st);
}

template <int DT>
hipError_t launch_dt(const AttnParams& p, const KvAttnPlan& plan, int d, hipStream_t st) {
    const bool cap = p.cap > 0.f;
    if (d == 64) return cap ? launch_cap<DT, 64, true>(p, plan, st) : launch_cap<DT, 64, false>(p, plan, st);
    if (d == 128) return cap ? launch_cap<DT, 128, true>(p, plan, st) : launch_cap<DT, 128, false>(p, plan, st);
    return cap ? launch_cap<DT, 256, true>(p, plan, st) : launch_cap<DT, 256, false>(p, plan, st);
}

}  // namespace

hipError_t launch_kv_attention(const KvAttnPlan& plan, const void* q, int dtype, int64_t ldq, int heads_q,
                               const KvIndex& ix, const int8_t* k, const int8_t* v, const float* ks, const float* vs,
                               int heads, int d, float sm_scale, float cap, void* out, int64_t ldo, void* ws,
                               hipStream_t st) {
    const AttnParams p = attn_params(plan, q, ldq, heads_q, ix, k, v, ks, vs, heads, d, sm_scale, cap, nullptr, 0, out, ldo, ws);
    return dtype == F16 ? launch_dt<F16>(p, plan, d, st) : launch_dt<BF16>(p, plan, d, st);
}

}  // namespace qlin
