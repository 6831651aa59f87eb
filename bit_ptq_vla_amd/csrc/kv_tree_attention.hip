// Attention of a tree of drafted tokens over the paged int8 cache, for gfx950: the
// arithmetic of the attention over the cache, for rows that all see the cached keys
// and, of the new ones, those of their masks.

#include "kv_attn.h"

namespace qlin {

namespace {

// Up to 16 NQ query rows of one (sequence, kv head) against a range of its keys: four
// waves take the range's 64-key steps in turn and join through LDS, 16 rows at a time.
// A wave holds all of the rows, so that a step's codes are read and expanded to fp16
// once for NQ products with 16 queries each: expanding them (20 vector instructions to
// 16 codes) costs as much as the softmax of 16 rows.  As in that attention, a weight times
// its page's v scale is rounded to fp16 before the product with v's codes, for the matrix
// units' rate: by 2^-11 of itself, or 2^-25 of the largest in its row; the sum of the
// weights takes them unrounded, in fp32.
//
// Bound by latency where there is little (16 nodes over 816 keys of 32 heads, 7 MB: 11
// us, a join among them), by the vector units' issue where there is much: 64 trees of up
// to 16 nodes over up to 4080 keys, 8 heads of 128 for 32 (421 MB) take 127 us, 3.3 TB/s;
// a step of 32 rows and 64 keys is about 800 vector instructions, which keep the SIMDs
// 50 to 63% busy, the matrix units 15 to 20%.  Blocks of 16 rows whose row tiles did not share an L2
// took 212; a wave with 64 rows spills.
template <int DT, int D, bool CAP, int NQ>
__global__ __launch_bounds__(256, D < 256 ? 2 : 1) void kv_attn_tree_kernel(AttnParams p) {
    constexpr int NWV = 4;
    constexpr int NL = D / 64;     // 16-byte K loads per key row and lane
    constexpr int ND = D / 16;     // 16-dimension tiles of the output
    extern __shared__ __attribute__((aligned(16))) char lds[];
    constexpr int ROWS = 16 * NQ;
    const int rmax = p.ix.max_q * p.group < 16 ? p.ix.max_q * p.group : 16;
    float* lo = reinterpret_cast<float*>(lds);
    float* lm = lo + NWV * rmax * (D + 4);
    float* ll = lm + NWV * rmax;
    // Consecutive blocks go to the eight XCDs in turn, each with an L2 of its own: the
    // row tiles of a head's keys are eight blocks apart, so that one L2 serves them all.
    const int64_t units = static_cast<int64_t>(p.ix.batch) * p.heads * p.splits;
    const int rt = static_cast<int>(blockIdx.x / 8 % p.row_tiles);
    int64_t u = blockIdx.x / 8 / p.row_tiles * 8 + blockIdx.x % 8;
    if (u >= units) return;
    const int sp = static_cast<int>(u % p.splits);
    u /= p.splits;
    const int h = static_cast<int>(u % p.heads);
    const int b = static_cast<int>(u / p.heads);
    const KvSeq s = kv_seq(p.ix, b);
    const int rows = s.n * p.group, r0 = rt * ROWS;
    if (r0 >= rows) return;
    const int vis_hi = s.kv;                 // (keys behind the cached ones may be seen by any row)
    const int k0 = sp * p.split_keys;
    if (sp > 0 && k0 >= vis_hi) return;      // the join reads only the splits below the row's limit
    const int k1 = k0 + p.split_keys < vis_hi ? k0 + p.split_keys : vis_hi;

    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = lane & 15, g = lane >> 4;
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

    // the lane's part of its queries, one of each 16 rows: dimensions 64 j + 16 g .. + 15
    h8 qf[NQ][2 * NL];
    float qmul[NQ];
    const uint32_t* mask[NQ];
    bool ok[NQ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        const int r = r0 + 16 * n + c;
        const Row row = row_of<true>(p, s, b, h, r < rows ? r : rows - 1);
        ok[n] = r < rows;
        mask[n] = p.mask + row.token * p.mask_ld;
        qmul[n] = p.sm_scale;
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
            qmul[n] = __builtin_amdgcn_ldexpf(p.sm_scale, -e);
        }
#pragma unroll
        for (int j = 0; j < 2 * NL; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                qf[n][j][i] = static_cast<_Float16>(DT == BF16 ? __builtin_amdgcn_ldexpf(f[j][i], e) : f[j][i]);
        qmul[n] *= CAP ? 2.f * kLog2e / p.cap : kLog2e;
        __builtin_amdgcn_sched_barrier(0);
    }
    const float cap_out = CAP ? p.cap * kLog2e : 0.f;

    f4 o[NQ][ND];
    float m[NQ], l[NQ], vr = 0.f;
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        m[n] = kNegInf;
        l[n] = 0.f;
#pragma unroll
        for (int t = 0; t < ND; ++t) o[n][t] = f4{0.f, 0.f, 0.f, 0.f};
    }
    for (int t0 = first; t0 < k1; t0 += 64 * NWV) {
        live = live_next;
        const float ks_t = live ? ksc : 0.f, vs_t = live ? vsc : 0.f;
        const bool more = t0 + 64 * NWV < k1;

        float x[NQ][16];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            f4 acc[NQ];
#pragma unroll
            for (int n = 0; n < NQ; ++n) acc[n] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < NL; ++j) {
                const u4 w = kw[t][j];
                const h8 lo8 = codes_f16(w[0], w[1]), hi8 = codes_f16(w[2], w[3]);
#pragma unroll
                for (int n = 0; n < NQ; ++n) {
                    acc[n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(lo8, qf[n][2 * j], acc[n], 0, 0, 0);
                    acc[n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(hi8, qf[n][2 * j + 1], acc[n], 0, 0, 0);
                }
            }
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) x[n][4 * t + i] = acc[n][i];
            __builtin_amdgcn_sched_barrier(0);       // (codes are expanded as they are used: all at once would take 128 registers)
        }
        if (more) load_k();
        const float vn = fmaxf(vr, groups_max(vs_t)), vlog = scale_log(vs_t, vn), vinv = __builtin_amdgcn_exp2f(-vlog);
        // all 64 keys seen by all rows: most steps
        const bool plain = t0 + 64 <= s.first && __all(live);
        h8 pf[NQ][2];
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            const float mul = qmul[n] * ks_t;
#pragma unroll
            for (int i = 0; i < 16; ++i) x[n][i] = score<CAP>(x[n][i], mul, cap_out, vlog);
            if (!plain || !ok[n]) {
                const uint32_t bits = live && ok[n] ? kv_tree_bits(mask[n], s, t0 + 16 * g) : 0;
#pragma unroll
                for (int i = 0; i < 16; ++i) x[n][i] = bits >> i & 1 ? x[n][i] : kNegInf;
            }
            float top = x[n][0];
#pragma unroll
            for (int i = 1; i < 16; ++i) top = fmaxf(top, x[n][i]);
            top = groups_max(top);
            // the reference follows the maximum once that is 2^8 past it (weights stay
            // far inside fp16): most steps rescale nothing
            if (__any(top > m[n] + 8.f || vn != vr)) {
                float vo = vr;
                const float ro = follow(m[n], l[n], vo, vn, top);
#pragma unroll
                for (int t = 0; t < ND; ++t) o[n][t] *= ro;
            }
            const float base = m[n] > kNegInf ? m[n] : 0.f;      // nothing seen yet: all weights 0
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float w = __builtin_amdgcn_exp2f(x[n][i] - base);
                sum += w;
                pf[n][i >> 3][i & 7] = static_cast<_Float16>(w);
            }
            l[n] = fmaf(sum, vinv, l[n]);
            __builtin_amdgcn_sched_barrier(0);
        }
        vr = vn;
#pragma unroll
        for (int t = 0; t < ND; ++t) {
            const u4 w = vw[t];
            const h8 lo8 = codes_f16(w[0], w[1]), hi8 = codes_f16(w[2], w[3]);
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
                o[n][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(lo8, pf[n][0], o[n][t], 0, 0, 0);
                o[n][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(hi8, pf[n][1], o[n][t], 0, 0, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if (more) {
            load_v(t0 + 64 * NWV);
            nk = page_ahead(t0 + 128 * NWV, gk);
            nv = page_ahead(t0 + 128 * NWV, g);
        }
    }

    // join the waves: element i of tile t is dimension 16 t + 4 g + i of query c
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        const int rn = r0 + 16 * n;
        if (n > 0 && rn >= rows) break;
        if (n > 0) __syncthreads();
        const float ln = groups_sum(l[n]);
        const float vo = ln < kOnlyZeros ? vr : 0.f;
        if (c < rmax) {
#pragma unroll
            for (int t = 0; t < ND; ++t)
                *reinterpret_cast<float4*>(lo + (wave * rmax + c) * (D + 4) + 16 * t + 4 * g) =
                    make_float4(o[n][t][0] * vo, o[n][t][1] * vo, o[n][t][2] * vo, o[n][t][3] * vo);
            if (g == 0) {
                lm[wave * rmax + c] = m[n];
                ll[wave * rmax + c] = ln;
            }
        }
        __syncthreads();
        for (int e = threadIdx.x; e < rmax * (D / 8); e += 64 * NWV) {
            const int r = e / (D / 8), d = e % (D / 8) * 8;
            if (rn + r >= rows) continue;
            const Row x = row_of<true>(p, s, b, h, rn + r);
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
}

// ---- many rows ---------------------------------------------------------------

// The blocks deal the call's steps (64 keys of one block of rows, "unit") evenly: all
// units' steps in a row, sequence by sequence, are cut into p.even shares of one length,
// whatever the sequences' lengths are, so that all CUs end together.  A share covers the
// end of a unit, whole ones, and the beginning of another; what is not whole leaves
// partial results, 2 slots of rows to a block: one for a unit that the share does not
// begin with.
struct Shares {
    uint32_t even, total;
    __device__ __forceinline__ uint32_t from(uint32_t j) const {
        return static_cast<uint32_t>(static_cast<uint64_t>(j) * total / even);
    }
    // The share that a step lies in: the last one that begins no later.
    __device__ __forceinline__ uint32_t of(uint32_t step) const { return ((step + 1) * even - 1) / total; }   // (below 2^31)
};
template <int D>
__device__ __forceinline__ int units_of(const AttnParams& p, const KvSeq& s) {       // of a head
    return (s.n * p.group + kPhaseRows<D> - 1) / kPhaseRows<D>;
}
__device__ __forceinline__ uint32_t steps_of(const KvSeq& s) { return s.kv > 0 ? (s.kv + 63) >> 6 : 1; }

// 4 trees of up to 256 nodes over up to 16100 keys, 8 heads of 128 for 32, capped (176
// GFLOP): 337 us, keys cut at one length for all sequences 403.  Bound by the matrix units
// and the softmax's issue, as the kernel for prompts; 11% of the products are of rows past
// the last block's end.
template <int DT, int D, bool CAP>
__global__ __launch_bounds__(512, 2) void kv_attn_tree_phase_kernel(AttnParams p) {
    extern __shared__ __attribute__((aligned(16))) char lds[];
    constexpr int ROWS = kPhaseRows<D>;
    uint32_t* upto = reinterpret_cast<uint32_t*>(lds + 2 * 2 * 64 * D * 2);     // [64] running sums
    uint32_t* steps = upto + 64;
    uint32_t at = 0, end = 1, share = 0, begin = 0;
    if (p.even) {
        if (threadIdx.x < 64) {
            const int b = threadIdx.x;
            uint32_t n = 0, w = 0;
            if (b < p.ix.batch) {
                const KvSeq s = kv_seq(p.ix, b);
                n = steps_of(s);
                w = n * static_cast<uint32_t>(units_of<D>(p, s)) * static_cast<uint32_t>(p.heads);
            }
            w = wave_sum_up(w);
            upto[b] = w;
            steps[b] = n;
            if (blockIdx.x == 0) p.shares[b] = w;
        }
        __syncthreads();
        const Shares shares{p.even, upto[63]};
        // consecutive shares, often of one head's keys, to one XCD
        share = p.even % 8 ? blockIdx.x : blockIdx.x % 8 * (p.even / 8) + blockIdx.x / 8;
        at = begin = __builtin_amdgcn_readfirstlane(shares.from(share));
        end = __builtin_amdgcn_readfirstlane(shares.from(share + 1));
        if (at >= end) return;
    }
    do {
        int b, h, rt, k0, k1;
        int64_t slot = -1;
        KvSeq s;
        if (p.even) {
            b = __builtin_ctzll(__ballot(upto[threadIdx.x & 63] > at));
            s = kv_seq(p.ix, b);
            const uint32_t n = __builtin_amdgcn_readfirstlane(steps[b]);
            const uint32_t off = at - (b > 0 ? __builtin_amdgcn_readfirstlane(upto[b - 1]) : 0), unit = off / n;
            const uint32_t step = off - unit * n, left = end - at, len = n - step < left ? n - step : left;
            const int units = units_of<D>(p, s);
            h = static_cast<int>(unit) / units;
            rt = static_cast<int>(unit) % units;
            k0 = 64 * static_cast<int>(step);
            k1 = s.kv - k0 > 64 * static_cast<int>(len) ? k0 + 64 * static_cast<int>(len) : s.kv;
            if (len < n) slot = (2 * static_cast<int64_t>(share) + (at > begin ? 1 : 0)) * ROWS;
            at += len;
        } else {
            at = end;
            h = static_cast<int>(blockIdx.x % p.heads);
            b = static_cast<int>(blockIdx.x / p.heads % p.ix.batch);
            rt = static_cast<int>(blockIdx.x / p.heads / p.ix.batch);
            s = kv_seq(p.ix, b);
            if (rt * ROWS >= s.n * p.group) return;
            k0 = 0;
            k1 = s.kv;
        }
        phase_unit<DT, D, CAP, true>(p, lds, s, b, h, rt * ROWS, k0, k1,
                                     [&](const Row&, int r) -> int64_t { return slot < 0 ? -1 : slot + r; });
        if (at < end) __syncthreads();
    } while (at < end);
}

// Joins the partial results of the rows whose units lie in several shares, D / 8 lanes
// to each row.
template <int DT, int D>
__global__ __launch_bounds__(256) void kv_attn_tree_join_kernel(AttnParams p) {
    constexpr int LANES = D / 8, ROWS = kPhaseRows<D>;
    const int64_t u = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) / LANES;
    const int64_t at = u / p.heads_q;
    const int head = static_cast<int>(u % p.heads_q), d = threadIdx.x % LANES * 8;
    const int b = static_cast<int>(at / p.ix.max_q), i = static_cast<int>(at % p.ix.max_q);
    if (b >= p.ix.batch) return;
    const KvSeq s = kv_seq(p.ix, b);
    if (i >= s.n) return;
    const Shares shares{p.even, p.shares[63]};
    const int r = i * p.group + head % p.group;
    const uint32_t n = steps_of(s), unit = head / p.group * units_of<D>(p, s) + r / ROWS;
    const uint32_t from = (b > 0 ? p.shares[b - 1] : 0) + unit * n;
    const uint32_t first = shares.of(from), last = shares.of(from + n - 1);
    if (first == last) return;                // the result is there
    float m = kNegInf, sum = 0.f, f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (uint32_t j = first; j <= last; ++j) {
        const uint32_t begin = shares.from(j);
        if (begin == shares.from(j + 1)) continue;            // (fewer steps than shares)
        const int64_t part = (2 * static_cast<int64_t>(j) + (from > begin ? 1 : 0)) * ROWS + r % ROWS;
        const float ms = p.part_ml[2 * part], ls = p.part_ml[2 * part + 1];
        float v[8];
        load8<F32>(p.part_o + part * D + d, v);
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

template <int DT, int D, bool CAP>
hipError_t launch_many(AttnParams p, const KvAttnPlan& plan, void* ws, hipStream_t st) {
    if (plan.even) {
        p.even = static_cast<uint32_t>(plan.even);
        p.shares = static_cast<uint32_t*>(ws);
        p.part_o = static_cast<float*>(ws) + 64;
        p.part_ml = p.part_o + 2 * static_cast<int64_t>(plan.even) * kPhaseRows<D> * D;
    }
    const hipError_t e =
        launch_lds(kv_attn_tree_phase_kernel<DT, D, CAP>, plan.blocks, 512, 2 * 2 * 64 * D * 2 + 512, p, st);
    if (e != hipSuccess || !plan.even) return e;
    const int64_t lanes = static_cast<int64_t>(p.ix.batch) * p.ix.max_q * p.heads_q * (D / 8);
    kv_attn_tree_join_kernel<DT, D><<<dim3(static_cast<unsigned>((lanes + 255) / 256)), 256, 0, st>>>(p);
    return hipGetLastError();
}


template <int DT, int D, bool CAP>
hipError_t launch_cap(const AttnParams& p, const KvAttnPlan& plan, void* ws, hipStream_t st) {
    if (plan.many) return launch_many<DT, D, CAP>(p, plan, ws, st);
    hipError_t e;
    if (D == 256 || plan.tile == 16)        // (32 rows of a 256-wide head do not fit a wave's registers)
        e = launch_lds(kv_attn_tree_kernel<DT, D, CAP, 1>, plan.blocks, 256, plan.lds_bytes, p, st);
    else
        e = launch_lds(kv_attn_tree_kernel<DT, D, CAP, D == 256 ? 1 : 2>, plan.blocks, 256, plan.lds_bytes, p, st);
    return e != hipSuccess ? e : launch_join<DT, D>(p, st);
}

template <int DT>
hipError_t launch_dt(const AttnParams& p, const KvAttnPlan& plan, int d, void* ws, hipStream_t st) {
    const bool cap = p.cap > 0.f;
    if (d == 64) return cap ? launch_cap<DT, 64, true>(p, plan, ws, st) : launch_cap<DT, 64, false>(p, plan, ws, st);
    if (d == 128) return cap ? launch_cap<DT, 128, true>(p, plan, ws, st) : launch_cap<DT, 128, false>(p, plan, ws, st);
    return cap ? launch_cap<DT, 256, true>(p, plan, ws, st) : launch_cap<DT, 256, false>(p, plan, ws, st);
}

}  // namespace

hipError_t launch_kv_attention_tree(const KvAttnPlan& plan, const void* q, int dtype, int64_t ldq, int heads_q,
                                    const KvIndex& ix, const int8_t* k, const int8_t* v, const float* ks,
                                    const float* vs, int heads, int d, float sm_scale, float cap, const uint32_t* mask,
                                    int64_t mask_ld, void* out, int64_t ldo, void* ws, hipStream_t st) {
    const AttnParams p =
        attn_params(plan, q, ldq, heads_q, ix, k, v, ks, vs, heads, d, sm_scale, cap, mask, mask_ld, out, ldo, ws);
    return dtype == F16 ? launch_dt<F16>(p, plan, d, ws, st) : launch_dt<BF16>(p, plan, d, ws, st);
}

}  // namespace qlin
