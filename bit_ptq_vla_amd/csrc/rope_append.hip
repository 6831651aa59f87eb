// Rotary positions on the q and k columns of a q|k|v projection, and the new
// keys and values into a paged int8 cache, for gfx950.
//
//   pair (a, b) at position p, angle index i:
//     a' = a cos[p][i] - b sin[p][i],  b' = b cos[p][i] + a sin[p][i]
//   page scale s = max(s_old, fp32(max|new| / 127))  (s_old: the page already
//     holds tokens), codes rne(v / s), held codes rne(c s_old / s).
//
// One launch.  A block owns one (page, head) of K or of V and every token the
// call adds to it, so the page's scale is decided in one place; the blocks
// after those turn q.  K is rotated in float64: a 16-bit value times an fp32
// cosine is exact there, so scales and codes are those of exact arithmetic
// (q's pairs take fp32, one rounding of the products more than its own).
//
// A task is 16 values of a head: the two 8-value chunks that hold each other's
// partners (halves layout: 8s and 8s + rot/2; interleaved: 16s and 16s + 8).
// V's codes cross LDS to lie keys-first ([d][page]) as the attention reads
// them.

#include "device_common.h"
#include "kv_index.h"
#include "qlin_internal.h"

namespace qlin {

namespace {

struct AppendParams {
    KvIndex ix;
    const void* qkv;
    int64_t ld;
    const float* rope;
    int64_t rope_len;
    const int32_t* positions;
    int8_t* k;
    int8_t* v;
    float* ks;
    float* vs;
    void* q_out;
    int64_t ldq;
    int heads_q, heads, rot, interleaved;
    int touched;       // pages per sequence the grid covers
    int64_t kv_blocks;
};

// Columns of the two chunks of task s (of D / 16) and the angle its pairs start at.
struct Task {
    int ca, cb, angle;
    bool turn;
};

__device__ __forceinline__ Task task_of(int s, int rot, int interleaved) {
    Task t;
    t.turn = 16 * s < rot;
    t.angle = t.turn ? 8 * s : 0;
    if (t.turn && !interleaved) {
        t.ca = 8 * s;
        t.cb = 8 * s + rot / 2;
    } else {
        t.ca = 16 * s;
        t.cb = 16 * s + 8;
    }
    return t;
}

// a, b: the task's chunks, turned in place by the angles cs (cosines) and sn.
template <typename F>
__device__ __forceinline__ void turn16(F (&a)[8], F (&b)[8], const float cs[8], const float sn[8], int interleaved) {
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const F c0 = cs[i], s0 = sn[i], c1 = cs[4 + i], s1 = sn[4 + i];
            const F x = a[2 * i], y = a[2 * i + 1], z = b[2 * i], w = b[2 * i + 1];
            a[2 * i] = x * c0 - y * s0;
            a[2 * i + 1] = y * c0 + x * s0;
            b[2 * i] = z * c1 - w * s1;
            b[2 * i + 1] = w * c1 + z * s1;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const F c = cs[i], s = sn[i], x = a[i], y = b[i];
            a[i] = x * c - y * s;
            b[i] = y * c + x * s;
        }
    }
}

__device__ __forceinline__ const float* rope_row(const AppendParams& p, int64_t row, int64_t place) {
    int64_t pos = p.positions ? p.positions[row] : place;
    pos = pos < 0 ? 0 : pos >= p.rope_len ? p.rope_len - 1 : pos;
    return p.rope + pos * p.rot;
}

template <int DT>
__device__ __forceinline__ void load16(const AppendParams& p, int64_t row, int64_t col0, const Task& t, bool turn,
                                       int64_t place, double (&a)[8], double (&b)[8]) {
    const char* src = static_cast<const char*>(p.qkv) + (row * p.ld + col0) * 2;
    float fa[8], fb[8];
    load8<DT>(src + t.ca * 2, fa);
    load8<DT>(src + t.cb * 2, fb);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        a[i] = fa[i];
        b[i] = fb[i];
    }
    if (turn) {
        const float* r = rope_row(p, row, place) + t.angle;
        float cs[8], sn[8];
        load8<F32>(r, cs);
        load8<F32>(r + p.rot / 2, sn);
        turn16<double>(a, b, cs, sn, p.interleaved);
    }
}

__device__ __forceinline__ double finite_abs(double v) {
    const double a = fabs(v);
    return a <= 1.7976931348623157e308 ? a : 0.0;   // infinities and NaN do not set the scale
}

// rne(v / s) on the grid: infinities at its ends, NaN as 0.
__device__ __forceinline__ int code_of(double v, double s) {
    if (!(s > 0.0) || v != v) return 0;
    return static_cast<int>(fmin(fmax(rint(v / s), -127.0), 127.0));
}

template <int DT, int D, int TPB>
__device__ __forceinline__ void store_page(const AppendParams& p, int64_t unit) {
    constexpr int S = D / 16;
    __shared__ double red[TPB / 64];
    __shared__ uint8_t tile[D * 64];
    const int tid = threadIdx.x;
    const bool is_v = unit & 1;
    const int h = static_cast<int>((unit >> 1) % p.heads);
    const int64_t rest = (unit >> 1) / p.heads;
    const int b = static_cast<int>(rest / p.touched);
    const KvSeq seq = kv_seq(p.ix, b);
    if (seq.n == 0) return;
    const KvSpan span = kv_touched(p.ix, seq, static_cast<int>(rest % p.touched));
    if (span.hi <= span.lo) return;
    const int page = kv_page(p.ix, b, span.idx);
    if (page == kNoPage) return;

    const int ps = p.ix.page_size;
    const int start = span.idx * ps, o_lo = span.lo - start, count = span.hi - span.lo;
    const int64_t col0 = (static_cast<int64_t>(p.heads_q) + (is_v ? p.heads : 0) + h) * D;
    const int64_t slot = static_cast<int64_t>(page) * p.heads + h;
    float* scale = (is_v ? p.vs : p.ks) + slot;
    int8_t* base = (is_v ? p.v : p.k) + slot * ps * D;
    const float s_old = o_lo > 0 ? *scale : 0.f;

    double top = 0.0;
    for (int i = tid; i < count * S; i += TPB) {
        const int j = span.lo + i / S;
        const Task t = task_of(i % S, is_v ? 0 : p.rot, p.interleaved);
        double a[8], c[8];
        load16<DT>(p, seq.row0 + (j - seq.first), col0, t, !is_v && t.turn, j, a, c);
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmax(top, fmax(finite_abs(a[e]), finite_abs(c[e])));
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) top = fmax(top, __shfl_xor(top, d, 64));
    if (TPB > 64) {
        if ((tid & 63) == 0) red[tid >> 6] = top;
        __syncthreads();
        for (int w = 0; w < TPB / 64; ++w) top = fmax(top, red[w]);
    }
    const float s_new = fmaxf(s_old, static_cast<float>(top / 127.0));
    const bool grown = o_lo > 0 && s_new != s_old;
    const double s = s_new;
    if (tid == 0) *scale = s_new;

    for (int i = tid; i < count * S; i += TPB) {
        const int j = span.lo + i / S;
        const Task t = task_of(i % S, is_v ? 0 : p.rot, p.interleaved);
        double a[8], c[8];
        load16<DT>(p, seq.row0 + (j - seq.first), col0, t, !is_v && t.turn, j, a, c);
        const int off = j - start;
        if (is_v) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                tile[(t.ca + e) * ps + off] = static_cast<uint8_t>(code_of(a[e], s));
                tile[(t.cb + e) * ps + off] = static_cast<uint8_t>(code_of(c[e], s));
            }
        } else {
            uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                w[e >> 2] |= (static_cast<uint32_t>(code_of(a[e], s)) & 0xFFu) << (8 * (e & 3));
                w[2 + (e >> 2)] |= (static_cast<uint32_t>(code_of(c[e], s)) & 0xFFu) << (8 * (e & 3));
            }
            *reinterpret_cast<uint2*>(base + off * D + t.ca) = make_uint2(w[0], w[1]);
            *reinterpret_cast<uint2*>(base + off * D + t.cb) = make_uint2(w[2], w[3]);
        }
    }
    // the page's earlier codes follow its scale
    if (grown) {
        const double so = s_old;
        for (int i = tid; i < o_lo * D; i += TPB) {
            const int off = is_v ? i % o_lo : i / D, col = is_v ? i / o_lo : i % D;
            int8_t* at = is_v ? base + col * ps + off : base + off * D + col;
            *at = static_cast<int8_t>(code_of(static_cast<double>(*at) * so, s));
        }
    }
    if (is_v) {
        __syncthreads();
        for (int i = tid; i < D * ps / 4; i += TPB) {
            const int col = i / (ps / 4), off = i % (ps / 4) * 4;
            const uint32_t w = *reinterpret_cast<const uint32_t*>(tile + col * ps + off);
            if (off >= o_lo && off + 4 <= o_lo + count) {
                *reinterpret_cast<uint32_t*>(base + col * ps + off) = w;
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (off + e >= o_lo && off + e < o_lo + count)
                        base[col * ps + off + e] = static_cast<int8_t>(w >> (8 * e));
            }
        }
    }
}

template <int DT, int D, int TPB>
__device__ __forceinline__ void turn_q(const AppendParams& p, int64_t block) {
    constexpr int S = D / 16;
    const int64_t i = block * TPB + threadIdx.x;
    const int64_t head = i / S, row = head / p.heads_q;
    if (row >= p.ix.tokens) return;
    // the row's sequence: the last one that starts at or before it
    int lo = 0, hi = p.ix.batch;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.ix.q_start[mid] <= row) lo = mid;
        else hi = mid;
    }
    // rows behind the last sequence (or in front of the first) stay as they are
    const KvSeq seq = kv_seq(p.ix, lo);
    if (row < seq.row0 || row >= seq.row0 + seq.n) return;
    const Task t = task_of(static_cast<int>(i % S), p.rot, p.interleaved);
    const int64_t col0 = (head % p.heads_q) * D;
    const char* src = static_cast<const char*>(p.qkv) + (row * p.ld + col0) * 2;
    char* dst = static_cast<char*>(p.q_out) + (row * p.ldq + col0) * 2;
    float a[8], b[8];
    load8<DT>(src + t.ca * 2, a);
    load8<DT>(src + t.cb * 2, b);
    if (t.turn) {
        const float* r = rope_row(p, row, seq.first + (row - seq.row0)) + t.angle;
        float cs[8], sn[8];
        load8<F32>(r, cs);
        load8<F32>(r + p.rot / 2, sn);
        turn16<float>(a, b, cs, sn, p.interleaved);
    }
    store8<DT>(dst + t.ca * 2, a);
    store8<DT>(dst + t.cb * 2, b);
}

template <int DT, int D, int TPB>
__global__ __launch_bounds__(TPB) void rope_append_kernel(AppendParams p) {
    const int64_t block = blockIdx.x;
    if (block < p.kv_blocks)
        store_page<DT, D, TPB>(p, block);
    else
        turn_q<DT, D, TPB>(p, block - p.kv_blocks);
}

template <int DT, int D, int TPB>
hipError_t launch_tpb(AppendParams p, hipStream_t st) {
    p.kv_blocks = static_cast<int64_t>(p.ix.batch) * p.touched * p.heads * 2;
    const int64_t q_blocks = (p.ix.tokens * p.heads_q * (D / 16) + TPB - 1) / TPB;
    rope_append_kernel<DT, D, TPB><<<dim3(static_cast<unsigned>(p.kv_blocks + q_blocks)), TPB, 0, st>>>(p);
    return hipGetLastError();
}

template <int DT, int D>
hipError_t launch_d(const AppendParams& p, hipStream_t st) {
    // a block per (page, head): one wave where a call adds few values to each
    if (p.ix.max_q * (D / 16) <= 64) return launch_tpb<DT, D, 64>(p, st);
    return launch_tpb<DT, D, 256>(p, st);
}

template <int DT>
hipError_t launch_dt(const AppendParams& p, int d, hipStream_t st) {
    if (d == 64) return launch_d<DT, 64>(p, st);
    if (d == 128) return launch_d<DT, 128>(p, st);
    return launch_d<DT, 256>(p, st);
}

// angle(p, i) = p / stretch * base^(-2 i / rot), cos and sin in float64
__global__ __launch_bounds__(256) void rope_table_kernel(float* table, int64_t n, int half, double base,
                                                         double stretch) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= n * half) return;
    const int64_t pos = i / half;
    const int f = static_cast<int>(i % half);
    const double angle = static_cast<double>(pos) / stretch * pow(base, -static_cast<double>(f) / half);
    table[pos * 2 * half + f] = static_cast<float>(cos(angle));
    table[pos * 2 * half + half + f] = static_cast<float>(sin(angle));
}

}  // namespace

hipError_t launch_rope_append(const void* qkv, int dtype, int64_t ld, int heads_q, const float* rope, int64_t rope_len,
                              int rot, int interleaved, const int32_t* positions, const KvIndex& ix, int8_t* k,
                              int8_t* v, float* ks, float* vs, int heads, int d, void* q_out, int64_t ldq,
                              hipStream_t st) {
    AppendParams p{ix, qkv, ld, rope, rope_len, positions, k, v, ks, vs, q_out, ldq, heads_q, heads, rot, interleaved,
                   kv_max_touched(ix.max_q, ix.page_size), 0};
    return dtype == F16 ? launch_dt<F16>(p, d, st) : launch_dt<BF16>(p, d, st);
}

hipError_t launch_rope_table(float* table, int64_t positions, int rot, double base, double stretch, hipStream_t st) {
    const int64_t blocks = (positions * (rot / 2) + 255) / 256;
    rope_table_kernel<<<dim3(static_cast<unsigned>(blocks)), 256, 0, st>>>(table, positions, rot / 2, base, stretch);
    return hipGetLastError();
}

}  // namespace qlin
