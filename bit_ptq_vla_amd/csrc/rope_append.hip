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
// after those turn q.  Scales and codes are those of exact arithmetic, which
// float64 gives (a 16-bit value times an fp32 cosine is exact there): values
// are turned in fp32, and what fp32 cannot decide, the maximum among values
// close to it and the side of a half-integer a quotient lies on, is decided
// again in float64 by the threads concerned.  (All of it in float64 took 21
// vector instructions a value, more than the memory time of a prompt.)
//
// The values stay in registers between the scale's reduction and the codes,
// x * (1 / s) rounded by a magic add, whose distance from a half-integer is
// known.
//
// A K task is 16 values of a token's head: the two 8-value chunks that hold
// each other's partners (halves layout: 8s and 8s + rot/2; interleaved: 16s
// and 16s + 8).  A V task is 8 dimensions of four tokens, whose codes are four
// bytes each of the keys-first page.
//
// Prompts: q|k|v read once, q written, one byte a key and value.  52224 tokens of
// 8 + 8 + 8 heads of 256 (844 MB) take 248 us, 3.4 TB/s.  The k blocks bound it
// (of 266 us with larger blocks: q and v alone 167, q and k alone 263): 64 bytes
// of cosines and sines, from L2, to 32 of values, and a chain of loads, maximum,
// its check in float64, and codes in each.  A decode step is latency (64 requests
// of 8 heads: 7.4 us a call), with many heads the lines of V: a token's bytes lie
// in head_dim rows of its page, each a partly written line (256 requests of 32
// heads of 128: 30 us at pages of 64 tokens, 24 at 16).

#include "code_pack.h"
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
    uint32_t kv_blocks, q_blocks;   // blocks that store; blocks of a sequence's q
};

typedef unsigned short us2 __attribute__((ext_vector_type(2)));

// Columns of the two chunks of task s (of D / 16) and the angle its pairs start at.
struct Task {
    int ca, cb, angle;
    bool turn, neighbours;
};

__device__ __forceinline__ Task task_of(int s, int rot, int interleaved) {
    Task t;
    t.turn = 16 * s < rot;
    t.angle = t.turn ? 8 * s : 0;
    t.neighbours = t.turn && interleaved;
    if (t.turn && !interleaved) {
        t.ca = 8 * s;
        t.cb = 8 * s + rot / 2;
    } else {
        t.ca = 16 * s;
        t.cb = 16 * s + 8;
    }
    return t;
}

// Two chunks (the values at t.ca .. and at t.cb ..) to pairs (x[2 i], x[2 i + 1])
// and back: neighbours of a chunk in the interleaved layout, else one of each.
__device__ __forceinline__ void to_pairs(const float a[8], const float b[8], bool neighbours, float x[16]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[2 * i] = neighbours ? (i < 4 ? a[(2 * i) & 7] : b[(2 * i) & 7]) : a[i];
        x[2 * i + 1] = neighbours ? (i < 4 ? a[(2 * i + 1) & 7] : b[(2 * i + 1) & 7]) : b[i];
    }
}
template <typename T>
__device__ __forceinline__ void to_chunks(const T x[16], bool neighbours, T a[8], T b[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        a[i] = neighbours ? x[i] : x[2 * i];
        b[i] = neighbours ? x[8 + i] : x[2 * i + 1];
    }
}

__device__ __forceinline__ const float* rope_row(const AppendParams& p, int64_t row, int64_t place) {
    int64_t pos = p.positions ? p.positions[row] : place;
    pos = pos < 0 ? 0 : pos >= p.rope_len ? p.rope_len - 1 : pos;
    return p.rope + pos * p.rot;
}

// A task's pairs and their angles (1, 0 where its columns do not turn).
template <int DT>
__device__ __forceinline__ void load_pairs(const AppendParams& p, int64_t row, int64_t col0, const Task& t,
                                           int64_t place, float x[16], float cs[8], float sn[8]) {
    const char* src = static_cast<const char*>(p.qkv) + (row * p.ld + col0) * 2;
    float a[8], b[8];
    load8<DT>(src + t.ca * 2, a);
    load8<DT>(src + t.cb * 2, b);
    if (t.turn) {
        const float* r = rope_row(p, row, place) + t.angle;
        load8<F32>(r, cs);
        load8<F32>(r + p.rot / 2, sn);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            cs[i] = 1.f;
            sn[i] = 0.f;
        }
    }
    to_pairs(a, b, t.neighbours, x);
}

// The pairs turned in fp32.  (Columns that do not turn stay as they are: a
// product with 0 would make an infinity's partner NaN.)
template <int DT>
__device__ __forceinline__ void load16(const AppendParams& p, int64_t row, int64_t col0, const Task& t, int64_t place,
                                       float x[16]) {
    float cs[8], sn[8];
    load_pairs<DT>(p, row, col0, t, place, x, cs, sn);
    if (t.turn) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float u = x[2 * i], w = x[2 * i + 1];
            x[2 * i] = u * cs[i] - w * sn[i];
            x[2 * i + 1] = w * cs[i] + u * sn[i];
        }
    }
}

// f(i, u, w) for the pairs in float64, one at a time, so that few float64
// values live together.
template <int DT, typename F>
__device__ __forceinline__ void each_pair(const AppendParams& p, int64_t row, int64_t col0, const Task& t,
                                          int64_t place, F f) {
    float x[16], cs[8], sn[8];
    load_pairs<DT>(p, row, col0, t, place, x, cs, sn);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const double u = x[2 * i], w = x[2 * i + 1], c = cs[i], d = sn[i];
        f(i, t.turn ? u * c - w * d : u, t.turn ? w * c + u * d : w);
        __builtin_amdgcn_sched_barrier(0);
    }
}

// rne(v / s) on the grid: infinities at its ends, NaN as 0.
__device__ __forceinline__ int code_of(double v, double s) {
    if (!(s > 0.0) || v != v) return 0;
    return static_cast<int>(fmin(fmax(rint(v / s), -127.0), 127.0));
}

// rne(v / s) where r is within a small fraction of a step of v / s, by the sign
// of v - h s for the half-integer h next to r (h s is exact).
__device__ __forceinline__ int code_near(double v, double s, float r) {
    const float q = rintf(r), h = r > q ? q + 0.5f : q - 0.5f;
    const double t = fma(-static_cast<double>(h), s, v);
    const int lower = static_cast<int>(h - 0.5f);
    const int code = t > 0.0 ? lower + 1 : t < 0.0 ? lower : lower + (lower & 1);
    return code < -127 ? -127 : code > 127 ? 127 : code;
}

// The codes of n fp32 values in the low bytes of cb.  False where a value lies
// so near a half-integer of v / s that fp32 cannot tell its side.  A turned
// value fma(a, c, -(b d)) is off by 2^-24 (|b d| + |v|), and |b d| is at most
// sqrt 2 times the page's maximum M, since a turn is a product of complex
// numbers: 2.5 x 2^-24 M, 127 of which are 1.9e-5 in steps of s = M / 127; 1 / s
// and its use add 127.5 x 2^-23 = 1.6e-5.  The window is wider.
constexpr float kMagic = 12582912.f;   // 1.5 x 2^23: the sum's low bits are the rounded value
template <int N>
__device__ __forceinline__ bool codes_f32(const float* v, float inv, uint32_t* cb) {
    float worst = 0.f;
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const float qb = fmaf(v[e], inv, kMagic);
        worst = fmaxf(worst, fabsf(fmaf(v[e], inv, kMagic - qb)));
        cb[e] = __float_as_uint(qb);
    }
    return worst < 0.5f - 6e-5f;
}

// rne(c s_old / s_new) of a word's four codes.  fp32 leaves c s_old / s_new
// within 127 x 2^-23 (1.6e-5); what comes nearer than that to a half-integer
// is decided in float64, where c s_old is exact.
__device__ __forceinline__ uint32_t rescale4(uint32_t was, float ratio, double s_old, double s_new) {
    float c[4];
    uint32_t cb[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) c[e] = static_cast<float>(static_cast<int8_t>(was >> (8 * e)));
    if (!(ratio >= 0.f && ratio <= 1.f)) {              // what no append leaves in a scale
#pragma unroll 1
        for (int e = 0; e < 4; ++e) cb[e] = static_cast<uint32_t>(code_of(c[e] * s_old, s_new));
    } else if (!codes_f32<4>(c, ratio, cb)) {
#pragma unroll
        for (int e = 0; e < 4; ++e) cb[e] = static_cast<uint32_t>(code_near(c[e] * s_old, s_new, c[e] * ratio));
    }
    return __builtin_amdgcn_perm(cb[1], cb[0], 0x0C0C0400u) | __builtin_amdgcn_perm(cb[3], cb[2], 0x04000C0Cu);
}

// A page's `held` earlier codes follow its scale: 16 codes to a thread, four
// such loads under way together.  K's are contiguous; of a V row's only the
// first `held` bytes are the page's.
template <int TPB, int D>
__device__ __forceinline__ void rescale_page(int8_t* base, bool is_v, int held, int ps, double s_old, double s_new) {
    const float ratio = static_cast<float>(s_old) / static_cast<float>(s_new);
    const int row = is_v ? (held + 15) >> 4 : 1, n = is_v ? row * D : held * (D / 16);
#pragma unroll 1
    for (int i0 = threadIdx.x; i0 < n; i0 += 4 * TPB) {
        uint4 was[4];
        int off[4], at[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = i0 + u * TPB < n ? i0 + u * TPB : i0, r = is_v ? i / row : 0;
            off[u] = is_v ? (i - r * row) * 16 : 0;
            at[u] = is_v ? r * ps + off[u] : 16 * i;
            was[u] = *reinterpret_cast<const uint4*>(base + at[u]);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (i0 + u * TPB >= n) break;
            const uint32_t w[4] = {was[u].x, was[u].y, was[u].z, was[u].w};
            uint32_t now[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) now[e] = rescale4(w[e], ratio, s_old, s_new);
            if (!is_v || off[u] + 16 <= held) {
                *reinterpret_cast<uint4*>(base + at[u]) = make_uint4(now[0], now[1], now[2], now[3]);
            } else {
#pragma unroll 1
                for (int e = 0; off[u] + e < held; ++e) {
                    const uint32_t word = e < 8 ? e < 4 ? now[0] : now[1] : e < 12 ? now[2] : now[3];
                    base[at[u] + e] = static_cast<int8_t>(word >> (8 * (e & 3)));
                }
            }
        }
    }
}

template <int TPB>
__device__ __forceinline__ float block_max(float top, float* red) {
    top = wave_max(top, 64);
    if (TPB > 64) {
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < TPB / 64; ++w) top = fmaxf(top, red[w]);
    }
    return top;
}

template <int DT, int D, int TPB>
__device__ __forceinline__ void store_page(const AppendParams& p, uint32_t unit) {
    constexpr int S = D / 16;
    // most tasks a thread takes: 64 tokens (a page), or 64 / S of them to a wave
    constexpr int KT = TPB == 64 ? 1 : 64 * S / TPB, VT = TPB == 64 ? 1 : 16 * (D / 8) / TPB > 0 ? 16 * (D / 8) / TPB : 1;
    __shared__ float red[TPB / 64];
    __shared__ unsigned long long exact;
    const int tid = threadIdx.x;
    // the k blocks first, then the v blocks: 266 us for 52224 tokens of 8 heads of
    // 256 in blocks of 512 threads, alternating 293
    const uint32_t half = p.kv_blocks >> 1;
    const bool is_v = unit >= half;
    if (is_v) unit -= half;
    const uint32_t pair = unit / p.heads, h = unit - pair * p.heads;
    const int b = static_cast<int>(pair / p.touched);
    const KvSeq seq = kv_seq(p.ix, b);
    if (seq.n == 0) return;
    const KvSpan span = kv_touched(p.ix, seq, static_cast<int>(pair - b * p.touched));
    if (span.hi <= span.lo) return;
    const int page = kv_page(p.ix, b, span.idx);

    const int ps = p.ix.page_size;
    const int start = span.idx * ps, o_lo = span.lo - start, count = span.hi - span.lo;
    const int64_t col0 = (static_cast<int64_t>(p.heads_q) + (is_v ? p.heads : 0) + h) * D;
    const int64_t row0 = seq.row0 + (span.lo - seq.first);        // the span's first row

    // the span's values, and their maximum
    const int wf = o_lo >> 2, nw = ((o_lo + count + 3) >> 2) - wf;       // V: words of four tokens
    float kx[KT][16];                         // K: turned, fp32
    uint4 vraw[VT][4];
    float top = 0.f;
    bool odd = false;                         // an infinity or a NaN among the thread's values
    if (!is_v) {
        float nan = 0.f;
#pragma unroll
        for (int n = 0; n < KT; ++n) {
            const int i = tid + n * TPB;
            if (i < count * S) {
                const Task t = task_of(i % S, p.rot, p.interleaved);
                load16<DT>(p, row0 + i / S, col0, t, span.lo + i / S, kx[n]);
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                    top = max3_abs(top, kx[n][e], kx[n][e + 1]);
                    nan = fmaf(kx[n][e], 0.f, fmaf(kx[n][e + 1], 0.f, nan));
                }
            }
        }
        odd = nan != nan;
        if (odd) top = __builtin_inff();
    } else {
#pragma unroll
        for (int n = 0; n < VT; ++n) {
            const int i = tid + n * TPB;
            if (i < nw * (D / 8)) {
                const int c8 = i / nw, w = wf + i - c8 * nw;
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const int at = 4 * w + t - o_lo;              // token of the span
                    const bool in = at >= 0 && at < count;
                    const char* src = static_cast<const char*>(p.qkv) + ((row0 + (in ? at : 0)) * p.ld + col0 + 8 * c8) * 2;
                    vraw[n][t] = *reinterpret_cast<const uint4*>(src);
                    if (!in) vraw[n][t] = make_uint4(0, 0, 0, 0);
                }
            }
        }
        // magnitudes of 16-bit floats order as their bits (infinities and NaN last)
        us2 m = {0, 0};
#pragma unroll
        for (int n = 0; n < VT; ++n) {
            if (tid + n * TPB < nw * (D / 8)) {
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const uint32_t w[4] = {vraw[n][t].x, vraw[n][t].y, vraw[n][t].z, vraw[n][t].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const us2 x = __builtin_bit_cast(us2, w[e] & 0x7FFF7FFFu);
                        m = m > x ? m : x;
                    }
                }
            }
        }
        const uint16_t lo = m[0], hi = m[1], bits = lo > hi ? lo : hi;
        odd = bits >= (DT == BF16 ? 0x7F80 : 0x7C00);
        top = odd ? __builtin_inff() : DT == BF16 ? bf16_to_f32(bits) : f16_bits_to_f32(bits);
    }
    if (page == kNoPage) return;              // (the whole block)
    const int64_t slot = static_cast<int64_t>(page) * p.heads + h;
    float* scale = (is_v ? p.vs : p.ks) + slot;
    int8_t* base = (is_v ? p.v : p.k) + slot * ps * D;
    const float s_old = o_lo > 0 ? *scale : 0.f;
    if (tid == 0) exact = 0;
    const float mine = top;
    top = block_max<TPB>(top, red);
    // The maximum in exact arithmetic: V's is what it is; a turned K value is off
    // by 2.5 x 2^-24 of it, so the threads whose own maximum comes within 2^-20
    // (or within 1e-36, where products leave fp32's normal range) look again.  With an infinity or a NaN in the page, all threads do, past those.
    double most = top;
    if (TPB == 64) __syncthreads();           // exact is set
    if (!(top < __builtin_inff()) || (!is_v && p.rot > 0)) {
        if (!(top < __builtin_inff()) || mine >= top * (1.f - 0x1p-20f) - 1e-36f) {
            double m = 0.0;
#pragma unroll 1
            for (int i = tid; i < count * S; i += TPB) {
                const Task t = task_of(i % S, is_v ? 0 : p.rot, p.interleaved);
                each_pair<DT>(p, row0 + i / S, col0, t, span.lo + i / S, [&](int, double u, double w) {
                    u = fabs(u), w = fabs(w);
                    if (u <= 1.7976931348623157e308) m = fmax(m, u);
                    if (w <= 1.7976931348623157e308) m = fmax(m, w);
                });
            }
            atomicMax(&exact, static_cast<unsigned long long>(__double_as_longlong(m)));   // m >= 0: ordered bits
        }
        __syncthreads();
        most = __longlong_as_double(static_cast<long long>(exact));
    }
    const float s_new = fmaxf(s_old, static_cast<float>(most / 127.0));
    const double s = s_new;
    // 1 / s in fp32; a scale so small that it overflows takes the quotients
    const float inv = s_new > 1e-36f ? 1.f / s_new : 0.f;
    const bool plain = !odd && (s_new > 1e-36f || s_new == 0.f);
    if (tid == 0) *scale = s_new;

    if (!is_v) {
#pragma unroll
        for (int n = 0; n < KT; ++n) {
            const int i = tid + n * TPB;
            if (i < count * S) {
                const Task t = task_of(i % S, p.rot, p.interleaved);
                uint32_t cb[16];
                if (!(codes_f32<16>(kx[n], inv, cb) && plain)) {
                    each_pair<DT>(p, row0 + i / S, col0, t, span.lo + i / S, [&](int e, double u, double w) {
                        cb[2 * e] = plain ? code_near(u, s, kx[n][2 * e] * inv) : code_of(u, s);
                        cb[2 * e + 1] = plain ? code_near(w, s, kx[n][2 * e + 1] * inv) : code_of(w, s);
                    });
                }
                uint32_t ca[8], cc[8];
                to_chunks(cb, t.neighbours, ca, cc);
                int8_t* dst = base + (o_lo + i / S) * D;
                *reinterpret_cast<uint2*>(dst + t.ca) = pack8_i8(ca);
                *reinterpret_cast<uint2*>(dst + t.cb) = pack8_i8(cc);
            }
        }
    } else {
#pragma unroll
        for (int n = 0; n < VT; ++n) {
            const int i = tid + n * TPB;
            if (i < nw * (D / 8)) {
                const int c8 = i / nw, w = wf + i - c8 * nw;
                uint32_t cb[4][8];
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    float x[8];
                    unpack8<DT>(vraw[n][t], x);
                    if (!(codes_f32<8>(x, inv, cb[t]) && plain)) {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            cb[t][e] = static_cast<uint32_t>(plain ? code_near(x[e], s, x[e] * inv) : code_of(x[e], s));
                    }
                }
                const int off = 4 * w;
                const bool whole = off >= o_lo && off + 4 <= o_lo + count;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    int8_t* dst = base + (8 * c8 + e) * ps + off;
                    const uint32_t lo = __builtin_amdgcn_perm(cb[1][e], cb[0][e], 0x0C0C0400u);
                    const uint32_t hi = __builtin_amdgcn_perm(cb[3][e], cb[2][e], 0x04000C0Cu);
                    if (whole) {
                        *reinterpret_cast<uint32_t*>(dst) = lo | hi;
                    } else {
#pragma unroll
                        for (int t = 0; t < 4; ++t)
                            if (off + t >= o_lo && off + t < o_lo + count) dst[t] = static_cast<int8_t>(cb[t][e]);
                    }
                }
            }
        }
    }
    if (o_lo > 0 && s_new != s_old) rescale_page<TPB, D>(base, is_v, o_lo, ps, s_old, s_new);
}

template <int DT, int D, int TPB>
__device__ __forceinline__ void turn_q(const AppendParams& p, uint32_t block) {
    constexpr int S = D / 16;
    // blocks of one sequence: its rows' q heads, 16 values to a thread
    const uint32_t b = block / p.q_blocks;
    const KvSeq seq = kv_seq(p.ix, static_cast<int>(b));
    const uint32_t i = (block - b * p.q_blocks) * TPB + threadIdx.x;
    const uint32_t head = i / S, r = head / p.heads_q;
    if (r >= static_cast<uint32_t>(seq.n)) return;
    const int64_t row = seq.row0 + r;
    const Task t = task_of(static_cast<int>(i % S), p.rot, p.interleaved);
    const int64_t col0 = static_cast<int64_t>(head - r * p.heads_q) * D;
    char* dst = static_cast<char*>(p.q_out) + (row * p.ldq + col0) * 2;
    float x[16];
    load16<DT>(p, row, col0, t, seq.first + static_cast<int64_t>(r), x);
    float a[8], c[8];
    to_chunks(x, t.neighbours, a, c);
    store8<DT>(dst + t.ca * 2, a);
    store8<DT>(dst + t.cb * 2, c);
}

template <int DT, int D, int TPB>
__global__ __launch_bounds__(TPB, TPB > 64 && D == 256 ? 3 : 4) void rope_append_kernel(AppendParams p) {
    if (blockIdx.x < p.kv_blocks)
        store_page<DT, D, TPB>(p, blockIdx.x);
    else
        turn_q<DT, D, TPB>(p, blockIdx.x - p.kv_blocks);
}

template <int DT, int D, int TPB>
hipError_t launch_tpb(AppendParams p, hipStream_t st) {
    p.kv_blocks = static_cast<uint32_t>(p.ix.batch) * p.touched * p.heads * 2;
    p.q_blocks = static_cast<uint32_t>((static_cast<int64_t>(p.ix.max_q) * p.heads_q * (D / 16) + TPB - 1) / TPB);
    rope_append_kernel<DT, D, TPB><<<dim3(p.kv_blocks + p.q_blocks * p.ix.batch), TPB, 0, st>>>(p);
    return hipGetLastError();
}

template <int DT, int D>
hipError_t launch_d(const AppendParams& p, hipStream_t st) {
    // A block per (page, head): one wave where a call adds few values to each (256
    // tokens of 32 heads of 128: 30 us, 256 threads 68), else 256 threads, so that
    // several pages share a CU and hide each other's waits (52224 tokens of 8 heads
    // of 256: 248 us, 512 threads 265, 1024 354; 6528 of 32 heads of 128: 75, 512
    // threads 94, 128 threads 86).
    if (p.ix.max_q * (D / 16) <= 64 && (p.ix.max_q + 6) / 4 * (D / 8) <= 64) return launch_tpb<DT, D, 64>(p, st);
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
                   kv_max_touched(ix.max_q, ix.page_size), 0, 0};
    return dtype == F16 ? launch_dt<F16>(p, d, st) : launch_dt<BF16>(p, d, st);
}

hipError_t launch_rope_table(float* table, int64_t positions, int rot, double base, double stretch, hipStream_t st) {
    const int64_t blocks = (positions * (rot / 2) + 255) / 256;
    rope_table_kernel<<<dim3(static_cast<unsigned>(blocks)), 256, 0, st>>>(table, positions, rot / 2, base, stretch);
    return hipGetLastError();
}

}  // namespace qlin
