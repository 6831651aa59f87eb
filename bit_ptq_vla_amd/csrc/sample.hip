// A token from each row of logits, for gfx950: temperature, min-p, top-k, top-p
// and a given random number.
//
//   w_i = 2^-y_i, y_i = (max - l_i) log2(e) / t; in the order of falling logits
//   (the lowest index first among equals) the kept tokens are a prefix, and the
//   token is its first whose running mass passes u times the prefix's mass.
//
// Masses are integers in units of 2^-44 (at most 2^18 weights of at most 2^44:
// below 2^62), so sums have no order: any split of a row over threads, and any
// order of their atomics, gives the same token.  A weight is evaluated in float64
// to 2^-46 of itself: the token is that of exact weights but for a u or a top-p
// within about 2^-40 of a border.
//
// Each filter, and the token itself, is one question: the first element of the
// order at which the running count, or mass, passes a target.  A histogram over y
// (32 bins to an octave, 46 octaves: weights below 2^-45 count nothing) leaves one
// bin; its few elements are gathered in LDS and sorted.  Where they are many (flat
// rows, equal logits) histograms over their key, the logit as an ordered integer,
// narrow them down; equal logits have equal weights, so among them the place is a
// division.

#include "device_common.h"
#include "qlin_internal.h"

namespace qlin {

namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr int kBins = 46 * 32;           // level 0
constexpr int kSub = 2048;               // bins of a further level
constexpr int kList = 2048;              // elements that are sorted at once
constexpr double kYEnd = 46.0;
constexpr uint64_t kOne = 1ull << 44;

struct Shared {
    double exp2_tab[1024];               // 2^(-i / 1024)
    uint64_t mass[kSub];                 // level 0: running sums, kept for every question
    uint32_t count[kSub];
    union {
        struct {
            uint64_t mass[kSub];
            uint32_t count[kSub];
        } sub;
        uint64_t list[kList];
    };
    uint64_t part64[kWaves];
    uint32_t part32[kWaves];
    uint64_t found64[2];
    uint32_t found32[4];
};

// Logits as ordered integers; equal logits (the zeros too) have equal keys.  NaN is 0,
// as -infinity: neither is ever taken.
__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t b = __float_as_uint(v + 0.f);
    if (v != v) return 0x007FFFFFu;
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float logit_of(uint32_t key) {
    return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}
constexpr uint32_t kKeyNone = 0x007FFFFFu;      // of -infinity

struct Row {
    const char* at;
    int vocab;
    float top;          // the largest logit
    double scale;       // log2(e) / t
    uint64_t least;     // min-p as a mass
};

__device__ __forceinline__ double y_of(const Row& r, float v) {
    return v == r.top ? 0.0 : (static_cast<double>(r.top) - static_cast<double>(v)) * r.scale;
}

// 2^-y in units of 2^-44, y in [0, kYEnd): 2^(-i / 1024) from the table times the
// exponential's series to its fourth power (the rest is below 2^-59).
__device__ __forceinline__ uint64_t mass_of(double y, const double* tab) {
    const int n = static_cast<int>(y * 1024.0);
    const double z = (y * 1024.0 - n) * -6.769015435155716e-4;      // -ln 2 / 1024
    const double p = fma(z, fma(z, fma(z, fma(z, 1.0 / 24, 1.0 / 6), 0.5), 1.0), 1.0);
    const double w = ldexp(tab[n & 1023] * p, 44 - (n >> 10));
    return static_cast<uint64_t>(__double_as_longlong(w + 0x1p52)) & 0xFFFFFFFFFFFFFull;
}

template <int DT>
__device__ __forceinline__ float load_one(const char* row, int i) {
    if constexpr (DT == F32) return reinterpret_cast<const float*>(row)[i];
    const uint16_t b = reinterpret_cast<const uint16_t*>(row)[i];
    return DT == BF16 ? bf16_to_f32(b) : f16_bits_to_f32(b);
}

// f(index, logit) over the row, each thread's indices in rising order.
template <int DT, typename F>
__device__ __forceinline__ void scan_row(const Row& r, F f) {
    const int full = r.vocab & ~7;
    for (int i = 8 * threadIdx.x; i < full; i += 8 * kThreads) {
        float v[8];
        load8<DT>(r.at + static_cast<int64_t>(i) * (DT == F32 ? 4 : 2), v);
#pragma unroll
        for (int j = 0; j < 8; ++j) f(i + j, v[j]);
    }
    if (full + static_cast<int>(threadIdx.x) < r.vocab) f(full + threadIdx.x, load_one<DT>(r.at, full + threadIdx.x));
}

template <typename T>
__device__ __forceinline__ T wave_scan(T v) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const T o = __shfl_up(v, d, 64);
        if (lane >= d) v += o;
    }
    return v;
}

// Inclusive sum over the block's threads.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T* parts) {
    v = wave_scan(v);
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 63) parts[wave] = v;
    __syncthreads();
    T before = 0;
    for (int w = 0; w < wave; ++w) before += parts[w];
    __syncthreads();
    return v + before;
}

__device__ __forceinline__ uint64_t block_max(uint64_t v, uint64_t* parts) {
#pragma unroll
    for (int d = 32; d; d /= 2) {
        const uint64_t o = __shfl_xor(v, d, 64);
        v = v > o ? v : o;
    }
    if ((threadIdx.x & 63) == 0) parts[threadIdx.x >> 6] = v;
    __syncthreads();
    v = parts[0];
    for (int w = 1; w < kWaves; ++w) v = v > parts[w] ? v : parts[w];
    __syncthreads();
    return v;
}

// Histogram (mass, count)[n] to its running sums, n <= 2048.
__device__ __forceinline__ void run_up(uint64_t* mass, uint32_t* count, int n, Shared& s) {
    const int i = 2 * threadIdx.x;
    const uint64_t m0 = i < n ? mass[i] : 0, m1 = i + 1 < n ? mass[i + 1] : 0;
    const uint32_t c0 = i < n ? count[i] : 0, c1 = i + 1 < n ? count[i + 1] : 0;
    const uint64_t m = block_scan<uint64_t>(m0 + m1, s.part64);
    const uint32_t c = block_scan<uint32_t>(c0 + c1, s.part32);
    if (i < n) {
        mass[i] = m - m1;
        count[i] = c - c1;
    }
    if (i + 1 < n) {
        mass[i + 1] = m;
        count[i + 1] = c;
    }
    __syncthreads();
}

// First bin whose running sum passes the target (some bin does).
template <typename T>
__device__ __forceinline__ int first_past(const T* run, int n, T target, Shared& s) {
    for (int i = threadIdx.x; i < n; i += kThreads)
        if (run[i] > target && (i == 0 || run[i - 1] <= target)) s.found32[0] = i;
    __syncthreads();
    const int b = s.found32[0];
    __syncthreads();
    return b;
}

// Where an order passes a target: the mass up to and with that element, and which it is.
struct Place {
    uint64_t mass;
    uint32_t key;
    int index;
};

// The first element at which the running count (BY_COUNT) or mass passes target.
// The token's index is found only with INDEX.
template <int DT, bool BY_COUNT, bool INDEX>
__device__ Place pass(const Row& r, uint64_t target, Shared& s) {
    int bin = BY_COUNT ? first_past<uint32_t>(s.count, kBins, static_cast<uint32_t>(target), s)
                       : first_past<uint64_t>(s.mass, kBins, target, s);
    uint64_t mass_before = bin ? s.mass[bin - 1] : 0;
    uint32_t count_before = bin ? s.count[bin - 1] : 0;
    uint32_t n = s.count[bin] - count_before;
    const int bin0 = bin;
    // of the bin's elements, those whose key lies in [lo, hi]
    uint32_t lo = 0, hi = 0xFFFFFFFFu;
    auto member = [&](float v, double& y) {
        y = y_of(r, v);
        if (!(y < kYEnd) || static_cast<int>(y * 32.0) != bin0) return false;
        if (mass_of(y, s.exp2_tab) < r.least) return false;
        const uint32_t k = key_of(v);
        return k >= lo && k <= hi;
    };
    if (n > kList) {
        // the range of their keys, then 2048 parts of it at a time
        uint64_t top = 0, low = 0;
        scan_row<DT>(r, [&](int, float v) {
            double y;
            if (member(v, y)) {
                const uint64_t k = key_of(v), nk = 0xFFFFFFFFu - k;
                top = top > k ? top : k;
                low = low > nk ? low : nk;
            }
        });
        hi = static_cast<uint32_t>(block_max(top, s.part64));
        lo = 0xFFFFFFFFu - static_cast<uint32_t>(block_max(low, s.part64));
    }
    while (n > kList) {
        const uint32_t range = hi - lo;
        const int shift = range < kSub ? 0 : 32 - __builtin_clz(range) - 11;
        const uint32_t start = hi;
        for (int i = threadIdx.x; i < kSub; i += kThreads) {
            s.sub.mass[i] = 0;
            s.sub.count[i] = 0;
        }
        __syncthreads();
        scan_row<DT>(r, [&](int, float v) {
            double y;
            if (member(v, y)) {
                const uint32_t b = (start - key_of(v)) >> shift;
                atomicAdd(reinterpret_cast<unsigned long long*>(&s.sub.mass[b]), mass_of(y, s.exp2_tab));
                atomicAdd(&s.sub.count[b], 1u);
            }
        });
        __syncthreads();
        run_up(s.sub.mass, s.sub.count, kSub, s);
        const int b = BY_COUNT ? first_past<uint32_t>(s.sub.count, kSub, static_cast<uint32_t>(target) - count_before, s)
                               : first_past<uint64_t>(s.sub.mass, kSub, target - mass_before, s);
        n = s.sub.count[b] - (b ? s.sub.count[b - 1] : 0);
        const uint64_t here = s.sub.mass[b] - (b ? s.sub.mass[b - 1] : 0);
        mass_before += b ? s.sub.mass[b - 1] : 0;
        count_before += b ? s.sub.count[b - 1] : 0;
        const uint32_t was_lo = lo;
        hi = start - (static_cast<uint32_t>(b) << shift);
        const uint32_t width = (1u << shift) - 1;
        lo = hi - was_lo > width ? hi - width : was_lo;
        __syncthreads();
        if (shift == 0) {
            // one key: equal weights (a weight of 0 passes no target)
            const uint64_t w = here / n;
            const uint32_t nth = BY_COUNT ? static_cast<uint32_t>(target) - count_before
                                          : static_cast<uint32_t>((target - mass_before) / w);
            Place p{mass_before + (nth + 1) * w, hi, -1};
            if (INDEX) {
                // the nth element of that key, 8192 elements at a time
                uint32_t seen = 0;
                const int full = r.vocab & ~7;
                for (int i0 = 0; i0 < r.vocab; i0 += 8 * kThreads) {
                    const int i = i0 + 8 * threadIdx.x;
                    uint32_t bits = 0;
                    if (i < full) {
                        float v[8];
                        load8<DT>(r.at + static_cast<int64_t>(i) * (DT == F32 ? 4 : 2), v);
#pragma unroll
                        for (int j = 0; j < 8; ++j) bits |= key_of(v[j]) == hi ? 1u << j : 0;
                    } else {
                        for (int j = 0; j < 8 && i + j < r.vocab; ++j) bits |= key_of(load_one<DT>(r.at, i + j)) == hi ? 1u << j : 0;
                    }
                    const uint32_t upto = seen + block_scan<uint32_t>(__popc(bits), s.part32);
                    const uint32_t before = upto - __popc(bits);
                    if (nth >= before && nth < upto) {
                        for (uint32_t k = before; k < nth; ++k) bits &= bits - 1;
                        s.found32[1] = i + __builtin_ctz(bits);
                    }
                    if (threadIdx.x == kThreads - 1) s.found32[2] = upto;
                    __syncthreads();
                    seen = s.found32[2];
                    if (seen > nth) break;
                    __syncthreads();
                }
                p.index = static_cast<int>(s.found32[1]);
                __syncthreads();
            }
            return p;
        }
    }

    // few: sorted by falling key, then rising index
    if (threadIdx.x == 0) s.found32[1] = 0;
    __syncthreads();
    scan_row<DT>(r, [&](int i, float v) {
        double y;
        if (member(v, y)) s.list[atomicAdd(&s.found32[1], 1u)] = static_cast<uint64_t>(~key_of(v)) << 32 | static_cast<uint32_t>(i);
    });
    __syncthreads();
    int pow2 = 64;
    while (pow2 < static_cast<int>(n)) pow2 *= 2;
    for (int i = n + threadIdx.x; i < pow2; i += kThreads) s.list[i] = ~0ull;
    __syncthreads();
    for (int k = 2; k <= pow2; k *= 2)
        for (int j = k / 2; j; j /= 2) {
            for (int e = threadIdx.x; e < pow2 / 2; e += kThreads) {
                const int a = 2 * e - (e & (j - 1)), b = a + j;      // bit j of a is clear
                const uint64_t x = s.list[a], z = s.list[b];
                if ((x > z) == ((a & k) == 0)) {
                    s.list[a] = z;
                    s.list[b] = x;
                }
            }
            __syncthreads();
        }
    const int i = 2 * threadIdx.x;
    uint64_t w[2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
        w[j] = i + j < static_cast<int>(n) ? mass_of(y_of(r, logit_of(~static_cast<uint32_t>(s.list[i + j] >> 32))), s.exp2_tab) : 0;
    uint64_t run = mass_before + block_scan<uint64_t>(w[0] + w[1], s.part64) - w[0] - w[1];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const uint64_t next = run + w[j];
        const bool here = BY_COUNT ? count_before + i + j == target : run <= target && next > target;
        if (i + j < static_cast<int>(n) && here) {
            s.found64[0] = next;
            s.found64[1] = s.list[i + j];
        }
        run = next;
    }
    __syncthreads();
    Place p{s.found64[0], ~static_cast<uint32_t>(s.found64[1] >> 32), static_cast<int>(static_cast<uint32_t>(s.found64[1]))};
    __syncthreads();
    return p;
}

// floor(f * m), f in [0, 1) given in units of 2^-48; *exact: nothing was cut off.
__device__ __forceinline__ uint64_t part_of(uint64_t f48, uint64_t m, bool* exact) {
    const uint64_t hi = __umul64hi(f48, m), lo = f48 * m;
    *exact = (lo & 0xFFFFFFFFFFFFull) == 0;
    return hi << 16 | lo >> 48;
}

template <int DT>
__global__ __launch_bounds__(kThreads) void sample_kernel(SampleArgs a) {
    __shared__ Shared s;
    const int row = blockIdx.x, t = threadIdx.x;
    Row r;
    r.at = static_cast<const char*>(a.logits) + static_cast<int64_t>(row) * a.ld * (DT == F32 ? 4 : 2);
    r.vocab = a.vocab;

    // the largest logit, and the first that has it
    uint64_t best = 0;
    uint32_t best_key = kKeyNone;
    int best_at = 0;
    scan_row<DT>(r, [&](int i, float v) {
        const uint32_t k = key_of(v);
        if (k > best_key) {
            best_key = k;
            best_at = i;
        }
    });
    best = static_cast<uint64_t>(best_key) << 32 | (0xFFFFFFFFu - static_cast<uint32_t>(best_at));
    best = block_max(best, s.part64);
    best_key = static_cast<uint32_t>(best >> 32);
    best_at = static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(best));
    if (best_key == kKeyNone) {
        if (t == 0) {
            a.token[row] = -1;
            if (a.logprob) a.logprob[row] = __builtin_nanf("");
        }
        return;
    }
    const float temp = a.temperature ? a.temperature[row] : 1.f;
    if (!(temp > 0.f)) {
        if (t == 0) {
            a.token[row] = best_at;
            if (a.logprob) a.logprob[row] = 0.f;
        }
        return;
    }
    r.top = logit_of(best_key);
    r.scale = 1.4426950408889634 / static_cast<double>(temp);
    const float min_p = a.min_p ? a.min_p[row] : 0.f;
    r.least = !(min_p > 0.f) ? 0 : min_p >= 1.f ? kOne : static_cast<uint64_t>(ceil(static_cast<double>(min_p) * 0x1p44));

    for (int i = t; i < 1024; i += kThreads) s.exp2_tab[i] = exp2(-i / 1024.0);
    for (int i = t; i < kBins; i += kThreads) {
        s.mass[i] = 0;
        s.count[i] = 0;
    }
    __syncthreads();
    scan_row<DT>(r, [&](int, float v) {
        const double y = y_of(r, v);
        if (!(y < kYEnd)) return;            // (a NaN too)
        const uint64_t w = mass_of(y, s.exp2_tab);
        if (w < r.least) return;
        const int b = static_cast<int>(y * 32.0);
        atomicAdd(reinterpret_cast<unsigned long long*>(&s.mass[b]), w);
        atomicAdd(&s.count[b], 1u);
    });
    __syncthreads();
    run_up(s.mass, s.count, kBins, s);

    uint64_t mass = s.mass[kBins - 1];
    const uint32_t all = s.count[kBins - 1];
    const float top_p = a.top_p ? a.top_p[row] : 1.f;
    int64_t k = a.top_k ? a.top_k[row] : 0;
    if (top_p <= 0.f) k = 1;
    if (k > 0 && k < all) mass = pass<DT, true, false>(r, static_cast<uint64_t>(k - 1), s).mass;
    bool exact;
    if (top_p > 0.f && top_p < 1.f) {
        // kept: the tokens before which less than top_p of the mass lies
        const uint64_t f = part_of(static_cast<uint64_t>(static_cast<double>(top_p) * 0x1p48), mass, &exact);
        mass = pass<DT, false, false>(r, exact && f ? f - 1 : f, s).mass;
    }
    const float u = a.u[row];
    const uint64_t u48 = !(u > 0.f) ? 0 : u >= 1.f ? (1ull << 48) - 1 : static_cast<uint64_t>(static_cast<double>(u) * 0x1p48);
    const Place p = pass<DT, false, true>(r, part_of(u48, mass, &exact), s);
    if (t == 0) {
        a.token[row] = p.index;
        if (a.logprob)
            a.logprob[row] = static_cast<float>(-y_of(r, logit_of(p.key)) * 0.6931471805599453 - log(static_cast<double>(mass) * 0x1p-44));
    }
}

}  // namespace

hipError_t launch_sample(const SampleArgs& a, int dtype, void* ws, hipStream_t st) {
    (void)ws;
    const dim3 grid(static_cast<unsigned>(a.rows));
    if (dtype == F16) sample_kernel<F16><<<grid, kThreads, 0, st>>>(a);
    else if (dtype == BF16) sample_kernel<BF16><<<grid, kThreads, 0, st>>>(a);
    else sample_kernel<F32><<<grid, kThreads, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace qlin
