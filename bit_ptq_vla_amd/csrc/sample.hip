// A token from each row of logits, for gfx950: temperature, min-p, top-k, top-p
// and a given random number.
//
//   w_i = exp((l_i - max) / t); in the order of falling logits (the lowest index
//   first among equals) the kept tokens are a prefix, and the token is its first
//   whose running mass passes u times the prefix's mass.
//
// With a = 32 log2(e) l / t a token lies in bin rint(a), 32 of them to a factor of
// two, and its mass is 2^44 2^((a - rint(a)) / 32), an integer: bins do not depend on
// the row's maximum, so one pass over the row fills them without knowing it, and
// integer sums have no order: any split of a row over threads and blocks, and any
// order of their atomics, gives the same token.  The 64 octaves below the largest bin
// count (what lies lower weighs less than 2^-63 of it, all of it together less than
// 2^-45).  a - rint(a) is one fused product in float64, exact but for its last
// rounding, and the mass is evaluated in float64 to 2^-46 of itself.
//
// How far sums are off, in units of 2^-44 of the largest weight, of which a row's mass
// has 2^44 at least: bins come to the largest one's units with 20 bits behind the
// point, listed elements with 9, so that what 2048 bins or 512 elements cut off is one
// unit; a target, a bin's share of it and the mass behind a filter are rounded to one
// each.  With a weight's own rounding, 2^-44 of itself, a filter and the token are
// decided as exact weights decide them unless top_p or u lies within 2^-40 of a border.
//
// Each filter, and the token itself, is one question: the first element of the
// order at which the running count, or mass, passes a target.  The bins' running
// sums leave one bin; its keys (logits as ordered integers) are a range, found by a
// search over keys, and the few elements in it are listed in LDS.  Where they are
// many (flat rows, equal logits) histograms over the keys narrow them down; equal
// logits have equal masses, so among them the place is a division.  Where the filters
// leave few elements, those are listed once and every question is answered there, each
// element at its rank; a min-p, or a small top-k (by a histogram of counts), tells so
// before any mass is computed.
//
// A block takes a row, or a part of one where rows are few (the parts' bins then
// meet in a second launch).
//
// Bound by waiting: the pass that fills the bins takes about 25 vector instructions and
// an LDS atomic (two with a top-k) to a logit, and a chain of scans and barriers follows,
// 10 to 20 us.  1024 rows of 32003 bf16 logits with mixed filters (66 MB) take 51 us,
// vector units 28% busy, waves waiting 59% of their time; 256 of 257152 fp32 logits
// without any (263 MB, read again for the last bin) 133, two waves to a SIMD, 34% and 57%,
// 5.9 conflict cycles to an LDS instruction; one of 32000 21.

#include "device_common.h"
#include "qlin_internal.h"
#include "sample_keys.h"

namespace qlin {

namespace {

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / 64;
constexpr int kSlots = 2048;             // of the ring of bins
constexpr int kBins = kSampleBins;       // 64 octaves: every slot of the ring
constexpr int kSub = 2048;               // bins of a histogram over keys
constexpr int kList = 1408;              // elements that are listed at once (two blocks fill a CU's LDS)
constexpr int kNear = 512;               // of them, that are all ranked
constexpr int kFew = 64;                 // of them, that answer one question
constexpr int kFine = 9;                 // bits of listed elements' masses behind a unit (kNear of them stay below 2^63)
constexpr uint64_t kOne = 1ull << 44;
static_assert(kBins == kSlots, "the window is the ring");

// The thread's number, new to the compiler at every use: it would otherwise compute what
// follows from it for all the phases of a row at once, and spill 70 registers.
__device__ __forceinline__ int thread() {
    int t = threadIdx.x;
    asm volatile("" : "+v"(t));
    return t;
}

// A value that all lanes hold, in scalar registers.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __builtin_amdgcn_readfirstlane(static_cast<int>(x)); }
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ float uniform(float x) { return __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(x))); }
__device__ __forceinline__ uint64_t uniform(uint64_t x) {
    return static_cast<uint64_t>(uniform(static_cast<uint32_t>(x >> 32))) << 32 | uniform(static_cast<uint32_t>(x));
}
__device__ __forceinline__ double uniform(double x) {
    return __longlong_as_double(static_cast<long long>(uniform(static_cast<uint64_t>(__double_as_longlong(x)))));
}

struct Scale {
    double c;           // 32 log2(e) / t
    double top;         // kMagic + the largest bin
    // The largest bin is so far from 0 (an infinite logit, a tiny temperature) that only
    // the largest logit itself lies in the window: all else weighs nothing.
    bool lone;
    float top_logit;
};
constexpr double kMagic = 0x1.8p52;     // x + kMagic: rint(x) in the low bits of the significand

// kMagic + the bin of a logit (below 2^51 either side).
__device__ __forceinline__ double bin_at(const Scale& s, float v) { return fma(static_cast<double>(v), s.c, kMagic); }
__device__ __forceinline__ int slot_of(double bin) {
    return static_cast<int>(__double_as_longlong(bin)) & (kSlots - 1);
}
// 2^44 2^(f / 32), |f| <= 1/2, rounded to an integer: the exponential's series, what is
// left out is below 2^-48 of it; the added 2^52 leaves the integer in the significand.
struct Series {
    double c5, c4, c3, c2, c1, c0;
    __device__ __forceinline__ Series() {
        constexpr double z = 0.69314718055994530942 / 32;
        c0 = 0x1p52 + 0x1p44;
        c1 = 0x1p44 * z;
        c2 = 0x1p44 * z * z / 2;
        c3 = 0x1p44 * z * z * z / 6;
        c4 = 0x1p44 * z * z * z * z / 24;
        c5 = 0x1p44 * z * z * z * z * z / 120;
        // scalar registers: an addend of a product there needs no copy
        asm("" : "+s"(c0), "+s"(c1), "+s"(c2), "+s"(c3), "+s"(c4));
    }
    __device__ __forceinline__ uint64_t operator()(double f) const {
        const double p = fma(fma(fma(fma(fma(c5, f, c4), f, c3), f, c2), f, c1), f, c0);
        return static_cast<uint64_t>(__double_as_longlong(p)) & 0xFFFFFFFFFFFFFull;
    }
};
__device__ __forceinline__ uint64_t mass_in(const Series& series, const Scale& s, float v, double bin) {
    return series(fma(static_cast<double>(v), s.c, kMagic - bin));
}
// Of a logit in the window.
__device__ __forceinline__ uint64_t mass_of(const Scale& s, float v) {
    return s.lone ? v == s.top_logit ? kOne : 0 : mass_in(Series(), s, v, bin_at(s, v));
}
// How far below the largest bin, to 63 octaves.
__device__ __forceinline__ int depth_of(const Scale& s, float v) {
    const double d = s.lone ? 0.0 : s.top - bin_at(s, v);
    return static_cast<int>(d < 2047.0 ? d : 2047.0);
}
__device__ __forceinline__ void set_top(Scale& s, float v) {
    s.top_logit = uniform(v);
    s.top = uniform(bin_at(s, v));
    s.lone = !(fabs(s.top - kMagic) < 0x1p40);
    if (s.lone) s.top = kMagic;
}

__device__ __forceinline__ bool counts(const SampleArgs& a, int row) {
    return a.top_k && a.top_k[row] > 0 && a.top_k[row] < a.vocab;
}

__device__ __forceinline__ Scale scale_of(float temp) {
    Scale sc{uniform(46.166241308446828384 / static_cast<double>(temp)), kMagic, false, 0.f};
    if (sc.c < 1e-300) sc.c = 1e-300;               // (an infinite temperature: equal weights)
    return sc;
}

// A word of memory behind a pointer that is known to be global: a load that might go
// anywhere waits for all that are on their way.
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef const __attribute__((address_space(1))) u4* GlobalWords;
__device__ const u4 kNoWord = {0, 0, 0, 0};        // (of a row that is shorter than a word)

template <int DT>
struct Sampler {
    struct Shared {
        uint64_t mass[kSlots + 64];          // of a bin, in the ring
        uint32_t count[kSlots + 64];
        uint64_t run_mass[kBins];            // running sums from the largest bin down, in its units
        uint32_t run_count[kBins];           // (where nothing counts: no fewer, about a hundredth more)
        union {
            struct {
                uint64_t mass[kSub];
                uint32_t count[kSub];
            } sub;
            struct {
                uint64_t order[kList + 8];   // falling key, then rising index
                uint64_t mass[kList + 8];
                union {
                    struct {
                        uint64_t mass[kThreads];
                        uint32_t count[kThreads];
                        uint64_t few_order[kFew + 8], few_mass[kFew + 8];
                    } part;
                    struct {
                        uint64_t order[kNear], ahead[kNear];
                    } sorted;
                };
            } list;
        };
        uint64_t down[32];                   // 2^63 2^(-i / 32)
        double up[32];                       // 2^(i / 32)
        int offset[kMaxSampleParts];
        uint64_t part64[kWaves];
        uint32_t part32[kWaves];
        uint64_t found64[2];
        uint32_t found32[4];
    };

    // 16-byte words of a row in a thread's registers: element e of word j is index
    // first + (512 j + thread) N + e, -infinity past the end.
    struct Chunk {
        static constexpr int N = DT == F32 ? 4 : 8;
        static constexpr int kWords = 4;
        static constexpr int kSize = kThreads * N * kWords;
        uint4 w[kWords];

        __device__ __forceinline__ static int index(int first, int j, int e) {
            return first + (kThreads * j + thread()) * N + e;
        }
        // The word at element i, of which all that lies below end was loaded if that was all of
        // it; -infinity from the end on.
        __device__ __forceinline__ static uint4 ended(uint4 loaded, const char* row, int i, int end) {
            constexpr uint32_t none = DT == F32 ? 0xFF800000u : DT == BF16 ? 0xFF80FF80u : 0xFC00FC00u;
            if (i + N <= end) return loaded;
            uint32_t x[4] = {none, none, none, none};
            if (i < end) {
#pragma unroll
                for (int e = 0; e < N - 1; ++e) {
                    if (i + e >= end) continue;
                    if constexpr (DT == F32) {
                        x[e] = reinterpret_cast<const uint32_t*>(row)[i + e];
                    } else {
                        const uint32_t b = reinterpret_cast<const uint16_t*>(row)[i + e];
                        x[e / 2] = e & 1 ? (x[e / 2] & 0xFFFFu) | b << 16 : (x[e / 2] & 0xFFFF0000u) | b;
                    }
                }
            }
            return make_uint4(x[0], x[1], x[2], x[3]);
        }
        // (loads that every thread makes, whatever the row's end: behind one that may not be
        // made, all that are on their way would be waited for)
        template <typename R>
        __device__ __forceinline__ void load(const R& row, int first) {
#pragma unroll
            for (int j = 0; j < kWords; ++j) w[j] = row.word((index(first, j, 0) - row.from) / N);
        }
        template <typename R>
        __device__ __forceinline__ void end(const R& row, int first) {
            if (first + kSize <= row.to) return;
#pragma unroll
            for (int j = 0; j < kWords; ++j) w[j] = ended(w[j], row.at, index(first, j, 0), row.to);
        }
        __device__ __forceinline__ static float value(uint4 word, int e) {
            const uint32_t x[4] = {word.x, word.y, word.z, word.w};
            if constexpr (DT == F32) return __uint_as_float(x[e]);
            if constexpr (DT == BF16) return __uint_as_float(e & 1 ? x[e / 2] & 0xFFFF0000u : x[e / 2] << 16);
            return f16_bits_to_f32(static_cast<uint16_t>(e & 1 ? x[e / 2] >> 16 : x[e / 2] & 0xFFFFu));
        }
        // The same for an element that is known late.
        __device__ __forceinline__ static float value_late(uint4 word, int e) {
            const int at = e / (N / 4);
            const uint32_t lo = at & 1 ? word.y : word.x, hi = at & 1 ? word.w : word.z, x = at & 2 ? hi : lo;
            if constexpr (DT == F32) return __uint_as_float(x);
            if constexpr (DT == BF16) return __uint_as_float(e & 1 ? x & 0xFFFF0000u : x << 16);
            return f16_bits_to_f32(static_cast<uint16_t>(e & 1 ? x >> 16 : x & 0xFFFFu));
        }
        template <typename F>
        __device__ __forceinline__ void words(F f) const {
#pragma unroll
            for (int j = 0; j < kWords; ++j) f(w[j]);
        }
    };

    // A row, or a part of it.
    struct Row {
        const char* at;
        int from, to;
        GlobalWords whole;           // its whole words, and how many follow the first
        uint32_t more;
        __device__ __forceinline__ Row(const char* at_, int from_, int to_) : at(at_), from(from_), to(to_) {
            const bool any = to - from >= Chunk::N;
            whole = any ? (GlobalWords)(at + static_cast<int64_t>(from) * (16 / Chunk::N)) : (GlobalWords)&kNoWord;
            more = any ? (to - from) / Chunk::N - 1 : 0;
        }
        // The word of that number, the last whole one behind it.
        __device__ __forceinline__ uint4 word(int number) const {
            const uint32_t n = static_cast<uint32_t>(number);
            const u4 w = whole[n < more ? n : more];
            return make_uint4(w[0], w[1], w[2], w[3]);
        }
        // f(index of its first element, word) for the thread's words, two more on their way:
        // from the first on, or from the last, whose words a pass before left in the caches.
        // (In pairs that start together: one load at a time, four ahead, read 263 MB again in
        // 40 us where this takes 30.)
        template <bool BACK, typename F>
        __device__ __forceinline__ void words_to(F f) const {
            constexpr int step = kThreads * Chunk::N, AHEAD = 2;
            const int n = (to - from + step - 1) / step, t = thread();
            auto number = [&](int k) { return (BACK ? n - 1 - k : k) * kThreads + t; };
            uint4 w[AHEAD], next[AHEAD];
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) w[j] = word(number(j));
            for (int k = 0; k < n; k += AHEAD) {
#pragma unroll
                for (int j = 0; j < AHEAD; ++j) next[j] = word(number(k + j + AHEAD));
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int j = 0; j < AHEAD; ++j) {
                    if (k + j >= n) break;
                    const int i = from + number(k + j) * Chunk::N;
                    f(i, Chunk::ended(w[j], at, i, to));
                }
#pragma unroll
                for (int j = 0; j < AHEAD; ++j) w[j] = next[j];
            }
        }
        template <typename F>
        __device__ __forceinline__ void words(F f) const { words_to<false>(f); }
        template <typename F>
        __device__ __forceinline__ void words_back(F f) const { words_to<true>(f); }
    };

    // Inclusive sum over the block's threads.
    template <typename T>
    static __device__ __forceinline__ T block_scan(T v, T* parts) {
        v = wave_sum_up(v);
        const int wave = thread() >> 6;
        if ((thread() & 63) == 63) parts[wave] = v;
        __syncthreads();
        T before = 0;
#pragma unroll
        for (int w = 0; w < kWaves - 1; ++w) before += w < wave ? parts[w] : 0;
        __syncthreads();
        return v + before;
    }

    template <typename T>
    static __device__ __forceinline__ T block_max(T v, T* parts) {
        auto more = [](T a, T b) { return a > b ? a : b; };
        v = more(v, dpp_u<0x111, 0xF>(v));
        v = more(v, dpp_u<0x112, 0xF>(v));
        v = more(v, dpp_u<0x114, 0xF>(v));
        v = more(v, dpp_u<0x118, 0xF>(v));
        v = more(v, dpp_u<0x142, 0xA>(v));
        v = more(v, dpp_u<0x143, 0xC>(v));
        if ((thread() & 63) == 63) parts[thread() >> 6] = v;
        __syncthreads();
        v = parts[0];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) v = more(v, parts[w]);
        __syncthreads();
        return uniform(v);
    }

    // Running sums of mass and count [kThreads * PER], from f(i, mass, count) to g(i, ..).
    template <int PER, typename C, typename F, typename G>
    static __device__ __forceinline__ void run_up(uint64_t* parts64, C* parts, F f, G g) {
        uint64_t m[PER], mass = 0;
        C c[PER], count = 0;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            f(PER * thread() + j, m[j], c[j]);
            mass += m[j];
            count += c[j];
        }
        uint64_t before = block_scan(mass, parts64) - mass;
        C ahead = block_scan(count, parts) - count;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            before += m[j];
            ahead += c[j];
            g(PER * thread() + j, before, ahead);
        }
        __syncthreads();
    }

    // First of the N bins whose running sum passes the target (some bin does).
    template <int N, typename T>
    static __device__ __forceinline__ int first_past(const T* run, T target, Shared& s) {
        const int t = thread();
#pragma unroll
        for (int j = 0; j < (N + kThreads - 1) / kThreads; ++j) {
            const int i = t + kThreads * j, at = i < N ? i : N - 1;
            const T before = run[at > 0 ? at - 1 : 0];
            if (i < N && run[at] > target && (i == 0 || before <= target)) s.found32[0] = i;
        }
        __syncthreads();
        const int b = uniform(s.found32[0]);
        __syncthreads();
        return b;
    }

    // The smallest key in (kKeyNone, top] for which holds() is true (it stays true from
    // there on, and holds for top), by the 64 lanes of a wave.
    template <typename F>
    static __device__ __forceinline__ uint32_t first_key(uint32_t top, F holds) {
        uint32_t lo = kKeyNone, hi = top;                // not at lo, at hi
        while (hi - lo > 1) {
            const uint32_t step = (hi - lo - 1) / 64 + 1;
            const uint64_t at = static_cast<uint64_t>(lo) + static_cast<uint64_t>(step) * ((thread() & 63) + 1);
            const uint64_t votes = __ballot(at >= hi || holds(static_cast<uint32_t>(at)));
            const uint32_t n = __builtin_ctzll(votes);   // (the last lane is at hi or behind it)
            const uint64_t next = static_cast<uint64_t>(lo) + static_cast<uint64_t>(step) * (n + 1);
            lo += step * n;
            hi = next < hi ? static_cast<uint32_t>(next) : hi;
        }
        return hi;
    }

    // m (below 2^63) in units of a bin i below the largest, in those of the largest: whole
    // ones, and 2^-20 of them; and back.
    struct Mass {
        uint64_t whole;
        uint32_t part;
    };
    static __device__ __forceinline__ Mass to_top(uint64_t m, int i, const Shared& s) {
        const uint64_t down = s.down[i & 31], lo = m * down, hi = __umul64hi(m, down) << 1 | lo >> 63;
        const int k = i >> 5;
        const uint64_t rest = k ? hi << (64 - k) | lo << 1 >> k : lo << 1;
        return {hi >> k, static_cast<uint32_t>(rest >> 44)};
    }
    static __device__ __forceinline__ uint64_t from_top(uint64_t m, int i, uint64_t most, const Shared& s) {
        if (i == 0) return m;
        const double x = ldexp(static_cast<double>(m) * s.up[i & 31], i >> 5);   // (2^-52 of it is far below what bins round)
        return x < static_cast<double>(most) ? static_cast<uint64_t>(x) : most;
    }

    // f(index, value) for the elements with keys from lo_key to hi_key.
    template <typename F>
    static __device__ __forceinline__ void in_range(const Row& row, uint32_t lo_key, uint32_t hi_key, F f) {
        const float lo = logit_of(lo_key), hi = logit_of(hi_key);
        auto in = [&](uint4 word, int e) {
            const float v = Chunk::value(word, e);
            return __builtin_amdgcn_fmed3f(v, lo, hi) == v;
        };
        row.words_back([&](int i0, uint4 word) {
            bool any = false;
#pragma unroll
            for (int e = 0; e < Chunk::N; ++e) any |= in(word, e);
            if (!__any(any)) return;
            uint32_t bits = 0;
#pragma unroll
            for (int e = 0; e < Chunk::N; ++e) bits |= in(word, e) ? 1u << e : 0;
            while (bits) {
                const int e = __builtin_ctz(bits);
                f(i0 + e, Chunk::value_late(word, e));
                bits &= bits - 1;
            }
        });
    }

    // How many of the n elements come before one, and their mass.  The arrays hold
    // room for 7 more.
    static __device__ __forceinline__ void rank_of(uint64_t mine, const uint64_t* order, const uint64_t* mass, uint32_t n, uint32_t& rank,
                                            uint64_t& ahead) {
        rank = 0;
        ahead = 0;
        for (uint32_t e0 = 0; e0 < n; e0 += 8) {
            uint64_t o[8], m[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                o[e] = order[e0 + e];
                m[e] = mass[e0 + e];
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const bool first = o[e] < mine && e0 + e < n;
                ahead += first ? m[e] : 0;
                rank += first;
            }
        }
    }

    using Range = KeyRange;
    // Keys of the bin i below the largest.
    static __device__ __forceinline__ Range keys_of(const Scale& sc, uint32_t top_key, int i, Shared& s) {
        if (sc.lone) return {top_key, top_key};
        const int wave = thread() >> 6;
        if (wave < 2) {
            const double bin = sc.top - i + wave;        // (behind bin 0's keys there are none)
            const uint32_t k = first_key(top_key, [&](uint32_t key) { return bin_at(sc, logit_of(key)) >= bin; });
            if ((thread() & 63) == 0) s.found32[wave] = k;
        }
        __syncthreads();
        const Range range{uniform(s.found32[0]), i == 0 ? top_key : uniform(s.found32[1]) - 1};
        __syncthreads();
        return range;
    }

    // Mass and count of the elements with keys in the range.
    static __device__ __forceinline__ void sum_of(const Row& row, const Scale& sc, Range range, Shared& s, uint64_t& mass,
                                           uint32_t& count) {
        uint64_t m = 0;
        uint32_t n = 0;
        in_range(row, range.lo, range.hi, [&](int, float v) {
            m += mass_of(sc, v);
            ++n;
        });
        m = block_scan(m, s.part64);
        n = block_scan(n, s.part32);
        if (thread() == kThreads - 1) {
            s.found64[0] = m;
            s.found32[0] = n;
        }
        __syncthreads();
        mass = uniform(s.found64[0]);
        count = uniform(s.found32[0]);
        __syncthreads();
    }

    // Lists the elements with keys in the range: their orders and masses (in their bins'
    // units).  Returns how many there are; past kList only some are listed.
    static __device__ __forceinline__ uint32_t list_range(const Row& row, const Scale& sc, Range range, Shared& s) {
        if (thread() == 0) s.found32[1] = 0;
        __syncthreads();
        in_range(row, range.lo, range.hi, [&](int i, float v) {
            const uint32_t n = atomicAdd(&s.found32[1], 1u);
            if (n < kList) s.list.order[n] = static_cast<uint64_t>(~key_of(v)) << 32 | static_cast<uint32_t>(i);
        });
        __syncthreads();
        const uint32_t n = uniform(s.found32[1]);
        for (uint32_t e = thread(); e < n && e < kList; e += kThreads)
            s.list.mass[e] = mass_of(sc, logit_of(~static_cast<uint32_t>(s.list.order[e] >> 32)));
        __syncthreads();
        return n;
    }

    // Of the list's n elements the one at which the running count or mass passes left:
    // its order is in s.found64[1], the mass up to and with it in [0]; returns the mass
    // of those left out before.  While there are many, 512 parts of their range at a time.
    static __device__ __forceinline__ uint64_t of_list(bool by_count, uint64_t left, uint32_t n, Shared& s) {
        const uint32_t t = thread(), all = n;
        uint64_t lo = 0, hi = ~0ull, passed = 0;
        while (n > kFew) {
            uint64_t most = 0, least = 0;            // (the least by its complement)
            for (uint32_t e = t; e < all; e += kThreads) {
                const uint64_t o = s.list.order[e];
                if (o < lo || o > hi) continue;
                most = o > most ? o : most;
                least = ~o > least ? ~o : least;
            }
            hi = block_max(most, s.part64);
            lo = ~block_max(least, s.part64);
            const uint64_t width = hi - lo;
            const int shift = width < kThreads ? 0 : 64 - __builtin_clzll(width) - __builtin_ctz(kThreads);
            s.list.part.mass[t] = 0;
            s.list.part.count[t] = 0;
            __syncthreads();
            for (uint32_t e = t; e < all; e += kThreads) {
                const uint64_t o = s.list.order[e];
                if (o < lo || o > hi) continue;
                const uint32_t b = static_cast<uint32_t>((o - lo) >> shift);
                atomicAdd(reinterpret_cast<unsigned long long*>(&s.list.part.mass[b]), s.list.mass[e]);
                atomicAdd(&s.list.part.count[b], 1u);
            }
            __syncthreads();
            const uint64_t m = s.list.part.mass[t];
            const uint32_t c = s.list.part.count[t];
            const uint64_t mass = block_scan(m, s.part64);
            const uint32_t count = block_scan(c, s.part32);
            if (by_count ? count > left && count - c <= left : mass > left && mass - m <= left) {
                s.found64[0] = mass - m;
                s.found32[0] = count - c;
                s.found32[2] = c;
                s.found32[3] = t;
            }
            __syncthreads();
            passed += uniform(s.found64[0]);
            left -= by_count ? uniform(s.found32[0]) : uniform(s.found64[0]);
            n = uniform(s.found32[2]);
            lo += static_cast<uint64_t>(uniform(s.found32[3])) << shift;
            const uint64_t part = (1ull << shift) - 1;
            hi = hi - lo > part ? lo + part : hi;
            __syncthreads();
        }
        if (t == 0) s.found32[0] = 0;
        __syncthreads();
        for (uint32_t e = t; e < all; e += kThreads) {
            const uint64_t o = s.list.order[e];
            if (o < lo || o > hi) continue;
            const uint32_t at = atomicAdd(&s.found32[0], 1u);
            s.list.part.few_order[at] = o;
            s.list.part.few_mass[at] = s.list.mass[e];
        }
        __syncthreads();
        if (t < n) {
            const uint64_t mine = s.list.part.few_order[t], m = s.list.part.few_mass[t];
            uint64_t ahead;
            uint32_t rank;
            rank_of(mine, s.list.part.few_order, s.list.part.few_mass, n, rank, ahead);
            if (by_count ? rank == left : ahead <= left && left < ahead + m) {
                s.found64[0] = ahead + m;
                s.found64[1] = mine;
            }
        }
        __syncthreads();
        return passed;
    }

    // The part (of 2048) of the range in which the running count or mass passes left: the
    // range becomes that part, and what comes before it in the range moves from left to
    // passed (the mass).  Returns true where the part is a single key: nth is then the
    // place among its elements, one their mass.
    static __device__ __forceinline__ bool narrow(const Row& row, const Scale& sc, bool by_count, Range& range, uint64_t& left,
                                           uint64_t& passed, uint32_t& nth, uint64_t& one, Shared& s) {
        const uint32_t width = range.hi - range.lo;
        const int shift = width < kSub ? 0 : 21 - __builtin_clz(width);
        for (int i = thread(); i < kSub; i += kThreads) {
            s.sub.mass[i] = 0;
            s.sub.count[i] = 0;
        }
        __syncthreads();
        in_range(row, range.lo, range.hi, [&](int, float v) {
            const uint32_t b = (range.hi - key_of(v)) >> shift;
            atomicAdd(reinterpret_cast<unsigned long long*>(&s.sub.mass[b]), mass_of(sc, v));
            atomicAdd(&s.sub.count[b], 1u);
        });
        __syncthreads();
        run_up<kSub / kThreads>(
            s.part64, s.part32,
            [&](int i, uint64_t& m, uint32_t& c) {
                m = s.sub.mass[i];
                c = s.sub.count[i];
            },
            [&](int i, uint64_t m, uint32_t c) {
                s.sub.mass[i] = m;
                s.sub.count[i] = c;
            });
        const int b = by_count ? first_past<kSub>(s.sub.count, static_cast<uint32_t>(left), s)
                               : first_past<kSub>(s.sub.mass, left, s);
        const uint64_t mass_b = b ? uniform(s.sub.mass[b - 1]) : 0, mass_here = uniform(s.sub.mass[b]) - mass_b;
        const uint32_t count_b = b ? uniform(s.sub.count[b - 1]) : 0, count_here = uniform(s.sub.count[b]) - count_b;
        passed += mass_b;
        left -= by_count ? count_b : mass_b;
        range = part_of_range(range, shift, static_cast<uint32_t>(b));
        __syncthreads();
        if (range.lo != range.hi) return false;
        one = mass_here / count_here;
        nth = static_cast<uint32_t>(by_count ? left : left / one);
        return true;
    }

    // Index of the nth element with that key.
    static __device__ __forceinline__ int nth_of(const Row& row, uint32_t key, uint32_t nth, Shared& s) {
        constexpr int N = Chunk::N;
        uint32_t seen = 0;
        row.words([&](int i0, uint4 word) {
            if (seen > nth) return;
            uint32_t bits = 0;
#pragma unroll
            for (int e = 0; e < N; ++e) bits |= key_of(Chunk::value(word, e)) == key ? 1u << e : 0;
            const uint32_t here = __popc(bits), upto = seen + block_scan(here, s.part32);
            if (nth >= upto - here && nth < upto) {
                for (uint32_t k = upto - here; k < nth; ++k) bits &= bits - 1;
                s.found32[1] = i0 + __builtin_ctz(bits);
            }
            if (thread() == kThreads - 1) s.found32[2] = upto;
            __syncthreads();
            seen = uniform(s.found32[2]);
            __syncthreads();
        });
        const int i = uniform(static_cast<int>(s.found32[1]));
        __syncthreads();
        return i;
    }

    // floor(f * m), f in [0, 1) given in units of 2^-48; *exact: nothing was cut off.
    static __device__ __forceinline__ uint64_t part_of(uint64_t f48, uint64_t m, bool* exact) {
        const uint64_t hi = __umul64hi(f48, m), lo = f48 * m;
        *exact = (lo & 0xFFFFFFFFFFFFull) == 0;
        return hi << 16 | lo >> 48;
    }

    // Bins of the elements from row.from to row.to into s and the largest of them into
    // sc; the largest key (kKeyNone: no element).
    static __device__ __forceinline__ uint32_t fill_bins(const Row& row, bool with_count, Scale& sc, Shared& s) {
        constexpr int N = Chunk::N;
        for (int i = thread(); i < kSlots; i += kThreads) {
            s.mass[i] = 0;
            s.count[i] = 0;
        }
        uint32_t top_key = kKeyNone;
        Chunk c;
        c.load(row, row.from);
        for (int from = row.from; from < row.to; from += Chunk::kSize) {
            Chunk next;
            next.load(row, from + Chunk::kSize);                 // on its way meanwhile
            c.end(row, from);
            float most = -__builtin_inff();
            c.words([&](uint4 word) {
#pragma unroll
                for (int e = 0; e < N; ++e) most = fmaxf(most, Chunk::value(word, e));     // (a NaN is passed over)
            });
            const uint32_t k = block_max(key_of(most), s.part32);
            if (k > top_key) {
                const Scale was = sc;
                set_top(sc, logit_of(k));
                const double rise = sc.top - was.top;
                if (top_key != kKeyNone) {
                    if (sc.lone || was.lone || rise >= kSlots) {     // far above all before: the ring starts anew
                        for (int i = thread(); i < kSlots; i += kThreads) {
                            s.mass[i] = 0;
                            s.count[i] = 0;
                        }
                    } else {                                         // slots between hold bins 64 octaves lower
                        for (int i = thread(); i < static_cast<int>(rise); i += kThreads) {
                            s.mass[slot_of(was.top + 1 + i)] = 0;
                            s.count[slot_of(was.top + 1 + i)] = 0;
                        }
                    }
                }
                top_key = k;
                __syncthreads();
            }
            if (top_key == kKeyNone) {
                // nothing yet
            } else if (sc.lone) {
                c.words([&](uint4 word) {
#pragma unroll
                    for (int e = 0; e < N; ++e)
                        if (Chunk::value(word, e) == sc.top_logit) {
                            atomicAdd(reinterpret_cast<unsigned long long*>(&s.mass[slot_of(kMagic)]), kOne);
                            if (with_count) atomicAdd(&s.count[slot_of(kMagic)], 1u);
                        }
                });
            } else {
                // (what lies below the window goes to slots of its own: no branch keeps the
                // elements' arithmetic apart)
                const double least = sc.top - kBins;
                const int none = kSlots + static_cast<int>(thread() & 63);
                const Series series;
                c.words([&](uint4 word) {
                    int slot[N];
#pragma unroll
                    for (int e = 0; e < N; ++e) {
                        const float v = Chunk::value(word, e);
                        const double bin = bin_at(sc, v);
                        slot[e] = bin > least ? slot_of(bin) : none;
                        atomicAdd(reinterpret_cast<unsigned long long*>(&s.mass[slot[e]]), mass_in(series, sc, v, bin));
                    }
                    if (with_count) {
#pragma unroll
                        for (int e = 0; e < N; ++e) atomicAdd(&s.count[slot[e]], 1u);
                    }
                });
            }
            c = next;
        }
        __syncthreads();
        return top_key;
    }

    // f in [0, 1) in units of 2^-48 (a NaN is 0).
    static __device__ __forceinline__ uint64_t units_of(float f) {
        return !(f > 0.f) ? 0 : f >= 1.f ? (1ull << 48) - 1 : static_cast<uint64_t>(static_cast<double>(f) * 0x1p48);
    }
    // The kept tokens are those before which less than top_p of the mass lies: the last
    // is the first at which the running mass passes this.
    static __device__ __forceinline__ uint64_t last_kept(float top_p, uint64_t mass) {
        bool exact;
        const uint64_t f = part_of(units_of(top_p), mass, &exact);
        return exact && f ? f - 1 : f;
    }

    struct Settings {
        float min_p, top_p, u;
        uint32_t top_k;            // 2^32 - 1: none
    };
    static __device__ __forceinline__ Settings settings_of(const SampleArgs& a, int r) {
        return {a.min_p ? a.min_p[r] : 0.f, a.top_p ? a.top_p[r] : 1.f, a.u[r],
                counts(a, r) ? static_cast<uint32_t>(a.top_k[r]) : 0xFFFFFFFFu};
    }

    // The smallest key with w >= min_p.
    static __device__ __forceinline__ uint32_t least_key(const Scale& sc, uint32_t top_key, float min_p, Shared& s) {
        if (thread() < 64) {
            const float top = logit_of(top_key);
            const double least = -log2(static_cast<double>(min_p)) * 32.0;
            const uint32_t k = first_key(top_key, [&](uint32_t key) {
                const float v = logit_of(key);
                return v == top || (static_cast<double>(top) - static_cast<double>(v)) * sc.c <= least;
            });
            if (thread() == 0) s.found32[3] = k;
        }
        __syncthreads();
        const uint32_t k = uniform(s.found32[3]);
        __syncthreads();
        return k;
    }

    struct Token {
        uint32_t key;
        int index;
        double mass;               // of all that was kept
    };

    // The list's n <= kNear elements, each at its rank, and the token.  All that the
    // filters keep is among them; whole is the row's mass where the list may end before
    // what top-p counts, else 0.
    static __device__ __forceinline__ Token among_list(const Scale& sc, uint32_t n, const Settings& set, uint32_t least,
                                                uint64_t whole, Shared& s) {
        const uint32_t t = thread();
        // ranks: where there are fewer elements than threads, several threads to each
        const uint32_t width = n > 1 ? 1u << (32 - __builtin_clz(n - 1)) : 1, share = (n * width + kThreads - 1) / kThreads;
        const uint32_t e = t & (width - 1), from = t / width * share, to = from + share < n ? from + share : n;
        uint64_t mine = e < n ? s.list.order[e] : 0, m = 0;
        if (t < n) m = to_top(s.list.mass[t] << kFine, depth_of(sc, logit_of(~static_cast<uint32_t>(mine >> 32))), s).whole;
        if (t < 8) s.list.order[n + t] = ~0ull;
        s.count[t] = 0;
        __syncthreads();
        if (e < n) {
            uint32_t rank = 0;
            for (uint32_t j0 = from; j0 < to; j0 += 8) {
                uint64_t o[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = s.list.order[j0 + j];
#pragma unroll
                for (int j = 0; j < 8; ++j) rank += o[j] < mine && j0 + j < to;
            }
            atomicAdd(&s.count[e], rank);
        }
        __syncthreads();
        if (t < n) {
            s.list.sorted.order[s.count[t]] = mine;
            s.list.sorted.ahead[s.count[t]] = m;
        }
        __syncthreads();
        mine = t < n ? s.list.sorted.order[t] : ~0ull;
        m = t < n ? s.list.sorted.ahead[t] : 0;
        const uint64_t behind = block_scan(m, s.part64), ahead = behind - m;       // (the mass up to and with it)
        if (t < n) s.list.sorted.ahead[t] = ahead;
        if (t == n - 1) s.found64[0] = behind;
        __syncthreads();
        const uint64_t all = s.found64[0];
        auto upto = [&](uint32_t kept) { return kept < n ? s.list.sorted.ahead[kept] : all; };
        uint32_t kept = __syncthreads_count(t < n && ~static_cast<uint32_t>(mine >> 32) >= least);
        kept = set.top_k < kept ? set.top_k : kept;
        uint64_t mass = upto(kept);
        if (set.top_p < 1.f) {
            const uint64_t last = whole ? last_kept(set.top_p, whole) << kFine | ((1u << kFine) - 1) : last_kept(set.top_p, mass);
            kept = __syncthreads_count(t < kept && ahead <= last);
            mass = upto(kept);
        }
        bool exact;
        const uint64_t goal = part_of(units_of(set.u), mass, &exact);
        const uint32_t at = __syncthreads_count(t < kept && behind <= goal);
        mine = s.list.sorted.order[at];
        return {~static_cast<uint32_t>(mine >> 32), static_cast<int>(static_cast<uint32_t>(mine)),
                static_cast<double>(mass) * (1.0 / (1 << kFine))};
    }

    static __device__ __forceinline__ void store_token(const SampleArgs& a, int r, const Scale& sc, const Token& token) {
        if (thread() != 0) return;
        a.token[r] = token.index;
        if (!a.logprob) return;
        const float v = logit_of(token.key);
        const double share = static_cast<double>(mass_of(sc, v)) / token.mass;
        const double y = log(share) - depth_of(sc, v) * (0.6931471805599453 / 32);
        a.logprob[r] = static_cast<float>(y < 0.0 ? y : 0.0);
    }

    // The largest logit of a row.
    static __device__ __forceinline__ uint32_t top_key_of(const Row& row, Shared& s) {
        float most = -__builtin_inff();
        row.words([&](int, uint4 word) {
#pragma unroll
            for (int e = 0; e < Chunk::N; ++e) most = fmaxf(most, Chunk::value(word, e));
        });
        return block_max(key_of(most), s.part32);
    }

    static __device__ __forceinline__ void store_largest(const SampleArgs& a, int r, uint64_t best) {
        if (thread() != 0) return;
        const bool none = static_cast<uint32_t>(best >> 32) == kKeyNone;
        a.token[r] = none ? -1 : static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(best));
        if (a.logprob) a.logprob[r] = none ? __builtin_nanf("") : 0.f;
    }

    // The smallest key that a small top-k can reach, from counts alone, over bins in fp32
    // (rounding is monotonic, so they are stretches of the order).  False where those keys
    // are too many.
    static __device__ __forceinline__ bool reach_of(const Row& row, const Scale& sc, uint32_t top_key, uint32_t top_k, Shared& s,
                                             uint32_t& from) {
        constexpr int N = Chunk::N;
        const float scale = static_cast<float>(sc.c), base = logit_of(top_key) * scale;
        auto place = [&](float v) { return fmaf(-v, scale, base); };      // (no number for a NaN; what is not below kBins is left out)
        for (int i = thread(); i < kSlots + 64; i += kThreads) s.count[i] = 0;
        __syncthreads();
        row.words([&](int, uint4 word) {
            int slot[N];
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const float d = place(Chunk::value(word, e));
                slot[e] = d < static_cast<float>(kBins) ? static_cast<int>(fmaxf(d, 0.f)) : kSlots + static_cast<int>(thread() & 63);
            }
#pragma unroll
            for (int e = 0; e < N; ++e) atomicAdd(&s.count[slot[e]], 1u);
        });
        __syncthreads();
        run_up<kBins / kThreads>(
            s.part64, s.part32,
            [&](int i, uint64_t& m, uint32_t& c) {
                m = 0;
                c = s.count[i];
            },
            [&](int i, uint64_t, uint32_t c) { s.run_count[i] = c; });
        if (s.run_count[kBins - 1] < top_k) return false;
        const int reach = first_past<kBins>(s.run_count, top_k - 1, s);
        if (s.run_count[reach] > kNear) return false;
        if (thread() < 64) {
            const uint32_t k = first_key(top_key, [&](uint32_t key) { return place(logit_of(key)) < static_cast<float>(reach + 1); });
            if (thread() == 0) s.found32[3] = k;
        }
        __syncthreads();
        from = uniform(s.found32[3]);
        __syncthreads();
        return true;
    }

    // The row's token.  fill() brings its bins and largest logit; top_key and sc's top are
    // known before only with `known`.
    template <typename F>
    static __device__ __forceinline__ void choose(const SampleArgs& a, int r, const Row& row, Scale& sc, uint32_t top_key,
                                           bool known, Shared& s, F fill) {
        const Settings set = settings_of(a, r);
        const bool counting = set.top_k != 0xFFFFFFFFu;
        uint32_t least = kKeyNone + 1;                   // keys from here on pass min-p
        int least_bin = kBins;
        int step = -1;                                   // what the list is for: all (-1), top-k, top-p, the token
        bool filled = false;
        Range range{0, 0};
        if (set.min_p > 0.f || set.top_k <= kNear / 2) {
            if (!known) {
                top_key = top_key_of(row, s);
                if (top_key != kKeyNone) set_top(sc, logit_of(top_key));
            }
            if (top_key == kKeyNone) {
                store_largest(a, r, static_cast<uint64_t>(kKeyNone) << 32);
                return;
            }
            range = {0, top_key};
            if (set.min_p > 0.f) range.lo = least = least_key(sc, top_key, set.min_p, s);
            else if (!reach_of(row, sc, top_key, set.top_k, s, range.lo)) range.lo = 0;
        }
        Token token{};
        uint64_t mass = 0, whole = 0, before = 0, left = 0, passed = 0;
        uint32_t all = 0;
        int bin = 0;
        while (true) {
            if (!filled && (step >= 0 || range.lo == 0)) {
                top_key = fill();
                filled = true;
                if (top_key == kKeyNone) {
                    store_largest(a, r, static_cast<uint64_t>(kKeyNone) << 32);
                    return;
                }
                // (a bin's count above the part of its mass behind the point, whose sums stay below 2^31)
                run_up<kBins / kThreads>(
                    s.part64, s.part64,
                    [&](int i, uint64_t& m, uint64_t& c) {
                        const uint64_t raw = s.mass[slot_of(sc.top - i)];
                        const Mass x = to_top(raw, i, s);
                        uint32_t n;
                        if (counting) {
                            n = s.count[slot_of(sc.top - i)];
                        } else {
                            // masses are within 1.1% of 2^44
                            const float f = static_cast<float>(raw) * 0x1p-44f;
                            n = static_cast<uint32_t>(rintf(f) + floorf(f * (1.f / 45)));
                        }
                        m = x.whole;
                        c = static_cast<uint64_t>(n) << 32 | x.part;
                    },
                    [&](int i, uint64_t m, uint64_t c) {
                        s.run_mass[i] = m + (static_cast<uint32_t>(c) >> 20);
                        s.run_count[i] = static_cast<uint32_t>(c >> 32);
                    });
                mass = uniform(s.run_mass[kBins - 1]);
                all = uniform(s.run_count[kBins - 1]);
                if (set.min_p > 0.f) {
                    const double below = uniform(sc.lone ? least == top_key ? 0.0 : kBins : sc.top - bin_at(sc, logit_of(least)));
                    least_bin = below < kBins ? static_cast<int>(below) : kBins;
                }
                // the last bin that any of it can reach
                int reach = least_bin < kBins ? least_bin : kBins - 1;
                if (set.top_k <= all) {
                    const int b = first_past<kBins>(s.run_count, set.top_k - 1, s);
                    reach = b < reach ? b : reach;
                } else if (least_bin == kBins && set.top_p < 1.f) {
                    reach = first_past<kBins>(s.run_mass, last_kept(set.top_p, mass), s);
                    whole = mass;
                }
                if (s.run_count[reach] <= kNear) {
                    step = -1;
                    range = {keys_of(sc, top_key, reach, s).lo, top_key};
                } else {
                    step = 0;
                    if (least_bin < kBins) {
                        uint64_t m;
                        uint32_t n;
                        sum_of(row, sc, {least, keys_of(sc, top_key, least_bin, s).hi}, s, m, n);
                        mass = (least_bin ? uniform(s.run_mass[least_bin - 1]) : 0) + uniform(to_top(m, least_bin, s).whole);
                        all = (least_bin ? uniform(s.run_count[least_bin - 1]) : 0) + n;
                    }
                }
            }
            if (step >= 0 && range.lo == 0) {
                // the next question: its target, bin, and what of the target lies in the bin
                uint64_t target;
                if (step == 0) {
                    if (set.top_k >= all) {
                        step = 1;
                        continue;
                    }
                    target = set.top_k - 1;
                } else if (step == 1) {
                    if (!(set.top_p < 1.f)) {
                        step = 2;
                        continue;
                    }
                    target = last_kept(set.top_p, mass);
                } else {
                    bool exact;
                    target = part_of(units_of(set.u), mass, &exact);
                }
                bin = step == 0 ? first_past<kBins>(s.run_count, static_cast<uint32_t>(target), s)
                                : first_past<kBins>(s.run_mass, target, s);
                before = bin ? uniform(s.run_mass[bin - 1]) : 0;
                left = step == 0 ? target - (bin ? uniform(s.run_count[bin - 1]) : 0)
                                 : uniform(from_top(target - before, bin, s.mass[slot_of(sc.top - bin)] - 1, s));
                passed = 0;
                range = keys_of(sc, top_key, bin, s);
            }
            const uint32_t n = list_range(row, sc, range, s);
            if (step < 0) {
                if (n <= kNear) {
                    token = among_list(sc, n, set, least, whole, s);
                    break;
                }
                // too many: those that a small top-k reaches, else bins (1024 mixed rows 52 us, bins
                // for all of these 54)
                const bool fewer = !filled && set.min_p > 0.f && set.top_k <= kNear / 2 && range.lo == least;
                uint32_t from;
                if (fewer && reach_of(row, sc, top_key, set.top_k, s, from) && from > least) {
                    range.lo = from;
                    continue;
                }
                range.lo = 0;
                step = 0;
                continue;
            }
            uint32_t nth;
            uint64_t one, upto;
            if (n <= kList) {
                passed += of_list(step == 0, left, n, s);
                upto = uniform(s.found64[0]);
                token.key = ~uniform(static_cast<uint32_t>(s.found64[1] >> 32));
                token.index = uniform(static_cast<int>(static_cast<uint32_t>(s.found64[1])));
                __syncthreads();
            } else {
                if (!narrow(row, sc, step == 0, range, left, passed, nth, one, s)) continue;
                upto = (nth + 1) * one;
                token.key = range.hi;
                if (step == 2) token.index = nth_of(row, range.hi, nth, s);
            }
            if (step == 2) {
                token.mass = static_cast<double>(mass);
                break;
            }
            mass = before + uniform(to_top(passed + upto, bin, s).whole);
            ++step;
            range.lo = 0;
        }
        store_token(a, r, sc, token);
    }

    // The largest key of a row and the first element that has it.
    static __device__ __forceinline__ uint64_t largest(const Row& row) {
        uint64_t best = 0;
        row.words([&](int i0, uint4 word) {
#pragma unroll
            for (int e = 0; e < Chunk::N; ++e) {
                const uint64_t x = static_cast<uint64_t>(key_of(Chunk::value(word, e))) << 32 | (0xFFFFFFFFu - static_cast<uint32_t>(i0 + e));
                best = x > best ? x : best;
            }
        });
        return best;
    }
    static __device__ __forceinline__ void fill_tables(Shared& s) {
        const int t = thread();
        if (t < 32) {
            s.down[t] = static_cast<uint64_t>(exp2(-t / 32.0) * 0x1p63);
            s.up[t] = exp2(t / 32.0);
        }
    }
};

__device__ __forceinline__ float temperature_of(const SampleArgs& a, int r) { return a.temperature ? a.temperature[r] : 1.f; }

template <int DT>
__device__ __forceinline__ const char* row_at(const SampleArgs& a, int r) {
    return static_cast<const char*>(a.logits) + static_cast<int64_t>(r) * a.ld * (DT == F32 ? 4 : 2);
}

// A block to a row.
template <int DT>
__global__ __launch_bounds__(kThreads, 4) void sample_kernel(SampleArgs a) {
    using S = Sampler<DT>;
    __shared__ typename S::Shared s;
    const int r = blockIdx.x;
    const typename S::Row row(row_at<DT>(a, r), 0, a.vocab);
    const float temp = temperature_of(a, r);
    if (!(temp > 0.f)) {
        S::store_largest(a, r, S::block_max(S::largest(row), s.part64));
        return;
    }
    S::fill_tables(s);
    Scale sc = scale_of(temp);
    S::choose(a, r, row, sc, kKeyNone, false, s, [&] { return S::fill_bins(row, counts(a, r), sc, s); });
}

// What a part of a row leaves for the second launch.
struct Part {
    uint64_t best;      // at temperature 0: the largest key and its first place; else the key only
    double top;
    uint64_t mass[kBins];
    uint32_t count[kBins];
};
static_assert(sizeof(Part) == kSamplePartBytes && kSamplePartBytes % 16 == 0, "workspace of a part");

// A block to a part of a row: its bins, from its own largest one down.
template <int DT>
__global__ __launch_bounds__(kThreads, 4) void sample_part_kernel(SampleArgs a, int parts, int size, Part* out) {
    using S = Sampler<DT>;
    __shared__ typename S::Shared s;
    const int r = blockIdx.x / parts, p = blockIdx.x % parts, from = p * size;
    const typename S::Row row(row_at<DT>(a, r), from, from + size < a.vocab ? from + size : a.vocab);
    const float temp = temperature_of(a, r);
    Part& o = out[blockIdx.x];
    if (!(temp > 0.f)) {
        const uint64_t best = S::block_max(S::largest(row), s.part64);
        if (thread() == 0) o.best = best;
        return;
    }
    Scale sc = scale_of(temp);
    const bool counting = counts(a, r);
    const uint32_t top = S::fill_bins(row, counting, sc, s);
    if (thread() == 0) {
        o.best = static_cast<uint64_t>(top) << 32;
        o.top = sc.lone ? -__builtin_inf() : sc.top;
    }
    for (int i = thread(); i < kBins; i += kThreads) {
        o.mass[i] = s.mass[slot_of(sc.top - i)];
        if (counting) o.count[i] = s.count[slot_of(sc.top - i)];
    }
}

// The parts of a row met.
template <int DT>
__global__ __launch_bounds__(kThreads, 4) void sample_join_kernel(SampleArgs a, int parts, const Part* in) {
    using S = Sampler<DT>;
    __shared__ typename S::Shared s;
    const int r = blockIdx.x, t = thread();
    in += static_cast<int64_t>(r) * parts;
    uint64_t best = 0;
    for (int p = t; p < parts; p += kThreads) best = in[p].best > best ? in[p].best : best;
    best = S::block_max(best, s.part64);
    const float temp = temperature_of(a, r);
    const uint32_t top = static_cast<uint32_t>(best >> 32);
    if (!(temp > 0.f) || top == kKeyNone) {
        S::store_largest(a, r, best);
        return;
    }
    const typename S::Row row(row_at<DT>(a, r), 0, a.vocab);
    // the row's first 128 KB, a line to a load, on their way to this XCD's cache
    uint4 line[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) line[j] = row.word(8 * (kThreads * j + t));
    S::fill_tables(s);
    Scale sc = scale_of(temp);
    set_top(sc, logit_of(top));
    S::choose(a, r, row, sc, top, true, s, [&] {
        // where the parts' bins lie below the row's (far below: at kBins)
        const bool counting = counts(a, r);
        for (int p = t; p < parts; p += kThreads) {
            const uint32_t key = static_cast<uint32_t>(in[p].best >> 32);
            const double below = sc.lone ? 0.0 : sc.top - in[p].top;       // (a lone part is far below)
            s.offset[p] = key == kKeyNone || (sc.lone && key != top) || !(below < kBins) ? kBins : static_cast<int>(below);
        }
        __syncthreads();
        // (loads that every thread makes: those of all bins are out together)
        constexpr int kEach = kBins / kThreads;
        uint64_t m[kEach] = {};
        uint32_t c[kEach] = {};
#pragma unroll 4
        for (int p = 0; p < parts; ++p) {
            const int below = s.offset[p];
#pragma unroll
            for (int j = 0; j < kEach; ++j) {
                const int at = t + kThreads * j - below;
                const uint64_t pm = in[p].mass[at < 0 ? 0 : at];
                m[j] += at < 0 ? 0 : pm;
                if (counting) c[j] += at < 0 ? 0 : in[p].count[at];
            }
        }
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            const int i = t + kThreads * j;
            s.mass[slot_of(sc.top - i)] = m[j];
            s.count[slot_of(sc.top - i)] = c[j];
        }
        __syncthreads();
        return top;
    });
#pragma unroll
    for (int j = 0; j < 2; ++j) asm volatile("" ::"v"(line[j].x));
}

template <int DT>
hipError_t launch_dt(const SampleArgs& a, void* ws, hipStream_t st) {
    const SamplePlan plan = plan_sample(a.rows, a.vocab, ws != nullptr);
    if (plan.parts == 1) {
        sample_kernel<DT><<<dim3(static_cast<unsigned>(a.rows)), kThreads, 0, st>>>(a);
        return hipGetLastError();
    }
    Part* parts = static_cast<Part*>(ws);
    sample_part_kernel<DT><<<dim3(static_cast<unsigned>(a.rows * plan.parts)), kThreads, 0, st>>>(a, plan.parts, plan.size, parts);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    sample_join_kernel<DT><<<dim3(static_cast<unsigned>(a.rows)), kThreads, 0, st>>>(a, plan.parts, parts);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_sample(const SampleArgs& a, int dtype, void* ws, hipStream_t st) {
    return dtype == F16 ? launch_dt<F16>(a, ws, st) : dtype == BF16 ? launch_dt<BF16>(a, ws, st) : launch_dt<F32>(a, ws, st);
}

}  // namespace qlin
