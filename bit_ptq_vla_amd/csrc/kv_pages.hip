// Pages of a paged int8 cache, for gfx950: which are in use, rows of the page
// table that share them, copies, and the tokens of an accepted path moved to
// their places.
//
// resize   One block holds the whole batch: the pages that rows give back, then
//   what each growing row needs (new pages, and a copy of its last page where
//   others hold it too), then the lowest free pages in the order of the rows, by
//   prefix sums over needs and over the words of free bits.  No list of free pages
//   is kept, so no order of atomics shows in the result.
// copy     A page of a layer is 16-byte pieces; blocks stride over (page, layer,
//   piece).
// compact  A wave owns a (sequence, layer, head) of k or of v and takes its
//   destination pages in turn: nodes only move towards the front, so a later
//   page's sources are not written before they are read.  Codes follow their
//   page's scale as exact quotients would round.

#include "device_common.h"
#include "kv_index.h"
#include "qlin_internal.h"

namespace qlin {

namespace {

typedef uint32_t u4 __attribute__((ext_vector_type(4)));

// Device-wide reads of words that this block's or other blocks' atomics changed.
__device__ __forceinline__ int32_t fresh(const int32_t* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint32_t fresh(const uint32_t* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__global__ __launch_bounds__(256) void pool_init_kernel(KvPoolArgs pool) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i < pool.pages) pool.refs[i] = 0;
    if (i < (pool.pages + 31) / 32) {
        const int64_t left = pool.pages - 32 * i;
        pool.free_bits[i] = left >= 32 ? 0xFFFFFFFFu : (1u << left) - 1;
    }
}

// Word w of the free bits, bits of pages past the pool's left out.
__device__ __forceinline__ uint32_t free_word(const KvPoolArgs& pool, int64_t w) {
    const int64_t left = pool.pages - 32 * w;
    return fresh(pool.free_bits + w) & (left >= 32 ? 0xFFFFFFFFu : (1u << left) - 1);
}

// Inclusive sum over the block's THREADS; every thread calls it.
template <int THREADS>
__device__ __forceinline__ int64_t block_scan(int64_t v, uint64_t* parts) {
    const uint64_t x = wave_sum_up(static_cast<uint64_t>(v));
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 63) parts[wave] = x;
    __syncthreads();
    uint64_t before = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 64 - 1; ++w) before += w < wave ? parts[w] : 0;
    __syncthreads();
    return static_cast<int64_t>(x + before);
}

// Place of the nth set bit (n below their number).
__device__ __forceinline__ int nth_bit(uint32_t bits, int n) {
    int at = 0;
#pragma unroll
    for (int half = 16; half; half /= 2) {
        const int low = __popc(bits >> at & ((1u << half) - 1));
        if (n >= low) {
            n -= low;
            at += half;
        }
    }
    return at;
}
// First place of rising values that is above x (there is one).
template <typename T>
__device__ __forceinline__ int first_above(const T* v, int n, int64_t x) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (v[mid] > x) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

// THREADS bounds the rows.
template <int THREADS>
__global__ __launch_bounds__(THREADS) void resize_kernel(KvPoolArgs pool, int32_t* table, int64_t ld, int cols, int rows,
                                                       int page_size, const int32_t* old_len, const int32_t* new_len,
                                                       int32_t* len_out, int32_t* moved) {
    __shared__ int have_s[THREADS], want_s[THREADS], shared_s[THREADS];
    __shared__ uint64_t parts[THREADS / 64], upto[THREADS];
    __shared__ uint8_t copy_s[THREADS];
    __shared__ int wide_s, bits_upto[THREADS];
    __shared__ uint32_t bits_s[THREADS];
    const int t = threadIdx.x;
    const int64_t most = static_cast<int64_t>(cols) * page_size;
    int64_t from = 0, to = 0;
    if (t < rows) {
        from = old_len[t];
        to = new_len[t];
        from = from < 0 ? 0 : from > most ? most : from;
        to = to < 0 ? 0 : to > most ? most : to;
    }
    const int have = static_cast<int>((from + page_size - 1) / page_size);
    const int want = static_cast<int>((to + page_size - 1) / page_size);
    have_s[t] = have;
    want_s[t] = want;
    __syncthreads();

    // pages behind the new lengths go back: all rows' at once, a row's widest release
    // from one row to the next
    if (t == 0) wide_s = 0;
    __syncthreads();
    if (have > want) atomicMax(&wide_s, have - want);
    __syncthreads();
    const int wide = wide_s;
    for (int64_t e = t; e < static_cast<int64_t>(rows) * wide; e += THREADS) {
        const int r = static_cast<int>(e / wide), i = want_s[r] + static_cast<int>(e % wide);
        if (i >= have_s[r]) continue;
        int32_t* entry = table + r * ld + i;
        const int32_t pg = *entry;
        *entry = -1;
        if (pg < 0 || pg >= pool.pages) continue;
        const int32_t held = atomicSub(pool.refs + pg, 1);
        if (held == 1) atomicOr(pool.free_bits + (pg >> 5), 1u << (pg & 31));
        if (held <= 0) atomicAdd(pool.refs + pg, 1);          // it was free: it stays so
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");       // (atomics that return nothing are waited for nowhere else)
    __syncthreads();

    // a last page that others hold too: all but the last of its growing holders take a copy
    int last = -1, holders = 0;
    if (to > from && from % page_size != 0) {
        last = table[t * ld + have - 1];
        if (last < 0 || last >= pool.pages) last = -1;
        if (last >= 0) holders = fresh(pool.refs + last);
    }
    shared_s[t] = last;
    __syncthreads();
    bool copy = false;
    if (holders > 1) {
#pragma unroll 8
        for (int r = 0; r < t; ++r) holders -= shared_s[r] == last;
        copy = holders > 1;
    }
    copy_s[t] = copy;
    const int64_t need = to > from ? want - have + (copy ? 1 : 0) : 0;
    const int64_t sum = block_scan<THREADS>(need, parts);
    const int64_t words = (pool.pages + 31) / 32;
    int64_t free_here = 0;
    for (int64_t w = t; w < words; w += THREADS) free_here += __popc(free_word(pool, w));
    upto[t] = block_scan<THREADS>(free_here, parts);
    __syncthreads();
    const int64_t free_pages = upto[THREADS - 1];
    __syncthreads();
    upto[t] = sum;
    bool ok = need == 0 || sum <= free_pages;
    const int64_t mine = ok && need > 0 ? sum : 0;
    __shared__ int64_t total_s;
    __shared__ int stays_s;                  // the first row that stays as it is
    if (t == 0) {
        total_s = 0;
        stays_s = rows;
    }
    __syncthreads();
    if (!ok) atomicMin(&stays_s, t);
    __syncthreads();
    if (ok && t > stays_s && last >= 0) {
        // holders before this row that stay hold its last page still
        int left = fresh(pool.refs + last);
        for (int r = 0; r < stays_s; ++r) left -= shared_s[r] == last;
        ok = left <= 1;
    }
    if (mine > 0) atomicMax(reinterpret_cast<unsigned long long*>(&total_s), static_cast<unsigned long long>(mine));
    if (t < rows) {
        len_out[t] = static_cast<int32_t>(ok ? to : from);
        moved[2 * t] = -1;
        moved[2 * t + 1] = -1;
    }
    __syncthreads();

    // the i-th free page from the lowest on goes to the row whose needs contain i: THREADS
    // words of free bits at a time, a thread to a page
    const int64_t total = total_s;
    int64_t base = 0;
    for (int64_t w0 = 0; w0 < words && base < total; w0 += THREADS) {
        const int64_t w = w0 + t;
        const uint32_t bits = w < words ? free_word(pool, w) : 0;
        const int n = __popc(bits), sum_here = static_cast<int>(block_scan<THREADS>(n, parts));
        bits_s[t] = bits;
        bits_upto[t] = sum_here;
        const int64_t left = total - base - (sum_here - n);      // pages taken from this word on
        if (left > 0 && n > 0) pool.free_bits[w] = left >= n ? 0 : bits & ~((2u << nth_bit(bits, static_cast<int>(left) - 1)) - 1);
        __syncthreads();
        const int here = bits_upto[THREADS - 1];
        for (int j = t; j < here && base + j < total; j += THREADS) {
            const int word = first_above(bits_upto, THREADS, j);
            const int bit = nth_bit(bits_s[word], j - (word > 0 ? bits_upto[word - 1] : 0));
            const int32_t pg = static_cast<int32_t>(32 * (w0 + word) + bit);
            const int r = first_above(upto, rows, base + j);
            int at = have_s[r] + static_cast<int>(base + j - (r > 0 ? upto[r - 1] : 0)) - copy_s[r];
            if (at < have_s[r]) {                 // the copy of the last page
                moved[2 * r] = shared_s[r];
                moved[2 * r + 1] = pg;
                atomicSub(pool.refs + shared_s[r], 1);
            }
            table[r * ld + at] = pg;
            pool.refs[pg] = 1;
        }
        base += here;
        __syncthreads();
    }
}

__global__ __launch_bounds__(256) void fork_kernel(KvPoolArgs pool, int32_t* table, int64_t ld, int cols, int rows,
                                                   int page_size, const int32_t* src, const int32_t* dst,
                                                   const int32_t* len) {
    const int a = src[blockIdx.x], b = dst[blockIdx.x];
    if (a < 0 || a >= rows || b < 0 || b >= rows || a == b) return;
    const int64_t n = (static_cast<int64_t>(len[blockIdx.x]) + page_size - 1) / page_size;
    for (int i = threadIdx.x; i < n && i < cols; i += 256) {
        int32_t pg = table[a * ld + i];
        if (pg < 0 || pg >= pool.pages || fresh(pool.refs + pg) < 1) pg = -1;
        else atomicAdd(pool.refs + pg, 1);
        table[b * ld + i] = pg;
    }
}

// ---- copies --------------------------------------------------------------------

constexpr int kWordsEach = 8;
constexpr int kPiece = 256 * kWordsEach;     // 16-byte words a block copies at a time

// Pairs (from, to): [n][2].  The pairs that copy anything are gathered first, 1024
// at a time and in their order (every block finds the same tasks), so that blocks
// without work end at once.  Bound by HBM: 128 pages of 64 tokens in 16 layers of 8
// heads of 128 (537 MB read and written) take 104 us, 5.15 TB/s as a plain copy; where
// they are copies of 16 pages, whose reads the caches serve, 88.  Stores that stay in the
// caches take 142 there.
__global__ __launch_bounds__(256) void copy_pages_kernel(KvStackArgs c, const int32_t* pairs, int64_t n) {
    __shared__ int32_t from[1024], to[1024];
    __shared__ int counts[16];
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int64_t page_words = static_cast<int64_t>(c.heads) * c.page_size * c.head_dim / 16;
    const int pieces = static_cast<int>((page_words + kPiece - 1) / kPiece);
    for (int64_t base = 0; base < n; base += 1024) {
        int a[4], b[4], place[4];
        bool good[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int64_t i = base + 256 * r + t;
            a[r] = i < n ? pairs[2 * i] : -1;
            b[r] = i < n ? pairs[2 * i + 1] : -1;
            good[r] = a[r] >= 0 && a[r] < c.pages && b[r] >= 0 && b[r] < c.pages && a[r] != b[r];
            const uint64_t votes = __ballot(good[r]);
            place[r] = __popcll(votes & ((1ull << lane) - 1));
            if (lane == 0) counts[4 * r + wave] = __popcll(votes);
        }
        __syncthreads();
        int found = 0;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const int r = k >> 2;
            if ((k & 3) == wave && good[r]) {
                from[found + place[r]] = a[r];
                to[found + place[r]] = b[r];
            }
            found += counts[k];
        }
        __syncthreads();
        const int64_t tasks = static_cast<int64_t>(found) * c.layers * 2 * pieces;
        for (int64_t u = blockIdx.x; u < tasks; u += gridDim.x) {
            const int piece = static_cast<int>(u % pieces);
            const int64_t v = u / pieces;
            const int which = static_cast<int>(v % (2 * c.layers)), at = static_cast<int>(v / (2 * c.layers));
            const KvLayerArgs& l = c.layer[which >> 1];
            const bool is_v = which & 1;
            const u4* s = reinterpret_cast<const u4*>(is_v ? l.v : l.k) + from[at] * page_words;
            u4* d = reinterpret_cast<u4*>(is_v ? l.v : l.k) + to[at] * page_words;
            u4 w[kWordsEach];
            const int64_t i0 = static_cast<int64_t>(piece) * kPiece + threadIdx.x;
            if (static_cast<int64_t>(piece + 1) * kPiece <= page_words) {
#pragma unroll
                for (int j = 0; j < kWordsEach; ++j) w[j] = __builtin_nontemporal_load(s + i0 + 256 * j);
#pragma unroll
                for (int j = 0; j < kWordsEach; ++j) __builtin_nontemporal_store(w[j], d + i0 + 256 * j);
            } else {
                for (int64_t i = i0; i < page_words; i += 256) d[i] = s[i];
            }
            if (piece == 0) {
                float* f = is_v ? l.vs : l.ks;
                for (int h = threadIdx.x; h < c.heads; h += 256)
                    f[static_cast<int64_t>(to[at]) * c.heads + h] = f[static_cast<int64_t>(from[at]) * c.heads + h];
            }
        }
        __syncthreads();
    }
}

// ---- compaction ----------------------------------------------------------------

// Sixteen codes (a word of memory) from scale `was` to `now`: rne(c was / now).  In
// fp32 a quotient is off by less than 2^-16 (two roundings of at most 127), which
// decides it unless it lies that close to a half-integer: then in float64, where the
// product is exact and the quotient's rounding cannot reach a half-integer.
__device__ __forceinline__ int follow_one(int c, float ratio, bool& close) {
    const float x = static_cast<float>(c) * ratio, n = rintf(x);
    close |= fabsf(x - n) > 0.5f - 0x1p-15f;
    return static_cast<int>(n);
}
__device__ __forceinline__ int follow_exact(int c, float was, float now) {
    return static_cast<int>(rint(static_cast<double>(c) * was / now));
}
__device__ __forceinline__ uint4 follow16(uint4 w, float was, float now) {
    uint32_t x[4] = {w.x, w.y, w.z, w.w};
    if (was == now) return w;
    const float ratio = was / now;
    bool close = false;
    uint32_t y[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 16; ++i)
        y[i / 4] |= (follow_one(static_cast<int8_t>(x[i / 4] >> 8 * (i % 4)), ratio, close) & 0xFF) << 8 * (i % 4);
    if (close) {
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
            uint32_t z = 0;
            for (int e = 0; e < 4; ++e) z |= (follow_exact(static_cast<int8_t>(x[0] >> 8 * e), was, now) & 0xFF) << 8 * e;
            x[0] = x[1];
            x[1] = x[2];
            x[2] = x[3];
            y[0] = y[1];
            y[1] = y[2];
            y[2] = y[3];
            y[3] = z;
        }
    }
    return make_uint4(y[0], y[1], y[2], y[3]);
}

// A block takes a sequence of a layer, a wave a head of its k or of its v and the
// destination pages in turn.  A page holds at most 64 tokens: lane i has the page and
// scale that its i-th one comes from.  k moves by 16-byte pieces of a token, a lane
// each; v by granules of 16 tokens of a dimension, a lane each, whose bytes come from
// wherever the tokens lie.
//
// Bound by the chain page table, scales, codes, stores at five waves to a SIMD, and by
// what shares the moved codes' cache lines: 64 paths of 8 of 32 nodes in 16 layers of 8
// heads of 128 (29 MB of moved codes, node 0's among them, which stays where it is; some
// 60 MB are read and 46 written, since v's move by whole granules, 16 bytes to a row of a
// page) take 36 us where no page's scale rises, 39 where scales do and kept tokens follow
// them; one path of 5 of 16 in 32 layers of 32 heads 8.  Granules of v whose tokens are all
// kept under the same scale are left alone (written back: 48 MB, 38 us).  A wave for a
// head's k and v takes 35 and 8, a wave for 64 dimensions of v 60 and 7 (both with those
// granules written): each wave repeats the chain.
__global__ __launch_bounds__(256) void compact_kernel(KvIndex ix, KvStackArgs c, const int32_t* path, int64_t path_ld,
                                                      const int32_t* count, int32_t* len_out, int groups) {
    __shared__ int16_t node[kMaxTreeNodes];
    __shared__ int valid;
    int64_t u = blockIdx.x;
    const int group = static_cast<int>(u % groups);
    u /= groups;
    const int layer = static_cast<int>(u % c.layers), b = static_cast<int>(u / c.layers);
    const KvSeq s = kv_seq(ix, b);
    const int t = threadIdx.x, lane = t & 63, d = c.head_dim, ps = c.page_size;
    int m = count[b];
    m = m < 0 || s.first < 0 ? 0 : m > s.n ? s.n : m;
    if (t == 0) valid = m;
    __syncthreads();
    for (int i = t; i < m; i += 256) {       // the path ends where it does not lead to a later node
        const int a = path[b * path_ld + i], before = i > 0 ? path[b * path_ld + i - 1] : -1;
        if (a <= before || a < 0 || a >= s.n) atomicMin(&valid, i);
        node[i] = static_cast<int16_t>(a);
    }
    __syncthreads();
    m = valid;
    if (len_out && group == 0 && layer == 0 && t == 0) len_out[b] = s.first < 0 ? s.kv : s.first + m;

    const int task = 4 * group + (t >> 6), h = task >> 1;
    if (m == 0 || h >= c.heads) return;
    const bool is_v = task & 1;
    const KvLayerArgs& l = c.layer[layer];
    int8_t* codes = is_v ? l.v : l.k;
    float* scales = is_v ? l.vs : l.ks;
    const int64_t page_bytes = static_cast<int64_t>(ps) * d;
    auto base_of = [&](int pg) { return codes + (static_cast<int64_t>(pg) * c.heads + h) * page_bytes; };
    auto scale_of = [&](int pg) { return scales + static_cast<int64_t>(pg) * c.heads + h; };
    for (int idx = s.first / ps; idx * ps < s.first + m; ++idx) {
        const int lo = idx * ps > s.first ? idx * ps - s.first : 0;                       // tokens of the path
        const int hi = (idx + 1) * ps < s.first + m ? (idx + 1) * ps - s.first : m;       // that end in this page
        const int pg = kv_page(ix, b, idx);
        if (pg == kNoPage || node[hi - 1] == hi - 1) continue;      // (a path that has not left its place)
        const int kept = idx * ps < s.first ? s.first - idx * ps : 0;
        int8_t* dst = base_of(pg);
        const float was = *scale_of(pg);
        // the lane's token: where it comes from
        int from = kNoPage, off = 0;
        float scale = 0.f;
        if (lane < hi - lo) {
            const int pos = s.first + node[lo + lane];
            from = kv_page(ix, b, pos / ps);
            off = pos % ps;
            if (from != kNoPage) scale = *scale_of(from);
        }
        float now = fmaxf(fabsf(scale), kept ? fabsf(was) : 0.f);
        now = wave_max(now, 64);
        if (!is_v) {
            const int per = d / 16;                  // pieces of a token
            if (kept && was != now)
                for (int e = lane; e < kept * per; e += 64) {
                    uint4* x = reinterpret_cast<uint4*>(dst) + e;
                    *x = follow16(*x, was, now);
                }
            for (int e0 = 0; e0 < (hi - lo) * per; e0 += 64) {
                const int e = e0 + lane, i = e / per, j = e % per;
                const int pg_i = __shfl(from, i & 63, 64), off_i = __shfl(off, i & 63, 64);
                const float scale_i = __shfl(scale, i & 63, 64);
                const bool there = e < (hi - lo) * per;
                uint4 w = make_uint4(0, 0, 0, 0);
                if (there && pg_i != kNoPage) w = reinterpret_cast<const uint4*>(base_of(pg_i) + off_i * d)[j];
                // (a token's old place is another one's new place: all lanes have read before one writes)
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                __builtin_amdgcn_wave_barrier();
                if (there && pg_i != kNoPage) w = follow16(w, scale_i, now);
                if (there) reinterpret_cast<uint4*>(dst + (kept + i) * d)[j] = w;
            }
        } else {
            for (int g = 0; g < ps; g += 16) {
                // places g .. g + 15 of the page: kept ones, then tokens, then others
                const int k1 = kept - g < 0 ? 0 : kept - g > 16 ? 16 : kept - g;
                const int i1 = kept + hi - lo - g > 16 ? 16 : kept + hi - lo - g;
                if (i1 <= 0 || (i1 <= k1 && was == now)) continue;
                for (int j = lane; j < d; j += 64) {
                    uint4* x = reinterpret_cast<uint4*>(dst + j * ps + g);
                    const uint4 old = *x;
                    const uint4 held = k1 > 0 ? follow16(old, was, now) : old;
                    const uint32_t o[4] = {old.x, old.y, old.z, old.w}, k[4] = {held.x, held.y, held.z, held.w};
                    int code[16];
                    float sc[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const int i = g + e - kept;              // token of the page, the same for all lanes
                        code[e] = 0;
                        sc[e] = now;
                        if (e < k1 || e >= i1) continue;
                        const int pg_i = __builtin_amdgcn_readlane(from, i), off_i = __builtin_amdgcn_readlane(off, i);
                        sc[e] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(scale), i));
                        if (pg_i != kNoPage) code[e] = base_of(pg_i)[j * ps + off_i];
                    }
                    uint32_t y[4] = {0, 0, 0, 0};
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        uint32_t v = e < k1 ? k[e / 4] >> 8 * (e % 4) : o[e / 4] >> 8 * (e % 4);
                        if (e >= k1 && e < i1) {
                            bool close = false;
                            int n = code[e];
                            if (sc[e] != now) {
                                n = follow_one(code[e], sc[e] / now, close);
                                if (close) n = follow_exact(code[e], sc[e], now);
                            }
                            v = n;
                        }
                        y[e / 4] |= (v & 0xFF) << 8 * (e % 4);
                    }
                    *x = make_uint4(y[0], y[1], y[2], y[3]);
                }
            }
        }
        if (lane == 0) *scale_of(pg) = now;
    }
}

}  // namespace

hipError_t launch_pool_init(const KvPoolArgs& pool, hipStream_t st) {
    pool_init_kernel<<<dim3(static_cast<unsigned>((pool.pages + 255) / 256)), 256, 0, st>>>(pool);
    return hipGetLastError();
}

hipError_t launch_kv_resize(const KvPoolArgs& pool, int32_t* table, int64_t ld, int cols, int rows, int page_size,
                            const int32_t* old_len, const int32_t* new_len, int32_t* len_out, int32_t* moved,
                            hipStream_t st) {
    // (a block of a few waves is through its barriers sooner: 5 rows that grow 5.1 us, 1024 threads 6.9)
    if (rows <= 256)
        resize_kernel<256><<<1, 256, 0, st>>>(pool, table, ld, cols, rows, page_size, old_len, new_len, len_out, moved);
    else
        resize_kernel<kMaxPoolRows><<<1, kMaxPoolRows, 0, st>>>(pool, table, ld, cols, rows, page_size, old_len, new_len,
                                                                len_out, moved);
    return hipGetLastError();
}

hipError_t launch_kv_fork(const KvPoolArgs& pool, int32_t* table, int64_t ld, int cols, int rows, int page_size,
                          const int32_t* src, const int32_t* dst, const int32_t* len, int n, hipStream_t st) {
    fork_kernel<<<dim3(static_cast<unsigned>(n)), 256, 0, st>>>(pool, table, ld, cols, rows, page_size, src, dst, len);
    return hipGetLastError();
}

hipError_t launch_kv_copy_pages(const KvStackArgs& c, const int32_t* pairs, int64_t n, hipStream_t st) {
    const int64_t words = static_cast<int64_t>(c.heads) * c.page_size * c.head_dim / 16;
    const int64_t tasks = n * c.layers * 2 * ((words + kPiece - 1) / kPiece);
    const int64_t most = 4 * static_cast<int64_t>(device_cus());
    copy_pages_kernel<<<dim3(static_cast<unsigned>(tasks < most ? tasks : most)), 256, 0, st>>>(c, pairs, n);
    return hipGetLastError();
}

hipError_t launch_kv_compact(const KvIndex& ix, const KvStackArgs& c, const int32_t* path, int64_t path_ld,
                             const int32_t* count, int32_t* len_out, hipStream_t st) {
    const int groups = (c.heads + 1) / 2;
    const int64_t blocks = static_cast<int64_t>(ix.batch) * c.layers * groups;
    compact_kernel<<<dim3(static_cast<unsigned>(blocks)), 256, 0, st>>>(ix, c, path, path_ld, count, len_out, groups);
    return hipGetLastError();
}

}  // namespace qlin
