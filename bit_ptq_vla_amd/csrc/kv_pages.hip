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
// compact  A block owns a (sequence, layer, head) of k or of v and takes its
//   destination pages in turn: nodes only move towards the front, so a later
//   page's sources are not written before they are read.  Codes follow their
//   page's scale by quotients in float64: the codes of exact arithmetic.

#include "device_common.h"
#include "kv_index.h"
#include "qlin_internal.h"

namespace qlin {

namespace {

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

constexpr int kRows = kMaxPoolRows;      // rows of a resize, and its threads
constexpr int kWaves = kRows / 64;

// Inclusive sum over the block's threads; every thread calls it.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* parts) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int64_t o = __shfl_up(v, d, 64);
        if (lane >= d) v += o;
    }
    if (lane == 63) parts[wave] = v;
    __syncthreads();
    int64_t before = 0;
    for (int w = 0; w < wave; ++w) before += parts[w];
    __syncthreads();
    return v + before;
}

__global__ __launch_bounds__(kRows) void resize_kernel(KvPoolArgs pool, int32_t* table, int64_t ld, int cols, int rows,
                                                       int page_size, const int32_t* old_len, const int32_t* new_len,
                                                       int32_t* len_out, int32_t* moved) {
    __shared__ int have_s[kRows], want_s[kRows], shared_s[kRows];
    __shared__ int64_t parts[kWaves], upto[kRows];
    __shared__ uint8_t copy_s[kRows];
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
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

    // pages behind the new lengths go back
    for (int r = wave; r < rows; r += kWaves)
        for (int i = want_s[r] + lane; i < have_s[r]; i += 64) {
            int32_t* e = table + r * ld + i;
            const int32_t pg = *e;
            *e = -1;
            if (pg < 0 || pg >= pool.pages) continue;
            const int32_t held = atomicSub(pool.refs + pg, 1);
            if (held == 1) atomicOr(pool.free_bits + (pg >> 5), 1u << (pg & 31));
            if (held <= 0) atomicAdd(pool.refs + pg, 1);      // it was free: it stays so
        }
    __threadfence();
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
        for (int r = 0; r < t; ++r) holders -= shared_s[r] == last;
        copy = holders > 1;
    }
    copy_s[t] = copy;
    const int64_t need = to > from ? want - have + (copy ? 1 : 0) : 0;
    const int64_t sum = block_scan(need, parts);
    const int64_t words = (pool.pages + 31) / 32;
    int64_t free_here = 0;
    for (int64_t w = t; w < words; w += kRows) free_here += __popc(free_word(pool, w));
    upto[t] = block_scan(free_here, parts);
    __syncthreads();
    const int64_t free_pages = upto[kRows - 1];
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

    // the i-th free page from the lowest on goes to the row whose needs contain i
    const int64_t total = total_s;
    int64_t base = 0;
    for (int64_t w0 = 0; w0 < words && base < total; w0 += kRows) {
        const int64_t w = w0 + t;
        uint32_t bits = w < words ? free_word(pool, w) : 0;
        const int64_t upto_here = block_scan(__popc(bits), parts);
        int64_t i = base + upto_here - __popc(bits);
        const uint32_t before = bits;
        while (bits && i < total) {
            const int bit = __builtin_ctz(bits);
            bits &= bits - 1;
            const int32_t pg = static_cast<int32_t>(32 * w + bit);
            int lo = 0, hi = rows - 1;            // first row with upto > i
            while (lo < hi) {
                const int mid = (lo + hi) / 2;
                if (upto[mid] > i) hi = mid;
                else lo = mid + 1;
            }
            const int64_t before_row = lo > 0 ? upto[lo - 1] : 0;
            int at = have_s[lo] + static_cast<int>(i - before_row) - copy_s[lo];
            if (at < have_s[lo]) {                // the copy of the last page
                moved[2 * lo] = shared_s[lo];
                moved[2 * lo + 1] = pg;
                atomicSub(pool.refs + shared_s[lo], 1);
            }
            table[lo * ld + at] = pg;
            pool.refs[pg] = 1;
            ++i;
        }
        if (bits != before) pool.free_bits[w] = bits;
        if (t == kRows - 1) total_s = upto_here;
        __syncthreads();
        base += total_s;
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

constexpr int kPiece = 256 * 4;        // 16-byte words a block copies at a time

// Pairs (from, to): [n][2].  The pairs that copy anything are gathered first, 1024
// at a time and in their order (every block finds the same tasks), so that blocks
// without work end at once.
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
            const uint4* s = reinterpret_cast<const uint4*>(is_v ? l.v : l.k) + from[at] * page_words;
            uint4* d = reinterpret_cast<uint4*>(is_v ? l.v : l.k) + to[at] * page_words;
            uint4 w[4];
            const int64_t i0 = static_cast<int64_t>(piece) * kPiece + threadIdx.x;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (i0 + 256 * j < page_words) w[j] = s[i0 + 256 * j];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (i0 + 256 * j < page_words) d[i0 + 256 * j] = w[j];
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

__device__ __forceinline__ int8_t follow_scale(int8_t code, float was, float now) {
    return was == now ? code : static_cast<int8_t>(rint(static_cast<double>(code) * was / now));
}

__global__ __launch_bounds__(256) void compact_kernel(KvIndex ix, KvStackArgs c, const int32_t* path, int64_t path_ld,
                                                      const int32_t* count, int32_t* len_out) {
    __shared__ int8_t buf[64 * 256];
    __shared__ int16_t node[kMaxTreeNodes];
    __shared__ int valid;
    __shared__ uint32_t top;
    int64_t u = blockIdx.x;
    const bool is_v = u & 1;
    u >>= 1;
    const int h = static_cast<int>(u % c.heads);
    u /= c.heads;
    const int layer = static_cast<int>(u % c.layers), b = static_cast<int>(u / c.layers);
    const KvSeq s = kv_seq(ix, b);
    const int t = threadIdx.x, d = c.head_dim, ps = c.page_size;
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
    if (len_out && is_v && h == 0 && layer == 0 && t == 0) len_out[b] = s.first < 0 ? s.kv : s.first + m;
    if (m == 0) return;

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
        __syncthreads();
        if (t == 0) top = 0;
        __syncthreads();
        const float was = *scale_of(pg);
        if (t < hi - lo) {
            const int from = kv_page(ix, b, (s.first + node[lo + t]) / ps);
            if (from != kNoPage) atomicMax(&top, __float_as_uint(fabsf(*scale_of(from))));
        } else if (t == 255 && kept) {
            atomicMax(&top, __float_as_uint(fabsf(was)));
        }
        __syncthreads();
        const float now = __uint_as_float(top);
        int8_t* dst = base_of(pg);
        if (kept && was != now)
            for (int e = t; e < kept * d; e += 256) {
                int8_t* x = is_v ? dst + e / kept * ps + e % kept : dst + e;
                *x = follow_scale(*x, was, now);
            }
        for (int e = t; e < (hi - lo) * d; e += 256) {
            const int i = lo + e / d, j = e % d, pos = s.first + node[i];
            const int from = kv_page(ix, b, pos / ps);
            int8_t code = 0;
            if (from != kNoPage) {
                const int8_t* x = base_of(from) + (is_v ? j * ps + pos % ps : pos % ps * d + j);
                code = follow_scale(*x, *scale_of(from), now);
            }
            buf[e] = code;
        }
        __syncthreads();
        for (int e = t; e < (hi - lo) * d; e += 256) {
            const int j = e % d, off = (s.first + lo + e / d) % ps;
            dst[is_v ? j * ps + off : off * d + j] = buf[e];
        }
        if (t == 0) *scale_of(pg) = now;
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
    resize_kernel<<<1, kRows, 0, st>>>(pool, table, ld, cols, rows, page_size, old_len, new_len, len_out, moved);
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
    const int64_t most = 8 * static_cast<int64_t>(device_cus());
    copy_pages_kernel<<<dim3(static_cast<unsigned>(tasks < most ? tasks : most)), 256, 0, st>>>(c, pairs, n);
    return hipGetLastError();
}

hipError_t launch_kv_compact(const KvIndex& ix, const KvStackArgs& c, const int32_t* path, int64_t path_ld,
                             const int32_t* count, int32_t* len_out, hipStream_t st) {
    const int64_t blocks = static_cast<int64_t>(ix.batch) * c.layers * c.heads * 2;
    compact_kernel<<<dim3(static_cast<unsigned>(blocks)), 256, 0, st>>>(ix, c, path, path_ld, count, len_out);
    return hipGetLastError();
}

}  // namespace qlin
