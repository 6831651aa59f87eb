// Where a batch's tokens lie: the index arithmetic that the append and the
// attention kernels share.  Plain C++ (no HIP types), so a host build can run
// it over any metadata, damaged ones included.
//
// What the host cannot check, since it lies on the device, is bounded here:
// token ranges are cut to the rows the call has, cache lengths to max_kv (the
// host has checked that the page table's rows hold that many), and a page
// number outside the pool reads as kNoPage: such a page is neither read nor
// written.
#pragma once

#include <stdint.h>

#ifdef __HIPCC__
#define QLIN_HD __host__ __device__ __forceinline__
#else
#define QLIN_HD inline
#endif

namespace qlin {

constexpr int kNoPage = -1;

struct KvIndex {
    const int32_t* page_table;   // [batch][table_ld]
    int64_t table_ld;
    const int32_t* q_start;      // [batch + 1]
    const int32_t* kv_len;       // [batch]
    const int32_t* prefix_len;   // [batch] or nullptr
    int64_t tokens;              // rows of q / q|k|v
    int64_t pages;               // pages in the pool
    int32_t batch, max_q, max_kv;
    int32_t page_size;
};

// A sequence of the batch: its new tokens are rows row0 .. row0 + n - 1 and
// stand at positions first .. first + n - 1 = kv - 1 (first is negative where
// the lengths contradict each other: those rows have no place in the cache).
struct KvSeq {
    int64_t row0;
    int32_t n, kv, first;
};

QLIN_HD KvSeq kv_seq(const KvIndex& x, int b) {
    int64_t lo = x.q_start[b], hi = x.q_start[b + 1];
    lo = lo < 0 ? 0 : lo > x.tokens ? x.tokens : lo;
    hi = hi < lo ? lo : hi > x.tokens ? x.tokens : hi;
    KvSeq s;
    s.row0 = lo;
    s.n = static_cast<int32_t>(hi - lo < x.max_q ? hi - lo : x.max_q);
    const int32_t kv = x.kv_len[b];
    s.kv = kv < 0 ? 0 : kv > x.max_kv ? x.max_kv : kv;
    s.first = s.kv - s.n;
    return s;
}

// The pool's page that holds positions idx * page_size ..; idx must be below
// ceil(max_kv / page_size).
QLIN_HD int kv_page(const KvIndex& x, int b, int idx) {
    const int32_t p = x.page_table[static_cast<int64_t>(b) * x.table_ld + idx];
    return (p < 0 || p >= x.pages) ? kNoPage : p;
}

// The new tokens that fall into the sequence's touched page number i (its
// pages from the first new token's on): positions lo .. hi - 1 of page idx.
struct KvSpan {
    int32_t idx, lo, hi;   // empty where hi <= lo
};

QLIN_HD KvSpan kv_touched(const KvIndex& x, const KvSeq& s, int i) {
    const int32_t from = s.first < 0 ? 0 : s.first;
    const int64_t idx = static_cast<int64_t>(from / x.page_size) + i;
    const int64_t start = idx * x.page_size, end = start + x.page_size;
    KvSpan r = {0, 0, 0};
    if (start >= s.kv) return r;
    r.idx = static_cast<int32_t>(idx);
    r.lo = static_cast<int32_t>(start > from ? start : from);
    r.hi = static_cast<int32_t>(end < s.kv ? end : s.kv);
    return r;
}

// Most pages that max_q new tokens of one sequence can touch.
QLIN_HD int kv_max_touched(int32_t max_q, int32_t page_size) {
    return max_q < 1 ? 0 : static_cast<int>((static_cast<int64_t>(max_q) + page_size - 2) / page_size + 1);
}

// Keys j a query at position p sees: j < kv_visible(...).
QLIN_HD int32_t kv_visible(const KvIndex& x, const KvSeq& s, int b, int32_t p) {
    int32_t e = p + 1;
    if (x.prefix_len) {
        const int32_t f = x.prefix_len[b];
        e = e > f ? e : f;
    }
    return e < 0 ? 0 : e < s.kv ? e : s.kv;
}

// What a node of a tree of new tokens sees of the 32 keys from j0 on, bit i for
// key j0 + i: the cached keys, and behind them the new tokens whose bits its mask
// row has (32 to a word, ceil(n / 32) words read, bits from n on count as none).
QLIN_HD uint32_t kv_tree_bits(const uint32_t* row, const KvSeq& s, int32_t j0) {
    const int32_t rel = j0 - s.first;
    if (rel <= -32) return 0xFFFFFFFFu;
    const int32_t at = rel < 0 ? 0 : rel;
    if (at >= s.n) return rel < 0 ? (1u << -rel) - 1 : 0;
    const int32_t w = at >> 5, sh = at & 31, left = s.n - 32 * w;   // new tokens from word w's first on
    uint32_t lo = row[w];
    if (left < 32) lo &= (1u << left) - 1;
    if (rel < 0) return lo << -rel | ((1u << -rel) - 1);
    if (sh == 0) return lo;
    uint32_t hi = 0;
    if (left > 32) {
        hi = row[w + 1];
        if (left < 64) hi &= (1u << (left - 32)) - 1;
    }
    return lo >> sh | hi << (32 - sh);
}

}  // namespace qlin
