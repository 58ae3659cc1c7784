// kv_index.h -- index arithmetic of the paged 4-bit cache and of attention
// over it, shared by the kernels, the host layer and the CPU tests (plain
// integer functions without device state).
//
// The cache holds, for K and for V, codes [num_pages][kv_heads][page_size]
// [head_dim / 2] and scale bytes [num_pages][kv_heads][page_size][head_dim /
// block]: a page's rows of one head are contiguous, and each row is laid out as
// fp4_quantize lays out a row of head_dim values.
#pragma once

#include <stdint.h>

#if defined(__HIPCC__)
#define FP4Q_HD __host__ __device__ __forceinline__
#else
#define FP4Q_HD inline
#endif

namespace fp4q {

constexpr int kKvGroup = 16;             // tokens the kernels address together; page_size is a multiple
constexpr int kKvMaxPage = 4096;         // bounds that keep DivBy exact (see there)
constexpr int64_t kKvMaxTokens = (int64_t)1 << 27;   // keys of one sequence

// Exact u / d for u < 2^32 / d, by one multiplication: M = ceil(2^32 / d) gives
// u M / 2^32 = u / d + u e / (d 2^32) with 0 <= e < d, and the excess stays
// below 1 / d.  Divides a token group's number (below 2^27 / 16) by the groups of a
// page (at most 256).
struct DivBy {
    uint64_t m;
    uint32_t d;
};

inline DivBy make_div(uint32_t d) { return DivBy{(((uint64_t)1 << 32) + d - 1) / d, d}; }

FP4Q_HD uint32_t div_by(uint32_t u, const DivBy& k) { return (uint32_t)((u * k.m) >> 32); }

// Exact g / d for any 64-bit g below 2^56 and d at most 256: the upper half of g M with M =
// ceil(2^64 / d), by the argument above (d = 1 has no such M).  A 64-bit division in
// each lane took most of the reader's time (131072 rows: 173 us).
struct DivBy64 {
    uint64_t m;
    uint32_t d;
};

inline DivBy64 make_div64(uint32_t d) { return DivBy64{d > 1 ? ~(uint64_t)0 / d + 1 : 0, d}; }

FP4Q_HD uint64_t div_by(uint64_t g, const DivBy64& k)
{
    if (k.d == 1) return g;
#if defined(__HIP_DEVICE_COMPILE__)
    return __umul64hi(g, k.m);
#else
    return (uint64_t)(((unsigned __int128)g * k.m) >> 64);
#endif
}

// Row of a slot (= page * page_size + place in the page) of one head: the row
// number to multiply by the bytes of a row, or -1 for a slot outside the cache.
FP4Q_HD int64_t kv_row_of_slot(int64_t slot, int64_t num_slots, const DivBy64& groups_per_page, int32_t heads, int32_t head)
{
    if (slot < 0 || slot >= num_slots) return -1;
    const int64_t page = (int64_t)div_by((uint64_t)slot / kKvGroup, groups_per_page);
    const int32_t page_size = (int32_t)groups_per_page.d * kKvGroup;
    return (page * heads + head) * page_size + (slot - page * page_size);
}

// The group of 16 tokens starting at token t of a sequence: its first row and
// whether it may be read.  Groups at or beyond the end of the keys never read
// the page table; a page number outside the cache makes its tokens absent.  An
// absent group reads the cache's first rows (any bytes) and masks them.
struct KvGroup {
    int64_t row;
    bool ok;
};

FP4Q_HD KvGroup kv_group(const int32_t* table_row, int32_t t, int32_t kv_end, const DivBy& groups_per_page,
                         int64_t num_pages, int32_t heads, int32_t head)
{
    KvGroup g{0, false};
    if (t < kv_end) {
        const uint32_t u = (uint32_t)t / kKvGroup;
        const uint32_t p = div_by(u, groups_per_page);
        const int32_t page = table_row[p];
        if (page >= 0 && page < num_pages) {
            const int32_t page_size = (int32_t)groups_per_page.d * kKvGroup;
            g.row = ((int64_t)page * heads + head) * page_size + (int64_t)(u - p * groups_per_page.d) * kKvGroup;
            g.ok = true;
        }
    }
    return g;
}

// A sequence's keys: its stated length, cut to what the page table can name
// and to the caller's bound.
FP4Q_HD int32_t kv_length(int32_t stated, int32_t max_kv, int32_t table_cols, int32_t page_size, int64_t num_pages)
{
    int64_t n = stated < 0 ? 0 : stated;
    if (n > max_kv) n = max_kv;
    const int64_t cap = (int64_t)table_cols * page_size;
    if (n > cap) n = cap;
    return num_pages > 0 ? (int32_t)n : 0;
}

// Queries of a sequence: rows [first, first + count) of q, cut to the tensor
// and to the caller's bound.
struct QueryRange {
    int32_t first, count;
};

FP4Q_HD QueryRange query_range(int32_t begin, int32_t end, int32_t total, int32_t max_q)
{
    if (begin < 0) begin = 0;
    if (begin > total) begin = total;
    if (end < begin) end = begin;
    if (end > total) end = total;
    const int32_t n = end - begin;
    return QueryRange{begin, n < max_q ? n : max_q};
}

// Keys [lo, hi) that the query at place i of n sees, of kv keys: causal puts the
// last query on the last key; a window keeps that many keys up to the query's own.
struct KeyRange {
    int32_t lo, hi;
};

FP4Q_HD KeyRange key_range(int32_t i, int32_t n, int32_t kv, int32_t causal, int32_t window)
{
    if (!causal) return KeyRange{0, kv};
    int32_t hi = kv - n + i + 1;
    if (hi < 0) hi = 0;
    int32_t lo = window > 0 ? hi - window : 0;
    if (lo < 0) lo = 0;
    return KeyRange{lo, hi};
}

// ---------------------------------------------------------------- keys of many rows
// A workgroup of many rows walks the keys of its rows in rounds of kv_round(head_dim) keys, from the
// round of the first row's first key.  Its keys may be cut into `splits` parts of `chunk` keys (a
// multiple of every round), one a workgroup.
constexpr int kTileRows = 128;           // rows (queries times heads of a group) of a workgroup
constexpr int kMaxSplits = 64;

FP4Q_HD constexpr int kv_round(int head_dim) { return head_dim == 64 ? 128 : 64; }

// Part `split` of the keys from the first row's range to the last row's; hi <= lo where it has none.
FP4Q_HD KeyRange tile_part(const KeyRange& first, const KeyRange& last, int32_t round, int32_t split, int32_t chunk)
{
    const int32_t lo = first.lo / round * round + split * chunk;
    return KeyRange{lo, last.hi < lo + chunk ? last.hi : lo + chunk};
}

struct TilePlan {
    int32_t splits, chunk;
};

// How the keys of many rows are cut, for sequences of up to max_q queries and `keys` keys.  Tiles of
// rows fill the chip by themselves, or their keys are split until they do once.
inline TilePlan plan_tiles(int64_t batch, int64_t heads, int64_t group, int64_t max_q, int64_t keys, int64_t window,
                           int head_dim)
{
    TilePlan p{1, 1 << 30};
    // a window's keys: those of the first row, one more for each later query, and what the start is
    // rounded down by
    const int64_t span = window + max_q - 1 + kv_round(head_dim) - 1;
    if (window > 0 && span < keys) keys = span;
    const int64_t blocks = batch * heads * ((max_q * group + kTileRows - 1) / kTileRows);
    int64_t want = blocks > 0 ? 256 / blocks : 1;
    if (want > keys / 512) want = keys / 512;
    if (want > kMaxSplits) want = kMaxSplits;
    if (batch > 0 && want > 65535 / batch) want = 65535 / batch;
    if (want <= 1) return p;
    p.splits = (int32_t)want;
    p.chunk = (int32_t)((keys + want * 128 - 1) / (want * 128) * 128);
    return p;
}

}  // namespace fp4q
