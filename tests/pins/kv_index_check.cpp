// The index functions of the paged cache against plain loops and divisions,
// on the host: every address formed from any slot, page number, length or
// query range lies within the buffers.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "../../block_scaled_fp4_amax_amd/csrc/kv_index.h"

using namespace fp4q;

#define CHECK(x)                                                            \
    do {                                                                    \
        if (!(x)) {                                                         \
            std::printf("line %d: %s\n", __LINE__, #x);                     \
            return 1;                                                       \
        }                                                                   \
    } while (0)

int main()
{
    // division by the groups of a page, over all group numbers' ends and a sample
    for (uint32_t d = 1; d <= (uint32_t)kKvMaxPage / kKvGroup; ++d) {
        const DivBy k = make_div(d);
        const uint32_t top = (uint32_t)(kKvMaxTokens / kKvGroup);
        for (uint32_t u = 0; u <= top; u += (u < 4096 || u > top - 4096) ? 1 : 977) CHECK(div_by(u, k) == u / d);
        for (uint32_t q = 1; q * d <= top && q < 4096; ++q)
            CHECK(div_by(q * d, k) == q && div_by(q * d - 1, k) == q - 1);
    }
    for (uint32_t d = 1; d <= (uint32_t)kKvMaxPage / kKvGroup; ++d) {
        const DivBy64 k = make_div64(d);
        const uint64_t top = (uint64_t)1 << 43;                // pages below 2^31 of at most 4096 tokens
        for (uint64_t q = 0; q < 3000; ++q)
            for (uint64_t g : {q, top - q, q * d, q * d + d - 1, top / d * d - q * d, top / d * d - q * d - 1, q * 2862933555777941757u % top})
                if (g <= top) CHECK(div_by(g, k) == g / d);
    }
    // slots
    const int64_t big[] = {INT64_MIN, -((int64_t)1 << 40), -1, 0, 1, 47, 48, 49, 7 * 48 - 1, 7 * 48, INT64_MAX};
    for (int64_t slot : big)
        for (int h = 0; h < 3; ++h) {
            const int64_t row = kv_row_of_slot(slot, 7 * 48, make_div64(48 / kKvGroup), 3, h);
            if (slot < 0 || slot >= 7 * 48) CHECK(row == -1);
            else CHECK(row == (slot / 48 * 3 + h) * 48 + slot % 48 && row < 7 * 3 * 48);
        }
    // groups of 16 tokens: bad pages are absent, entries at or beyond the end are not read
    const int pages = 5, heads = 2, page = 48, cols = 4;
    std::vector<int32_t> table = {4, -1, 5, INT32_MAX};
    for (int h = 0; h < heads; ++h)
        for (int end = 0; end <= cols * page; ++end)
            for (int t = 0; t < end + 64; t += 16) {
                // a table cut to what may be read: an access beyond is caught by the vector's bounds
                std::vector<int32_t> cut(table.begin(), table.begin() + (end + page - 1) / page);
                cut.push_back(3);                      // a sentinel that must not be used
                const KvGroup g = kv_group(cut.data(), t, end, make_div(page / kKvGroup), pages, heads, h);
                const bool ok = t < end && t / page < cols && table[t / page] >= 0 && table[t / page] < pages;
                CHECK(g.ok == ok);
                CHECK(g.row >= 0 && g.row + kKvGroup <= (int64_t)pages * heads * page);
                if (ok) CHECK(g.row == ((int64_t)table[t / page] * heads + h) * page + t % page);
            }
    // lengths and query ranges
    const int32_t any[] = {INT32_MIN, -1, 0, 1, 5, 100, 191, 192, 193, INT32_MAX};
    for (int32_t n : any)
        for (int32_t m : {0, 1, 150, INT32_MAX}) {
            const int32_t l = kv_length(n, m, cols, page, pages);
            CHECK(l >= 0 && l <= m && l <= cols * page && (n < 0 || l <= n));
            CHECK(kv_length(n, m, cols, page, 0) == 0);
            for (int32_t e : any) {
                const QueryRange q = query_range(n, e, 100, m);
                CHECK(q.first >= 0 && q.count >= 0 && q.count <= m && (int64_t)q.first + q.count <= 100);
            }
        }
    // what a query sees, against the definition
    for (int kv = 0; kv < 40; ++kv)
        for (int n = 1; n < 50; ++n)
            for (int i = 0; i < n; ++i)
                for (int w : {0, 1, 7, 100})
                    for (int c : {0, 1}) {
                        const KeyRange r = key_range(i, n, kv, c, c ? w : 0);
                        const int pos = kv - n + i;
                        for (int j = 0; j < kv; ++j) {
                            const bool see = !c || (j <= pos && (w == 0 || j > pos - w));
                            CHECK(see == (j >= r.lo && j < r.hi));
                        }
                        CHECK(r.lo >= 0 && r.hi >= 0 && r.hi <= kv);
                    }
    std::printf("ok\n");
    return 0;
}
