// The parts into which a call cuts the keys of many rows, against what those rows see: for every
// window, query count, group, length and head_dim tried, parts 0 .. splits - 1 of each tile of rows
// follow each other without a gap and hold every key from the first row's first to the last row's last.
// Prints the number of cases that were cut behind a window.
#include <cstdio>
#include <initializer_list>

#include "../../block_scaled_fp4_amax_amd/csrc/kv_index.h"

using namespace fp4q;

static long long cut_behind_window = 0;

// One sequence of kv keys and n queries in a call with these bounds.
static bool covered(int64_t batch, int64_t heads, int group, int max_q, int n, int64_t bound, int kv, int window, int dim)
{
    const TilePlan p = plan_tiles(batch, heads, group, max_q, bound, window, dim);
    if (p.splits < 1 || p.splits > kMaxSplits || p.chunk < 1 || (p.splits > 1 && p.chunk % 128)) return false;
    if (p.splits > 1 && window) ++cut_behind_window;
    const int rows = n * group, round = kv_round(dim);
    for (int r0 = 0; r0 < rows; r0 += kTileRows) {
        const int r1 = r0 + kTileRows < rows ? r0 + kTileRows : rows;
        const KeyRange first = key_range(r0 / group, n, kv, 1, window), last = key_range((r1 - 1) / group, n, kv, 1, window);
        int at = -1;
        for (int s = 0; s < p.splits; ++s) {
            const KeyRange part = tile_part(first, last, round, s, p.chunk);
            if (s == 0) {
                if (part.lo > first.lo || part.lo % round) return false;
            } else if (part.lo != at) {
                return false;
            }
            at = part.lo + p.chunk;
            if (part.hi > last.hi) return false;
        }
        if (at < last.hi) return false;                // keys that no part holds
    }
    return true;
}

int main()
{
    const int windows[] = {0, 1, 31, 480, 864, 960, 976, 984, 992, 1000, 1024, 1500, 1984, 2000, 2016, 4000, 4032, 4096, 8192};
    const int queries[] = {1, 5, 8, 9, 16, 33, 40, 64, 129, 300};
    const int dims[] = {64, 128, 256};
    const int groups[] = {1, 3, 4, 8, 33};
    struct { int batch, heads; } calls[] = {{1, 1}, {1, 8}, {2, 8}, {6, 8}, {9, 8}, {11, 8}, {64, 1}};
    long long cases = 0;
    for (int dim : dims)
        for (int w : windows)
            for (int q : queries)
                for (int g : groups)
                    for (auto c : calls)
                        for (int res = 0; res < 128; ++res) {
                            const int kv = w + q + 512 + res;
                            // bounds that the page table gives, and tight ones; fewer queries than the bound
                            for (int64_t bound : {(int64_t)kv, (int64_t)kv + 1000, (int64_t)1 << 20})
                                for (int n : {q, (q + 1) / 2}) {
                                    ++cases;
                                    if (!covered(c.batch, c.heads, g, q, n, bound, kv, w, dim)) {
                                        std::printf("lost keys: head_dim %d window %d max_q %d n %d group %d batch %d heads %d "
                                                    "bound %lld kv %d\n", dim, w, q, n, g, c.batch, c.heads, (long long)bound, kv);
                                        return 1;
                                    }
                                }
                        }
    // short sequences and rows that see nothing
    for (int dim : dims)
        for (int kv = 0; kv < 300; ++kv)
            for (int q : {1, 40, 129})
                for (int w : {0, 1, 100, 2000})
                    if (!covered(1, 8, 4, q, q, 1 << 16, kv, w, dim)) {
                        std::printf("lost keys: head_dim %d window %d max_q %d kv %d\n", dim, w, q, kv);
                        return 1;
                    }
    std::printf("ok %lld\n", cut_behind_window);
    return 0;
}
