// How a call cuts the keys of drafted trees, on the host: for batches of every kind (empty sequences, more than a
// wave's 64) the parts that the lengths give fit the launch and its scratch and hold every round of every tile once; and the
// launches fit the device's limits (2^32 lanes a dimension, 65535 workgroups in the second and third) with a
// workgroup for every tile of every head and sequence at all sizes that a call may have.
// Prints the number of calls that were cut.
#include <cstdint>
#include <cstdio>
#include <initializer_list>
#include <random>
#include <vector>

#include "../../block_scaled_fp4_amax_amd/csrc/kv_index.h"

using namespace fp4q;

struct Seq {
    int kv, n;
};

static bool covered(const std::vector<Seq>& seqs, int64_t heads, int group, int max_q, int max_kv, int window, int dim, long long& cut)
{
    const int round = kv_round(dim);
    const int64_t most = (int64_t)window + max_q + round, keys = window && most < max_kv ? most : max_kv;
    const TreePlan p = plan_tree((int64_t)seqs.size(), heads, (int64_t)max_q * group, keys, dim);
    if (p.slots == 0) return true;
    ++cut;
    int64_t rounds = 0, tiles = 0;
    for (const Seq& s : seqs) {
        rounds += (int64_t)tree_rounds(s.kv, s.n, window, round) * tile_count(s.n * group);
        tiles += tile_count(s.n * group);
    }
    if (rounds >= (int64_t)1 << 31) return false;
    const int share = tree_share((int)rounds, (int)tiles, p.slots, (int)heads);
    if (share < kMinRounds) return false;
    int64_t parts = 0;
    for (const Seq& s : seqs) {
        if (s.n == 0) continue;
        const int each = parts_of(tree_rounds(s.kv, s.n, window, round), share);
        parts += (int64_t)each * tile_count(s.n * group);
        const KeyRange first = tree_context(s.kv, s.n, window, 0);
        const KeyRange last{tree_context(s.kv, s.n, window, s.n).lo, s.kv};
        int at = first.lo / round * round;
        for (int i = 0; i < each; ++i) {
            const KeyRange part = tree_part(first, last, round, i, each);
            if (part.lo != at || part.lo % round) return false;
            if (part.hi > s.kv) return false;
            if (i + 1 < each) {
                if (part.hi <= part.lo || (part.hi - part.lo) % round) return false;
                at = part.hi;
            } else if (part.hi != s.kv && s.kv > at) {
                return false;
            }
        }
    }
    return parts <= p.parts && p.parts * heads < (int64_t)1 << 23;
}

static bool fits(int64_t batch, int64_t heads, int64_t rows, int64_t keys, int dim)
{
    const TreePlan p = plan_tree(batch, heads, rows, keys, dim);
    const TreeGrid g = tree_grid(p, batch, heads, rows);
    if ((int64_t)g.x * 512 >= (int64_t)1 << 32 || g.y > 65535 || g.z > 65535) return false;
    if (p.slots) return g.x == p.parts * heads && g.y == 1 && g.z == 1;
    return g.x == heads && g.z == batch && (int64_t)g.y * kTileRows >= rows && (int64_t)(g.y - 1) * kTileRows < rows;
}

int main()
{
    std::mt19937 rng(1);
    const auto below = [&](int n) { return (int)(rng() % (unsigned)n); };
    long long cut = 0;
    for (int dim : {64, 128, 256})
        for (int batch : {1, 2, 9, 63, 64, 65, 70, 128, 130, 300})
            for (int heads : {1, 2, 8, 40})
                for (int group : {1, 3, 8})
                    for (int window : {0, 1, 100, 1000, 5000})
                        for (int top : {300, 2100, 20000, 1 << 27})
                            for (int turn = 0; turn < 4; ++turn) {
                                const int max_q = 33 + below(100);
                                std::vector<Seq> seqs;
                                for (int b = 0; b < batch; ++b) {
                                    const int kind = below(8);
                                    Seq s{below(top) + 1, below(max_q) + 1};
                                    if (kind == 0) s.n = 0;
                                    if (kind == 1) s.kv = below(s.n + 1);
                                    if (kind == 2) s.kv = 0;
                                    if (kind == 3 || turn == 3) s = Seq{top, max_q};
                                    seqs.push_back(s);
                                }
                                if (!covered(seqs, heads, group, max_q, top, window, dim, cut)) {
                                    std::printf("head_dim %d batch %d heads %d group %d window %d keys %d max_q %d\n", dim, batch, heads,
                                                group, window, top, max_q);
                                    return 1;
                                }
                            }
    // the largest calls: batch <= 65535, batch * heads < 2^24, rows <= 2^22, heads <= 65535, keys <= 2^27
    for (int dim : {64, 128, 256})
        for (int64_t batch : {1, 2, 255, 256, 512, 16385, 65535})
            for (int64_t heads : {1, 8, 255, 256, 1024, 65535})
                for (int64_t rows : {33, 128, 129, 262144, 1 << 22})
                    for (int64_t keys : {0, 511, 513, 100000, 1 << 27})
                        if (batch * heads < (1 << 24) && !fits(batch, heads, rows, keys, dim)) {
                            std::printf("launch: head_dim %d batch %lld heads %lld rows %lld keys %lld\n", dim, (long long)batch,
                                        (long long)heads, (long long)rows, (long long)keys);
                            return 2;
                        }
    std::printf("ok %lld\n", cut);
    return 0;
}
