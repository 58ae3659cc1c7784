// tree_context() against its definition: a query that sees c of n drafted tokens sees, of the kv - n
// keys before them, all, or the last that make `window` keys with those c (one at least).
#include <cstdint>
#include <cstdio>
#include <initializer_list>

#include "../../block_scaled_fp4_amax_amd/csrc/kv_index.h"

int main()
{
    for (int kv = 0; kv <= 40; ++kv)
        for (int n = 0; n <= 45; ++n)
            for (int window = 0; window <= 50; ++window)
                for (int c = 0; c <= n; ++c) {
                    const fp4q::KeyRange r = fp4q::tree_context(kv, n, window, c);
                    int count = kv - n > 0 ? kv - n : 0;
                    const int end = count;
                    if (window > 0) {
                        int left = window - (c > 0 ? c : 1);
                        if (left < 0) left = 0;
                        if (left < count) count = left;
                    }
                    if (r.hi != end || r.lo != end - count) {
                        std::printf("kv %d n %d window %d c %d: [%d, %d)\n", kv, n, window, c, r.lo, r.hi);
                        return 1;
                    }
                    // the tile's ranges hold every row's
                    const fp4q::KeyRange a = fp4q::tree_context(kv, n, window, 0), b = fp4q::tree_context(kv, n, window, n);
                    if (a.lo > r.lo || b.lo < r.lo) return 2;
                }
    // the ends of the types
    for (int kv : {0, 1, (1 << 27), 0x7FFFFFFF})
        for (int n : {0, 1, 1 << 22})
            for (int window : {0, 1, 0x7FFFFFFF})
                for (int c : {0, 1, n}) {
                    const fp4q::KeyRange r = fp4q::tree_context(kv, n, window, c);
                    if (r.lo < 0 || r.lo > r.hi || r.hi != (kv > n ? kv - n : 0)) return 3;
                }
    std::puts("ok");
    return 0;
}
