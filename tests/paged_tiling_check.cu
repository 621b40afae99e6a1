// Host check of the paged forward's schedule (csrc/paged_schedule.cuh) with the tilings and the least
// shares that the kernels use, and histories up to 2^31 tokens: prints "ok" when the places before each
// row tile equal direct summation and the workers' stretches tile the line.  Built and run on the host
// by test_paged_tilings.py.
#include <cstdio>

#include "paged_schedule.cuh"

using namespace relation;

template <int ROWS, int KEYS, int EXTRA>
bool check() {
    using T = Tiling<ROWS, KEYS, EXTRA>;
    for (int group : {1, 2, 3, 5, 8, 16, 17, 128, 1024})
        for (int64_t c : {0ll, 1ll, 63ll, 64ll, 65ll, 127ll, 129ll, 4095ll, 100003ll, 2147480000ll})
            for (int fresh : {1, 2, 16, 17, 63, 130, 1025}) {
                const int rows = fresh * group;
                int64_t sum = 0;
                for (int q = 0; q < T::row_tiles(rows); ++q) {
                    if (T::places((int)c, rows, FastDiv(group), q) != sum)
                        return std::printf("rows/tile %d keys %d extra %d group %d cached %lld fresh %d: tile %d\n", ROWS,
                                           KEYS, EXTRA, group, (long long)c, fresh, q), false;
                    const int64_t last = (rows < (q + 1) * ROWS ? rows : (q + 1) * ROWS) - 1, n = (c + last / group) / KEYS + 1;
                    if (T::tiles((int)c, rows, FastDiv(group), q) != n) return std::printf("tiles of %d\n", q), false;
                    sum += EXTRA + n;
                }
                if (T::places((int)c, rows, FastDiv(group), T::row_tiles(rows)) != sum) return std::printf("all\n"), false;
            }
    return true;
}

int main() {
    // bf16 long requests; float32 up to 16 rows, and longer ones at up to 96 and at 128 columns
    if (!check<256, 128, 2>() || !check<16, 64, 1>() || !check<64, 64, 1>() || !check<128, 64, 1>()) return 1;
    for (int total : {0, 1, 3, 4, 5, 607, 608, 609, 99999, 2147483647})
        for (int workers : {152, 304, 456, 1824})
            for (int least : {1, 2, 4}) {
                const Share s(total, workers, least);
                int lo = total, hi = 0;
                for (int w = 0; w < workers; ++w) {
                    const int a = s.begin(w), b = s.begin(w + 1);
                    if (a > b || (b > a && (s.owner(a) != w || s.owner(b - 1) != w)))
                        return std::printf("share %d %d %d: worker %d\n", total, workers, least, w), 1;
                    if (w < s.used) lo = b - a < lo ? b - a : lo, hi = b - a > hi ? b - a : hi;
                }
                if (s.begin(0) != 0 || s.begin(workers) != total || hi - lo > 1 || (total >= least && lo < least))
                    return std::printf("share %d %d %d\n", total, workers, least), 1;
            }
    std::printf("ok\n");
    return 0;
}
