// Host walk of the paged forward's schedule (csrc/paged_schedule.cuh): prints
// "ok" when every request's row tiles add up to what places says, for every
// prefix, by direct summation.  Built and run on the host by test_paged_schedule.py.
#include <cstdio>

#include "paged_schedule.cuh"

using namespace relation;

template <int ROWS, int KEYS, int EXTRA>
bool check() {
    using T = Tiling<ROWS, KEYS, EXTRA>;
    for (int group : {1, 2, 3, 4, 5, 7, 8, 16, 17, 40, 128, 300})
        for (int c : {0, 1, 15, 16, 31, 32, 33, 127, 128, 129, 1000, 32767})
            for (int fresh : {1, 2, 3, 15, 16, 17, 31, 64, 100, 129, 777, 2048}) {
                const int rows = fresh * group;
                int64_t sum = 0;
                for (int q = 0; q <= T::row_tiles(rows); ++q) {
                    if (T::places(c, rows, FastDiv(group), q) != sum) {
                        std::printf("rows/tile %d keys %d group %d cached %d fresh %d: first %d tiles\n", ROWS, KEYS, group,
                                    c, fresh, q);
                        return false;
                    }
                    if (q == T::row_tiles(rows)) break;
                    // by definition: the tiles up to the position of the row tile's last token
                    const int last = (rows < (q + 1) * ROWS ? rows : (q + 1) * ROWS) - 1;
                    sum += EXTRA + (c + last / group) / KEYS + 1;
                }
            }
    return true;
}

int main() {
    for (uint32_t n : {1u, 2u, 3u, 5u, 7u, 12u, 40u, 127u, 128u, 129u, 1000u, 1024u})
        for (int64_t x : {0ll, 1ll, 2ll, 126ll, 127ll, 128ll, 999999ll, 2147483646ll, 2147483647ll})
            for (int64_t y = x > 3 ? x - 3 : 0; y <= x; ++y)
                if (FastDiv(n).div((int)y) != (int)(y / n)) return std::printf("div %u %ld\n", n, (long)y), 1;
    for (int64_t n : {0, 1, 2, 5, 17})
        for (int64_t m : {1, 2, 7, 128})
            for (int64_t a : {0, 1, 5, 129, 1000})
                for (int64_t b : {0, 3, 127, 4096}) {
                    int64_t s = 0;
                    for (int64_t i = 0; i < n; ++i) s += (a * i + b) / m;
                    if (s != floor_sum(n, m, a, b)) return std::printf("floor_sum %ld %ld %ld %ld\n", (long)n, (long)m, (long)a, (long)b), 1;
                }
    if (!check<256, 128, 2>() || !check<64, 64, 1>() || !check<16, 64, 0>()) return 1;
    // The workers' stretches tile the line, differ by one tile at most, and owner() inverts begin().
    for (int total : {0, 1, 2, 3, 7, 152, 153, 1000, 4097})
        for (int workers : {1, 2, 5, 152, 1824})
            for (int least : {1, 2, 3}) {
                const Share s(total, workers, least);
                int at = 0, lo = total, hi = 0;
                for (int w = 0; w < workers; ++w) {
                    const int n = s.begin(w + 1) - s.begin(w);
                    if (s.begin(w) != at || n < 0) return std::printf("share %d %d %d: worker %d\n", total, workers, least, w), 1;
                    for (int x = at; x < at + n; ++x)
                        if (s.owner(x) != w) return std::printf("owner %d %d %d: tile %d\n", total, workers, least, x), 1;
                    at += n;
                    if (w < s.used) lo = n < lo ? n : lo, hi = n > hi ? n : hi;
                }
                if (at != total || hi - lo > 1) return std::printf("share %d %d %d\n", total, workers, least), 1;
            }
    std::printf("ok\n");
    return 0;
}
