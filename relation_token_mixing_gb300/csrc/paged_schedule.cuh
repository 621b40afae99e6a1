// How the paged forward's work is cut among its workers.
//
// Unit: one (request, cache head, row tile): `rows_per_tile` of the request's
// packed rows (row = token * group + head in the group) against the history its
// last token sees, in key tiles of `keys`.  All units' key tiles in a fixed order
// (request, cache head, row tile, key tile), each unit preceded by the places that
// its beginning and end are worth, form one line, and the workers take consecutive
// stretches of it that differ by one place at most, whatever the requests' lengths
// are.  A unit that a boundary cuts is merged from its pieces afterwards.
//
// The line's length is known on the device only: every block sums the requests'
// tiles itself, so the host launches a fixed grid.
#pragma once

#include <stdint.h>

namespace relation {

// Quotients by a number known on the host, for dividends of 31 bits: with s =
// ceil(log2 n) and m = ceil(2^(31 + s) / n), x / n = (x m) >> (31 + s) for all x < 2^31
// (m n exceeds 2^(31 + s) by less than 2^s, so the error stays below 1 / n).
struct FastDiv {
    uint32_t n, m, shift;
    FastDiv() = default;
    explicit FastDiv(uint32_t d) : n(d), shift(0) {
        while ((1ull << shift) < d) ++shift;
        m = (uint32_t)(((1ull << (31 + shift)) + d - 1) / d);
    }
    __host__ __device__ __forceinline__ int div(int x) const {
        return (int)(((uint64_t)(uint32_t)x * m) >> (31 + shift));
    }
};

// sum_{i < n} floor((a i + b) / m) for n, a, b >= 0, m >= 1, by the Euclidean
// recursion: whole multiples of m leave a and b, then the lattice points under the
// line are counted along the other axis.
__host__ __device__ inline int64_t floor_sum(int64_t n, int64_t m, int64_t a, int64_t b) {
    int64_t sum = 0;
    while (n > 0) {
        sum += (a / m) * (n * (n - 1) / 2) + (b / m) * n;
        a %= m;
        b %= m;
        const int64_t top = a * n + b;
        if (top < m) break;
        n = top / m;
        b = top - n * m;
        const int64_t t = m;
        m = a;
        a = t;
    }
    return sum;
}

// kExtra: the places before each unit's key tiles.
template <int kRowsPerTile, int kKeys, int kExtra>
struct Tiling {
    static constexpr int extra = kExtra;
    // Key tiles of row tile q of a request with `rows` packed rows and c cached tokens.
    __host__ __device__ static int tiles(int c, int rows, const FastDiv& group, int q) {
        const int last = (rows < (q + 1) * kRowsPerTile ? rows : (q + 1) * kRowsPerTile) - 1;
        return (int)(((uint32_t)c + (uint32_t)group.div(last) + kKeys) / kKeys);
    }
    __host__ __device__ static int row_tiles(int rows) { return (rows + kRowsPerTile - 1) / kRowsPerTile; }
    // Places of the first n row tiles.  Key tiles of full row tiles: ceil((c + ceil(x / g)) / k)
    // with x = (q + 1) rows_per_tile is ceil((c g + x) / (g k)).
    __host__ __device__ static int64_t places(int c, int rows, const FastDiv& group, int n) {
        const int full = n < rows / kRowsPerTile ? n : rows / kRowsPerTile;
        int64_t s = (int64_t)n * kExtra;
        if (full <= 2) {
            for (int q = 0; q < full; ++q) s += tiles(c, rows, group, q);
        } else {
            const int64_t m = (int64_t)group.n * kKeys;
            s += floor_sum(full, m, kRowsPerTile, (int64_t)c * group.n + kRowsPerTile + m - 1);
        }
        return n > full ? s + tiles(c, rows, group, full) : s;
    }
};

// A line of `total` tiles cut among `workers`, at least min_tiles each while there
// are enough: the first `extra` of the `used` workers take one tile more than `each`.
struct Share {
    int used, each, extra;
    __host__ __device__ Share(int total, int workers, int min_tiles) {
        used = total / min_tiles;
        used = used < 1 ? 1 : (used > workers ? workers : used);
        each = total / used;
        extra = total - each * used;
    }
    __host__ __device__ int begin(int w) const {
        return w >= used ? each * used + extra : w * each + (w < extra ? w : extra);
    }
    // The worker that has tile x (x below the line's end).
    __host__ __device__ int owner(int x) const {
        const int wide = extra * (each + 1);
        return x < wide ? x / (each + 1) : extra + (x - wide) / each;
    }
};

}  // namespace relation
