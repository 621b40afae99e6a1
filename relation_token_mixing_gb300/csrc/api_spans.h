// Checks of pointer arguments that the serving entry points share.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace relation {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

struct ByteSpan {
    const void* p;
    size_t n;
};

inline bool overlap(const ByteSpan& a, const ByteSpan& b) {
    if (a.p == nullptr || b.p == nullptr || a.n == 0 || b.n == 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x < y + b.n && y < x + a.n;
}

// Every output apart from every input and every other output.
inline bool disjoint(const ByteSpan* in, int n_in, const ByteSpan* out, int n_out) {
    for (int o = 0; o < n_out; ++o) {
        for (int i = 0; i < n_in; ++i)
            if (overlap(out[o], in[i])) return false;
        for (int q = o + 1; q < n_out; ++q)
            if (overlap(out[o], out[q])) return false;
    }
    return true;
}

}  // namespace relation
