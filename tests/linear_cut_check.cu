// Host walk of how packed calls are cut (csrc/linear_cut.h): prints "ok" when, for offsets of every kind, no
// segment leaves the list that the call has room for, the requests of more than one segment fit theirs, every
// row is in one segment at most, and offsets that ascend lose none.  Built and run on the host by test_linear_cut.py.
// With an argument, every request is taken as if it were the first: what the list must not be given.
#include <cstdio>
#include <random>
#include <vector>

#include "linear_cut.h"

using namespace relation::lin;

static bool blind = false;
static long long calls = 0, cut_calls = 0, refused = 0;

static bool walk(const std::vector<int>& starts, int N, int H, int max_fresh, int sms) {
    const int R = (int)starts.size() - 1;
    const Cut c = cut_of(R, N, H, max_fresh, sms);
    ++calls;
    if (!c.segmented) return true;
    ++cut_calls;
    std::vector<char> taken(N, 0);
    long long at = 0, joins = 0;
    int end = 0;
    bool ascending = true;
    for (int r = 0; r < R; ++r) {
        const Span sp = span_between(starts[r], starts[r + 1], N, max_fresh);
        ascending = ascending && sp.count >= 0;
        const Segments sg = segments_of(sp, blind ? 0 : end, c.seg_tokens);
        end = std::max(end, sp.end());
        refused += sg.refused;
        if (sg.refused && ascending) return std::printf("request %d of ascending offsets is refused\n", r), false;
        if (sp.count > kFewTokens && !sg.refused && (sg.count < 1 || sg.tokens % kChunk || sg.tokens > c.seg_tokens + kChunk ||
                                                      sg.count >= kMaxSegs))
            return std::printf("request %d of %d tokens: %d segments of %d\n", r, sp.count, sg.count, sg.tokens), false;
        if (at + sg.count > c.items)
            return std::printf("N %d H %d R %d: request %d has segments %lld to %lld of %d\n", N, H, R, r, at, at + sg.count,
                               c.items), false;
        for (int k = 0; k < sg.count; ++k) {
            const int first = sp.first + k * sg.tokens, count = std::min(sg.tokens, sp.count - k * sg.tokens);
            if (count < 1 || first < 0 || first + count > N) return std::printf("request %d: segment %d\n", r, k), false;
            for (int x = first; x < first + count; ++x)
                if (taken[x]++) return std::printf("row %d is in two segments\n", x), false;
        }
        at += sg.count;
        joins += sg.count > 1;
        if (joins > c.joins) return std::printf("%lld requests to join, room for %d\n", joins, c.joins), false;
        if (ascending && sp.count > kFewTokens)
            for (int x = sp.first; x < sp.end(); ++x)
                if (!taken[x]) return std::printf("row %d is in no segment\n", x), false;
    }
    return true;
}

int main(int argc, char**) {
    blind = argc > 1;
    for (int N : {700, 1000, 4096, 32768, 100003})
        for (int H : {1, 2, 8, 16}) {
            if (!walk({0, N, 0, N}, N, H, 0 + N, 152)) return 1;           // all rows twice
            if (!walk({0, N, 0, N, 0, N, 0, N}, N, H, N, 152)) return 1;   // and four times
            if (!walk({0, N - 1, 1, N, N / 2, N}, N, H, N, 152)) return 1;
            if (!walk({N, 0, N}, N, H, N, 152)) return 1;
        }
    std::mt19937 gen(7);
    const auto to = [&](int n) { return (int)(gen() % (unsigned)n); };
    for (int round = 0; round < 20000; ++round) {
        const int R = 1 + to(round % 2 ? 6 : 300), N = 1 + to(round % 3 ? 6000 : 40000), H = 1 + to(16), sms = round % 5 ? 152 : 1;
        std::vector<int> starts(R + 1);
        for (int& s : starts) s = to(N + 1);
        const int kind = round % 4;
        if (kind != 0) std::sort(starts.begin(), starts.end());                        // ascending
        if (kind == 2) for (int k = 0; k < 3; ++k) starts[to(R + 1)] = to(2 * N) - N / 2;  // but for a few
        if (kind == 3) for (int r = 1; r <= R; r += 2) starts[r] = N - to(N / 4 + 1);   // up and down
        const int longest = round % 7 ? N : 1 + to(N);
        if (!walk(starts, N, H, longest, sms)) return 1;
    }
    if (cut_calls < 1000 || (refused < 1000 && !blind)) return std::printf("%lld calls, %lld cut, %lld refused\n", calls, cut_calls, refused), 1;
    std::printf("ok\n");
    return 0;
}
