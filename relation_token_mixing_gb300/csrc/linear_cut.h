// How a packed call of Linear Relation over a pool of states is cut (host and device arithmetic): which requests
// are followed, in how many segments, and how many of them a call can have.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace relation {
namespace lin {

// Tokens that the recurrence takes one by one. 64 requests, 16 heads of 64, of 16 tokens each: 18.6 us so, 27.1 as a
// chunk; of 24: 26.3 and 27.5, but room for 24 tokens' vectors leaves the long requests' kernels beside it less of an
// SM's memory (prompts of up to 2048 tokens, 8 heads of 60: 134 us against 125).
constexpr int kFewTokens = 16;

constexpr int kChunk = 64;  // tokens
constexpr int kMaxSegs = 1 << 15;
constexpr int kBlocksPerSm = 2;  // of the chunks' kernel
constexpr int kLeastCut = 256, kUncut = 640;

// A request's rows; count = -1: they cannot be followed.
struct Span {
    int first, count;
    __host__ __device__ int end() const { return count > 0 ? first + count : 0; }
};
__host__ __device__ inline Span span_between(int first, int next, int N, int max_fresh) {
    const int64_t n = (int64_t)next - first;
    if (first < 0 || n < 0 || next > N || n > max_fresh) return Span{0, -1};
    return Span{first, (int)n};
}

// The segments of a request with more than kFewTokens tokens. before: the end of the rows of all earlier requests; one
// that begins before it has none (refused).  So no row is in two requests' segments, and all requests have
// at most N / seg_tokens + min(R, N / (kFewTokens + 1)) of them, of which min(R, N / (seg_tokens + 1)) requests have
// more than one.
struct Segments {
    int count, tokens;  // of each but the last
    bool refused;
};
__host__ __device__ inline Segments segments_of(Span sp, int before, int seg_tokens) {
    if (sp.count <= kFewTokens) return Segments{0, 0, false};
    if (sp.first < before) return Segments{0, 0, true};
    const int chunks = (sp.count - 1) / kChunk + 1, segs = (sp.count - 1) / seg_tokens + 1, per = (chunks - 1) / segs + 1;
    return Segments{(chunks - 1) / per + 1, per * kChunk, false};
}

// How a packed call is cut: requests longer than `seg_tokens` in equal segments of that many at most.
struct Cut {
    bool chunked;     // a request may have more than kFewTokens new tokens
    bool segmented;   // and is worth cutting
    int seg_tokens, items;  // items: segments of all requests at most, where no row is two requests'
    int joins;        // requests of more than one segment
};
inline Cut cut_of(int R, int N, int H, int max_fresh, int num_sms) {
    Cut c{};
    c.chunked = max_fresh > kFewTokens;
    if (!c.chunked) return c;
    // share: a block's equal share of all tokens. A request of up to 1.5 of it, or of up to kUncut tokens, is left whole:
    // cutting costs the state pass (0.6 of the output pass), the join and two more launches (4 requests, 16 heads
    // of 64: 512 tokens each 25 us whole and 33 cut, 640: 31 and 33, 768: 36 and 35, 1536: 70 and 46).
    // One request is cut in equal shares; several in halves of one, kLeastCut at least, as their blocks are evened out by
    // the order (prompts of up to 2048, 8 heads of 60: 125 us, in whole shares 134, in 512 at least 131, in 128 at
    // least 125, but four requests of 1536 46 against 50; uncut 156).
    const int64_t share = (int64_t)N * H / (kBlocksPerSm * num_sms);
    int64_t seg = std::max<int64_t>(kLeastCut, ((R > 1 ? share / 2 : share) + kChunk - 1) / kChunk * kChunk);
    seg = std::max<int64_t>(seg, ((int64_t)max_fresh / (kMaxSegs - 1) + kChunk) / kChunk * kChunk);
    c.seg_tokens = (int)std::min<int64_t>(seg, (INT32_MAX - kChunk) / kChunk * kChunk);
    c.segmented = max_fresh > std::max<int64_t>({kUncut, share + share / 2, c.seg_tokens});
    c.items = c.segmented ? (int)std::min<int64_t>((int64_t)N / c.seg_tokens + std::min(R, N / (kFewTokens + 1)), INT32_MAX) : R;
    c.joins = std::min(R, N / (c.seg_tokens + 1));
    return c;
}

}  // namespace lin
}  // namespace relation
