// Block tables and slot maps of a paged Relation Cache, built on the device from
// the requests' lengths (the cache of "Ask Self, Ask Others", Sec. 5.3 and
// Appendix A.5, held in pages).
//
// Two exclusive sums over the requests place everything: of the new tokens
// (starts) and of the pages they newly need (which free page is whose).  Every
// block repeats both sums over all R requests (a pass over 8 R bytes that sit in
// L2, one barrier pair per 1024 requests) and then writes its own 1024 tokens, so
// one launch with no exchange between blocks does it all.  A token finds its
// request by a running maximum over the marks that the requests' first tokens
// leave in shared memory.  A page's free-list entry is written to the block table
// by the page's first token, which is always new.  Measured: 3.2 us for 64 decoding requests, 3.8
// for 1024 with up to 64 new tokens each; a launch is 2.5 of either.
#include "paged.h"

namespace relation {
namespace {

constexpr int kPlanThreads = 1024;

__global__ void __launch_bounds__(kPlanThreads)
    paged_plan_kernel(PagedProblem pp, const int* __restrict__ cached, const int* __restrict__ fresh,
                      const int* __restrict__ free_pages, int64_t free_count, int* table, int* __restrict__ starts,
                      int64_t* __restrict__ slots, int* __restrict__ positions, int* __restrict__ used,
                      unsigned int* status) {
    __shared__ int mark[kPlanThreads];       // 1 + request whose tokens begin here (0: none)
    __shared__ int mark_first[kPlanThreads];  // its first token's packed index
    __shared__ int mark_cached[kPlanThreads];
    __shared__ int mark_page[kPlanThreads];  // index of its first new page in the free list
    __shared__ int64_t warp_tok[32], warp_pg[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t t0 = (int64_t)blockIdx.x * kPlanThreads;
    const int capacity = pp.width << pp.page_shift;
    mark[tid] = 0;
    int64_t tok_base = 0, pg_base = 0;
    for (int r0 = 0; r0 < pp.R; r0 += kPlanThreads) {
        const int r = r0 + tid;
        int c = 0, f = 0, held = 0, grown = 0;
        if (r < pp.R) {
            c = cached[r];
            f = fresh[r];
            if (c < 0 || f < 0) {
                if (blockIdx.x == 0) record_status(status, kDevBadPosition);
                c = max(c, 0);
                f = 0;
            }
            held = min((int)(((int64_t)c + pp.page_mask) >> pp.page_shift), pp.width);
            grown = min((int)(((int64_t)c + f + pp.page_mask) >> pp.page_shift), pp.width) - held;
        }
        int64_t tok = f, pg = grown;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t a = __shfl_up_sync(0xffffffffu, tok, o), b = __shfl_up_sync(0xffffffffu, pg, o);
            if (lane >= o) tok += a, pg += b;
        }
        __syncthreads();  // the previous round's sums have been read (and mark is cleared)
        if (lane == 31) warp_tok[warp] = tok, warp_pg[warp] = pg;
        __syncthreads();
        int64_t a = warp_tok[lane], b = warp_pg[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
            if (lane >= o) a += x, b += y;
        }
        const int64_t tok_before = warp ? __shfl_sync(0xffffffffu, a, warp - 1) : 0;
        const int64_t pg_before = warp ? __shfl_sync(0xffffffffu, b, warp - 1) : 0;
        const int64_t last = tok_base + tok_before + tok, first = last - f;
        const int64_t page_first = pg_base + pg_before + pg - grown;
        if (r < pp.R) {
            if ((r0 / kPlanThreads) % gridDim.x == blockIdx.x) {
                starts[r + 1] = (int)min(last, (int64_t)INT32_MAX);
                if (r == 0) starts[0] = 0;
            }
            if (f > 0 && first < t0 + kPlanThreads && last > t0) {
                const int at = (int)(max(first, t0) - t0);
                mark[at] = r + 1;
                mark_first[at] = (int)first;
                mark_cached[at] = c;
                mark_page[at] = (int)min(page_first, (int64_t)INT32_MAX);
            }
        }
        tok_base += __shfl_sync(0xffffffffu, a, 31);
        pg_base += __shfl_sync(0xffffffffu, b, 31);
    }
    if (blockIdx.x == 0 && tid == 0) {
        used[0] = (int)min(pg_base, (int64_t)INT32_MAX);
        if (tok_base > pp.N) record_status(status, kDevBadPosition);
    }
    __shared__ int warp_mark[32];
    __syncthreads();
    int at = mark[tid] ? tid : -1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, at, o);
        if (lane >= o) at = max(at, x);
    }
    if (lane == 31) warp_mark[warp] = at;
    __syncthreads();
    const int before = __reduce_max_sync(0xffffffffu, lane < warp ? warp_mark[lane] : -1);
    at = max(at, before);
    const int64_t n = t0 + tid;
    if (n >= pp.N) return;
    int64_t slot = -1;
    int pos = 0;
    if (n < tok_base && at >= 0) {
        const int r = mark[at] - 1, c = mark_cached[at];
        const int64_t p64 = (int64_t)c + (n - mark_first[at]);
        pos = (int)min(p64, (int64_t)INT32_MAX);
        if (p64 < capacity) {
            const int k = pos >> pp.page_shift;
            const int held = min((int)(((int64_t)c + pp.page_mask) >> pp.page_shift), pp.width);
            int* entry = table + (size_t)r * pp.width + k;
            int page;
            if (k < held) {
                page = *entry;
            } else {
                const int64_t idx = (int64_t)mark_page[at] + (k - held);
                page = idx < free_count ? free_pages[idx] : -1;
                if ((pos & pp.page_mask) == 0) *entry = page;
            }
            if (page >= 0 && page < pp.pages) slot = ((int64_t)page << pp.page_shift) + (pos & pp.page_mask);
        }
    }
    slots[n] = slot;
    positions[n] = pos;
}

}  // namespace

cudaError_t launch_paged_plan(const PagedProblem& pp, const int* cached, const int* fresh, const int* free_pages,
                              int64_t free_count, int* table, int* starts, int64_t* slots, int* positions, int* used,
                              unsigned int* status, cudaStream_t s) {
    const unsigned blocks = pp.N ? (unsigned)(((int64_t)pp.N + kPlanThreads - 1) / kPlanThreads) : 1u;
    paged_plan_kernel<<<blocks, kPlanThreads, 0, s>>>(pp, cached, fresh, free_pages, free_count, table, starts, slots,
                                                     positions, used, status);
    return cudaGetLastError();
}

}  // namespace relation
