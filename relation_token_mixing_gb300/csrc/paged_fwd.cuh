// Shared device parts of the paged forward kernels: the schedule in shared
// memory, walking a worker's part of it, and the merge of cut units.
#pragma once

#include <math.h>

#include "paged.h"
#include "paged_schedule.cuh"
#include "ptx_sm100.cuh"

namespace relation {
namespace paged {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct FwdView {
    PagedProblem pp;
    const int *table, *starts, *cached;
    int max_fresh;
    int rows_above, rows_to;  // this kernel's requests: packed rows in (rows_above, rows_to]
    unsigned int* status;
};

// One request as the kernels see it (rows == 0: none of theirs).
struct Request {
    int first;  // packed token its new tokens begin at
    int c;      // cached tokens
    int rows;   // new tokens * group
};

// Lengths that cannot be followed give rows = 0 and are reported.
__device__ __forceinline__ Request request_of(const FwdView& v, int r) {
    Request q{v.starts[r], v.cached[r], 0};
    const int last = v.starts[r + 1];
    const int64_t f = (int64_t)last - q.first;
    if (q.first < 0 || f < 0 || last > v.pp.N || q.c < 0 || f > v.max_fresh ||
        q.c + f > ((int64_t)v.pp.width << v.pp.page_shift)) {
        record_status(v.status, kDevBadPosition);
        return q;
    }
    const int64_t rows = f * v.pp.group;
    if (rows > v.rows_above && rows <= v.rows_to) q.rows = (int)rows;
    return q;
}

// prefix[r] = key tiles of requests 0..r for one cache head.  All threads of the
// block; sums: one int per warp.  Returns the total (saturated to int).
template <typename Tl>
__device__ __forceinline__ int schedule_build(const FwdView& v, int* prefix, int* sums) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = (int)blockDim.x >> 5;
    int64_t base = 0;
    for (int r0 = 0; r0 < v.pp.R; r0 += (int)blockDim.x) {
        const int r = r0 + tid;
        int64_t n = 0;
        if (r < v.pp.R) {
            const Request q = request_of(v, r);
            if (q.rows) n = Tl::tiles_before(q.c, q.rows, v.pp.group, Tl::row_tiles(q.rows));
        }
        int x = (int)min(n, (int64_t)INT32_MAX / 2);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x = (int)min((int64_t)x + y, (int64_t)INT32_MAX / 2);
        }
        if (lane == 31) sums[warp] = x;
        __syncthreads();
        int64_t before = base, all = 0;
        for (int w = 0; w < warps; ++w) {
            before += w < warp ? sums[w] : 0;
            all += sums[w];
        }
        if (r < v.pp.R) prefix[r] = (int)min(before + x, (int64_t)INT32_MAX);
        base += all;
        __syncthreads();
    }
    return (int)min(base, (int64_t)INT32_MAX);
}

// A worker's position on the line.
struct Cursor {
    int64_t f;  // tile on the line
    int r, g, q, j, n;  // request, cache head, row tile, key tile, the unit's key tiles
    int S;      // the request's key tiles of one cache head
    Request rq;
};

template <typename Tl>
__device__ __forceinline__ void cursor_request(Cursor& k, const FwdView& v, const int* prefix, int r) {
    k.r = r;
    k.S = prefix[r] - (r ? prefix[r - 1] : 0);
    k.rq = Request{v.starts[r], v.cached[r], 0};
    k.rq.rows = (v.starts[r + 1] - k.rq.first) * v.pp.group;
}

// Places the cursor on tile f (f below the line's end).
template <typename Tl>
__device__ __forceinline__ void cursor_seek(Cursor& k, const FwdView& v, const int* prefix, int64_t f) {
    const int want = (int)(f / v.pp.G);
    int lo = 0, hi = v.pp.R - 1;
    while (lo < hi) {  // first request whose sum passes want
        const int mid = (lo + hi) >> 1;
        if (prefix[mid] > want) hi = mid; else lo = mid + 1;
    }
    cursor_request<Tl>(k, v, prefix, lo);
    const int64_t off = f - (int64_t)(lo ? prefix[lo - 1] : 0) * v.pp.G;
    k.g = (int)(off / k.S);
    const int rem = (int)(off - (int64_t)k.g * k.S);
    int a = 0, b = Tl::row_tiles(k.rq.rows) - 1;
    while (a < b) {  // last row tile that begins at or before rem
        const int mid = (a + b + 1) >> 1;
        if (Tl::tiles_before(k.rq.c, k.rq.rows, v.pp.group, mid) <= rem) a = mid; else b = mid - 1;
    }
    k.q = a;
    k.j = rem - (int)Tl::tiles_before(k.rq.c, k.rq.rows, v.pp.group, a);
    k.n = Tl::tiles(k.rq.c, k.rq.rows, v.pp.group, a);
    k.f = f;
}

// From a unit's end to the next unit (end: the worker's end of the line).
template <typename Tl>
__device__ __forceinline__ void cursor_next_unit(Cursor& k, const FwdView& v, const int* prefix, int64_t end) {
    k.j = 0;
    if (k.f >= end) return;
    if (++k.q == Tl::row_tiles(k.rq.rows)) {
        k.q = 0;
        if (++k.g == v.pp.G) {
            k.g = 0;
            int r = k.r + 1;
            while (prefix[r] == prefix[r - 1]) ++r;
            cursor_request<Tl>(k, v, prefix, r);
        }
    }
    k.n = Tl::tiles(k.rq.c, k.rq.rows, v.pp.group, k.q);
}

// Worker w's part of the line: at least min_tiles a worker while there are enough.
__device__ __forceinline__ void worker_range(int64_t total, int workers, int min_tiles, int w, int64_t* lo, int64_t* hi) {
    const int64_t used = max((int64_t)1, min((int64_t)workers, total / min_tiles));
    *lo = w < used ? total * w / used : total;
    *hi = w < used ? total * (w + 1) / used : total;
}

// What a worker leaves of the units that its ends cut: its first piece when that
// continues the worker before (slot 0), its last when it begins a unit that the
// next worker continues (slot 1).  A unit is named by its first tile on the line.
struct PieceMeta {
    int64_t head, tail;  // -1: none
    int first, c, g, q, rows;  // of the tail's unit
    int pad;
};

// Running maximum of a row in units of log2, raised only when a tile exceeds it by
// this much (a factor 256): exact, numerator and denominator share it.
constexpr float kRaise = 8.f;

}  // namespace paged

// The kernels' launches (paged_few.cu: a request's packed rows fit 32; paged_tc.cu:
// more; paged_f32.cu: float32).
constexpr int kPagedFewRows = 32;
size_t paged_few_workspace(const PagedProblem& pp, int num_sms);
cudaError_t launch_paged_few(const PagedProblem& pp, const PagedFwdArgs& a, void* workspace, cudaStream_t s);
size_t paged_tc_workspace(const PagedProblem& pp, int num_sms);
cudaError_t launch_paged_tc(const PagedProblem& pp, const PagedFwdArgs& a, void* workspace, cudaStream_t s);

// The 4-D map (column, token of a page, cache head, page) of a bf16 page pool, box
// 64 columns x box_rows tokens, 128-byte swizzle; columns past d read as zero.
cudaError_t make_page_map(CUtensorMap* map, const void* base, const PagedProblem& pp, int box_rows);

}  // namespace relation
