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

// A worker's partial rows: 2 slots of `rows` rows of `width` values, then (m, l) each.
__host__ __device__ constexpr size_t slot_floats(int rows, int width) { return (size_t)rows * (width + 2); }

__device__ __forceinline__ void store_pair(__nv_bfloat16* p, float a, float b) {
    *reinterpret_cast<uint32_t*>(p) = ptx::pack_bf16x2(a, b);
}
__device__ __forceinline__ void store_pair(float* p, float a, float b) {
    *reinterpret_cast<float2*>(p) = make_float2(a, b);
}

// Merges the unit that worker blockIdx.x begins and others continue: with the
// pieces' maxima m_p and sums l_p, weights w_p = 2^(m_p - max m), Y = sum w_p o_p /
// sum w_p l_p, pieces in the line's order.  One warp per row.
template <typename T, int kRows>
__global__ void __launch_bounds__(128)
    paged_merge_rows_kernel(const __grid_constant__ FwdView v, int width, const float* __restrict__ part,
                            const PieceMeta* __restrict__ meta, int workers, T* __restrict__ Y,
                            float* __restrict__ L) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const PagedProblem& pp = v.pp;
    const int w0 = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const PieceMeta mt = meta[w0];
    if (mt.tail < 0) return;
    int pieces = 1;  // worker w0's slot 1, then slots 0 of the workers after it
    for (int base = w0 + 1;; base += 32) {
        const bool more = base + lane < workers && meta[base + lane].head == mt.tail;
        const unsigned b = __ballot_sync(0xffffffffu, more);
        pieces += b == 0xffffffffu ? 32 : __ffs(~b) - 1;
        if (b != 0xffffffffu) break;
    }
    const size_t slot = slot_floats(kRows, width);
    auto piece = [&](int p) { return part + ((size_t)(w0 + p) * 2 + (p == 0 ? 1 : 0)) * slot; };
    const int rows = min(kRows, mt.rows - mt.q * kRows);
    for (int row = warp; row < rows; row += 4) {
        float m = -INFINITY;
        for (int p = lane; p < pieces; p += 32) m = fmaxf(m, piece(p)[kRows * width + 2 * row]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        float l = 0.f;
        float2 acc[2] = {};
        for (int p0 = 0; p0 < pieces; p0 += 32) {
            float wt = 0.f, lp = 0.f;
            if (p0 + lane < pieces) {
                const float2 ml = *reinterpret_cast<const float2*>(piece(p0 + lane) + kRows * width + 2 * row);
                wt = ptx::ex2_approx(ml.x - m);
                lp = wt * ml.y;
            }
            const int n = min(32, pieces - p0);
#pragma unroll 4
            for (int p = 0; p < n; ++p) {
                const float w = __shfl_sync(0xffffffffu, wt, p);
                l += __shfl_sync(0xffffffffu, lp, p);
                const float* src = piece(p0 + p) + row * width + 2 * lane;
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    if (64 * e + 2 * lane < width) {
                        const float2 x = *reinterpret_cast<const float2*>(src + 64 * e);
                        if (w != 0.f) {
                            acc[e].x = fmaf(w, x.x, acc[e].x);
                            acc[e].y = fmaf(w, x.y, acc[e].y);
                        }
                    }
            }
        }
        const int rho = mt.q * kRows + row, t = rho / pp.group, hd = mt.g * pp.group + (rho - t * pp.group);
        const size_t yr = (size_t)(mt.first + t) * pp.H + hd;
        const float inv = 1.f / l;
#pragma unroll
        for (int e = 0; e < 2; ++e)
            if (64 * e + 2 * lane < pp.d)
                store_pair(Y + yr * pp.d + 64 * e + 2 * lane, acc[e].x * inv, acc[e].y * inv);
        if (L != nullptr && lane == 0)
            L[yr] = (m + __log2f(l)) * kLn2 - pp.lambda * __logf((float)(mt.c + t + 1));
    }
}

// Launched as a programmatic dependent of the pass: resident before that ends, it
// waits for its writes in-kernel.
template <typename T, int kRows>
cudaError_t launch_merge_rows(const FwdView& v, int width, const float* part, const PieceMeta* meta, int workers,
                              void* Y, float* L, cudaStream_t s) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)workers);
    cfg.blockDim = dim3(128);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged_merge_rows_kernel<T, kRows>, v, width, part, meta, workers, (T*)Y, L);
}

}  // namespace paged

// The kernels' launches (paged_few.cu: a request's packed rows fit 32; paged_tc.cu:
// more; paged_f32.cu: float32).
constexpr int kPagedFewRows = 32;
size_t paged_few_workspace(const PagedProblem& pp, int num_sms);
cudaError_t launch_paged_few(const PagedProblem& pp, const PagedFwdArgs& a, void* workspace, cudaStream_t s);
size_t paged_tc_workspace(const PagedProblem& pp, int num_sms);
cudaError_t launch_paged_tc(const PagedProblem& pp, const PagedFwdArgs& a, void* workspace, cudaStream_t s);
size_t paged_f32_workspace(const PagedProblem& pp, int max_fresh, int num_sms);
cudaError_t launch_paged_f32(const PagedProblem& pp, const PagedFwdArgs& a, void* workspace, int* launches,
                             cudaStream_t s);

// The 4-D map (column, token of a page, cache head, page) of a bf16 page pool, box
// 64 columns x box_rows tokens, 128-byte swizzle; columns past d read as zero.
cudaError_t make_page_map(CUtensorMap* map, const void* base, const PagedProblem& pp, int box_rows);

}  // namespace relation
