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
    Request q{__ldg(v.starts + r), __ldg(v.cached + r), 0};
    const int last = __ldg(v.starts + r + 1);
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

// prefix[r] = sum over requests 0..r of places_of(request), the line's places of one
// cache head.  All threads of the block; sums: one per warp.  Returns the line's
// length over all cache heads, or 0 (and a report) if it passes 2^31 - 1 places.
template <typename PlacesOf>
__device__ __forceinline__ int schedule_build(const FwdView& v, int* prefix, int64_t* sums, PlacesOf places_of) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = (int)blockDim.x >> 5;
    int64_t base = 0;
    for (int r0 = 0; r0 < v.pp.R; r0 += (int)blockDim.x) {
        const int r = r0 + tid;
        int64_t x = 0;
        if (r < v.pp.R) {
            const Request q = request_of(v, r);
            if (q.rows) x = places_of(q);
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
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
    const int64_t total = base * v.pp.G;
    if (total > (int64_t)INT32_MAX) {
        record_status(v.status, kDevBadPosition);
        return 0;
    }
    return (int)total;
}

// The request that has place f of the line: the first whose sum passes f / G.
__device__ __forceinline__ int schedule_find(const FwdView& v, const int* prefix, int f) {
    const int want = v.pp.by_G.div(f);
    int lo = 0, hi = v.pp.R - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (prefix[mid] > want) hi = mid; else lo = mid + 1;
    }
    return lo;
}

// A worker's position on a line of units with many row tiles.
struct Cursor {
    int f;              // the key tile's place on the line
    int r, g, q, j, n;  // request, cache head, row tile, key tile, the unit's key tiles
    Request rq;
};

__device__ __forceinline__ void cursor_request(Cursor& k, const FwdView& v, int r) {
    k.r = r;
    k.rq.first = __ldg(v.starts + r);
    k.rq.c = __ldg(v.cached + r);
    k.rq.rows = (__ldg(v.starts + r + 1) - k.rq.first) * v.pp.group;
}

// Puts the cursor on the first key tile of its unit at or after place f (f below the
// line's end); that may be past a worker's end.
template <typename Tl>
__device__ __forceinline__ void cursor_seek(Cursor& k, const FwdView& v, const int* prefix, int f) {
    const int r = schedule_find(v, prefix, f), before = r ? prefix[r - 1] : 0, S = prefix[r] - before;
    cursor_request(k, v, r);
    const int off = f - before * v.pp.G;
    k.g = off / S;
    const int rem = off - k.g * S;
    int a = 0, b = Tl::row_tiles(k.rq.rows) - 1;
    while (a < b) {  // last row tile that begins at or before rem
        const int mid = (a + b + 1) >> 1;
        if (Tl::places(k.rq.c, k.rq.rows, v.pp.by_group, mid) <= rem) a = mid; else b = mid - 1;
    }
    k.q = a;
    const int in = rem - (int)Tl::places(k.rq.c, k.rq.rows, v.pp.by_group, a);
    k.j = max(0, in - Tl::extra);
    k.n = Tl::tiles(k.rq.c, k.rq.rows, v.pp.by_group, a);
    k.f = f + Tl::extra + k.j - in;
}

// From a unit's end to the next unit (end: the worker's end of the line).
template <typename Tl>
__device__ __forceinline__ void cursor_next_unit(Cursor& k, const FwdView& v, const int* prefix, int end) {
    k.j = 0;
    if (k.f >= end || (k.f += Tl::extra) >= end) return;
    if (++k.q == Tl::row_tiles(k.rq.rows)) {
        k.q = 0;
        if (++k.g == v.pp.G) {
            k.g = 0;
            int r = k.r + 1;
            while (prefix[r] == prefix[r - 1]) ++r;
            cursor_request(k, v, r);
        }
    }
    k.n = Tl::tiles(k.rq.c, k.rq.rows, v.pp.by_group, k.q);
}

// A block's partial rows in the workspace: slot 0 of its unit that continues the
// block before, slot 1 of the one that the next block continues.  Of the latter the
// block also leaves what the merge needs:
struct PieceMeta {
    int pieces;  // this block's and the following blocks' (0: no such unit)
    int first, c, rows;  // the unit's request
    int g, q;            // and its cache head and row tile
};

// Running maximum of a row in units of log2, raised only when a tile exceeds it by
// this much (a factor 256): exact, numerator and denominator share it.
constexpr float kRaise = 8.f;

// The maximum that a piece leaves of a row: -inf says that it begins past the row's own token
// and has none of its keys.  A piece that has some leaves a finite one or +inf even where all its
// scores are NaN (which no maximum takes in), so that the merge does not pass over its sum.
__device__ __forceinline__ float piece_max(bool has_keys, float m) {
    return has_keys ? fmaxf(m, -3.402823466e38f) : -INFINITY;
}

// A slot: `rows` rows of `width` values, then (m, l) each.
__host__ __device__ constexpr size_t slot_floats(int rows, int width) { return (size_t)rows * (width + 2); }

__device__ __forceinline__ void store_pair(__nv_bfloat16* p, float a, float b) {
    *reinterpret_cast<uint32_t*>(p) = ptx::pack_bf16x2(a, b);
}
__device__ __forceinline__ void store_pair(float* p, float a, float b) {
    *reinterpret_cast<float2*>(p) = make_float2(a, b);
}

// The kernels of a forward are launched as programmatic dependents, each on the SMs
// as soon as there is room.  The first one waits for what ran before it and only then
// releases the next, so whatever starts after that finds its inputs complete; the long
// requests' pass, which reads nothing of the one before, waits at its end only; and the
// merge waits for it, so the last kernel's end is that of all.
__device__ __forceinline__ void dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void dependency_release() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// A row's merged state: weights 2^(m_p - m) of the pieces so far, m their maximum.
template <int kQuads>
struct MergedRow {
    float m = -INFINITY, l = 0.f;
    float4 acc[kQuads] = {};
    __device__ __forceinline__ void add(float pm, float pl, const float4 (&x)[kQuads]) {
        if (pm == -INFINITY) return;  // none of the row's keys: the piece's values may not be there
        const float top = fmaxf(m, pm), f = ptx::ex2_approx(m - top), w = ptx::ex2_approx(pm - top);
        m = top;
        l = fmaf(w, pl, l * f);
#pragma unroll
        for (int e = 0; e < kQuads; ++e) {
            acc[e].x = fmaf(w, x[e].x, acc[e].x * f);
            acc[e].y = fmaf(w, x[e].y, acc[e].y * f);
            acc[e].z = fmaf(w, x[e].z, acc[e].z * f);
            acc[e].w = fmaf(w, x[e].w, acc[e].w * f);
        }
    }
    // Thread `sub` of the row's eight has columns 32 e + 4 sub and the next three.
    template <typename T>
    __device__ __forceinline__ void finish(const PagedProblem& pp, int first, int c, int g, int rho, int sub, T* Y,
                                           float* L) const {
        const int t = pp.by_group.div(rho), hd = g * pp.group + (rho - t * pp.group);
        const size_t yr = (size_t)(first + t) * pp.H + hd;
        const float inv = 1.f / l;
#pragma unroll
        for (int e = 0; e < kQuads; ++e) {
            const int col = 32 * e + 4 * sub;
            if (col >= pp.d) continue;
            store_pair(Y + yr * pp.d + col, acc[e].x * inv, acc[e].y * inv);
            store_pair(Y + yr * pp.d + col + 2, acc[e].z * inv, acc[e].w * inv);
        }
        if (L != nullptr && sub == 0) L[yr] = (m + __log2f(l)) * kLn2 - pp.lambda * __logf((float)(c + t + 1));
    }
};

// What a pass leaves to merge: its blocks' two partial slots each, and the unit that each
// begins and others continue.
struct MergeSide {
    const float* part;
    const PieceMeta* meta;
    int blocks;
};

// Merges 16 rows, from row0 on, of the unit that block x of the pass begins, pieces in the
// line's order, eight threads a row.  The time is that of the dependent loads: the unit, then
// four pieces' rows at once (a unit seldom has more).
constexpr int kMergeThreads = 128, kMergeRows = 16;

template <typename T, int kRows, int kWidth>
__device__ __forceinline__ void merge_rows(const PagedProblem& pp, const MergeSide& side, int x, int row0, T* Y,
                                           float* L) {
    constexpr int kQuads = kWidth / 32, kBatch = 4;
    constexpr size_t slot = slot_floats(kRows, kWidth);
    const int sub = threadIdx.x & 7, row = row0 + (threadIdx.x >> 3);
    if (x >= side.blocks) return;
    const PieceMeta mt = side.meta[x];
    const int rho = mt.q * kRows + row;
    if (mt.pieces == 0 || row >= kRows || rho >= mt.rows) return;
    // Piece 0 is this block's slot 1, piece p block (x + p)'s slot 0.
    const float* base = side.part + (size_t)x * 2 * slot;
    MergedRow<kQuads> out;
    for (int p0 = 0; p0 < mt.pieces; p0 += kBatch) {
        float2 ml[kBatch];
        float4 v[kBatch][kQuads];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int p = min(p0 + b, mt.pieces - 1);
            const float* src = base + (p ? (size_t)p * 2 : (size_t)1) * slot;
            ml[b] = *reinterpret_cast<const float2*>(src + kRows * kWidth + 2 * row);
            if (p0 + b >= mt.pieces) ml[b].x = -INFINITY;
#pragma unroll
            for (int e = 0; e < kQuads; ++e)
                v[b][e] = *reinterpret_cast<const float4*>(src + (size_t)row * kWidth + 32 * e + 4 * sub);
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) out.add(ml[b].x, ml[b].y, v[b]);
    }
    out.finish(pp, mt.first, mt.c, mt.g, rho, sub, Y, L);
}

// Merges the few rows' units alone (kFew rows each), or (kLong > 0) those of both passes.
template <typename T, int kFew, int kLong, int kWidth>
__global__ void __launch_bounds__(kMergeThreads)
    paged_merge_kernel(const __grid_constant__ FwdView v, const MergeSide few, const MergeSide longer,
                       T* __restrict__ Y, float* __restrict__ L) {
    static_assert(kFew <= kMergeRows, "one block a unit");
    dependency_release();
    dependency_wait();
    if constexpr (kLong > 0) {
        if (blockIdx.y > 0) {
            merge_rows<T, kLong, kWidth>(v.pp, longer, blockIdx.x, (blockIdx.y - 1) * kMergeRows, Y, L);
            return;
        }
    }
    merge_rows<T, kFew, kWidth>(v.pp, few, blockIdx.x, 0, Y, L);
}

// One kernel of the chain on stream s, resident before the kernel before it ends.
template <typename... P, typename... A>
cudaError_t launch_chained(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, P(args)...);
}

template <typename T, int kFew, int kLong, int kWidth>
cudaError_t launch_merge(const FwdView& v, const MergeSide& few, const MergeSide& longer, void* Y, float* L,
                         cudaStream_t s) {
    return launch_chained(paged_merge_kernel<T, kFew, kLong, kWidth>,
                          dim3((unsigned)(few.blocks > longer.blocks ? few.blocks : longer.blocks),
                               1 + kLong / kMergeRows),
                          kMergeThreads, 0, s, v, few, longer, (T*)Y, L);
}

}  // namespace paged

// The kernels' launches (paged_few.cu: a request's packed rows fit 16; paged_tc.cu:
// more; paged_f32.cu: float32).
constexpr int kPagedFewRows = 16;
size_t paged_few_workspace(const PagedProblem& pp, int max_fresh, int num_sms);
// left: what it leaves to the long requests' pass to merge, if that follows.
cudaError_t launch_paged_few(const PagedProblem& pp, const PagedFwdArgs& a, void* workspace, paged::MergeSide* left,
                             cudaStream_t s);
size_t paged_tc_workspace(const PagedProblem& pp, int num_sms);
cudaError_t launch_paged_tc(const PagedProblem& pp, const PagedFwdArgs& a, void* workspace,
                            const paged::MergeSide& few, cudaStream_t s);
size_t paged_f32_workspace(const PagedProblem& pp, int max_fresh, int num_sms);
cudaError_t launch_paged_f32(const PagedProblem& pp, const PagedFwdArgs& a, void* workspace, int* launches,
                             cudaStream_t s);

// The 4-D map (column, token of a page, cache head, page) of a bf16 page pool, box
// 64 columns x box_rows tokens, 128-byte swizzle; columns past d read as zero.
cudaError_t make_page_map(CUtensorMap* map, const void* base, const PagedProblem& pp, int box_rows);

}  // namespace relation
