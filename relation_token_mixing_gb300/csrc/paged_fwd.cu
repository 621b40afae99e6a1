// Relation of new tokens over a paged Relation Cache ("Ask Self, Ask Others",
// Sec. 3.1 eq.(1)-(3), Sec. 5.3 eq.(18), Appendix A.5): for the token at position
// i of its request,
//   U_j = p1 . p2_j / sqrt(d), R_i = sigmoid(U_i / tau_S), R_j = SiLU(U_j)
//   - lambda log(i + 1) for j < i,  Y = sum_{j <= i} softmax(R)_j I~_j.
// One warp per (token, head): lanes over 32 keys for U, over columns for Y.
#include <math.h>

#include <algorithm>

#include "paged_fwd.cuh"

namespace relation {
namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ float sigmoid_exact(float x) {
    const float e = expf(-fabsf(x));
    return x >= 0.f ? 1.f / (1.f + e) : e / (1.f + e);
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
    paged_fwd_rows_kernel(PagedProblem pp, const T* __restrict__ P1, const T* __restrict__ P2, const T* __restrict__ I,
                          const int* __restrict__ table, const int* __restrict__ starts,
                          const int* __restrict__ cached, int max_fresh, int rows_above, T* __restrict__ Y, float* __restrict__ L,
                          unsigned int* status) {
    __shared__ float sq[kThreads / 32][128];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * (kThreads / 32) + warp;
    const int64_t n = w / pp.H;
    const int h = (int)(w - n * pp.H), g = h / pp.group;
    if (n >= pp.N) return;
    // The request: the last one that starts at or before n.
    int lo = 0, hi = pp.R;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (starts[mid + 1] > n) hi = mid; else lo = mid + 1;
    }
    if (lo >= pp.R || starts[lo] > n) return;
    const int first = starts[lo], last = starts[lo + 1], c = cached[lo];
    const int64_t len = (int64_t)c + (last - first);
    if (first < 0 || last > pp.N || c < 0 || len > ((int64_t)pp.width << pp.page_shift) || last - first > max_fresh) {
        if (lane == 0) record_status(status, kDevBadPosition);
        return;
    }
    if ((int64_t)(last - first) * pp.group <= rows_above) return;
    const int i = c + (int)(n - first);
    const T* q = P1 + ((size_t)n * pp.H + h) * pp.d;
    for (int k = lane; k < pp.d; k += 32) sq[warp][k] = load_as_float(q + k) * pp.inv_sqrt_d;
    __syncwarp();
    const float corr = pp.lambda * logf((float)(i + 1));
    float m = -INFINITY, l = 0.f, acc[4] = {};
    for (int j0 = 0; j0 <= i; j0 += 32) {
        const int j = j0 + lane;
        float r = -INFINITY;
        int64_t row = -1;
        if (j <= i) {
            const int page = table[(size_t)lo * pp.width + (j >> pp.page_shift)];
            float u = 0.f;
            if (page >= 0 && page < pp.pages) {
                row = (int64_t)page_row_offset(pp, page, j & pp.page_mask, g);
                for (int k = 0; k < pp.d; ++k) u = fmaf(sq[warp][k], load_as_float(P2 + row + k), u);
            } else {
                record_status(status, kDevBadPosition);
            }
            r = j == i ? sigmoid_exact(u / pp.tau_S) + corr : u * sigmoid_exact(u);
        }
        float mt = r;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
        const float mn = fmaxf(m, mt), scale = expf(m - mn), p = expf(r - mn);
        m = mn;
        float ps = p;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, o);
        l = l * scale + ps;
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] *= scale;
        for (int k = 0; k < 32; ++k) {
            const float pk = __shfl_sync(0xffffffffu, p, k);
            const int64_t rk = __shfl_sync(0xffffffffu, row, k);
            if (rk < 0) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (lane + 32 * e < pp.d) acc[e] = fmaf(pk, load_as_float(I + rk + lane + 32 * e), acc[e]);
        }
    }
    T* y = Y + ((size_t)n * pp.H + h) * pp.d;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (lane + 32 * e < pp.d) store_from_float(y + lane + 32 * e, acc[e] / l);
    if (L != nullptr && lane == 0) L[(size_t)n * pp.H + h] = m + logf(l) - corr;
}

}  // namespace

size_t paged_fwd_workspace(const PagedProblem& pp, bool bf16, int max_fresh, int num_sms) {
    if (!bf16) return 16;
    // The two kernels run one after the other on the caller's stream and share the workspace.
    const size_t few = paged_few_workspace(pp, num_sms);
    return (int64_t)max_fresh * pp.group <= kPagedFewRows ? few : std::max(few, paged_tc_workspace(pp, num_sms));
}

cudaError_t launch_paged_fwd(const PagedProblem& pp, bool bf16, const PagedFwdArgs& a, int* launches, cudaStream_t s) {
    if (bf16) {
        const cudaError_t e = launch_paged_few(pp, a, a.workspace, s);
        *launches = 2;
        if (e != cudaSuccess || (int64_t)a.max_fresh * pp.group <= kPagedFewRows) return e;
        *launches = 4;
        return launch_paged_tc(pp, a, a.workspace, s);
    }
    const unsigned blocks = (unsigned)(((int64_t)pp.N * pp.H + kThreads / 32 - 1) / (kThreads / 32));
    *launches = 1;
    paged_fwd_rows_kernel<float><<<blocks, kThreads, 0, s>>>(
        pp, (const float*)a.P1, (const float*)a.P2_pages, (const float*)a.I_pages, a.table, a.starts, a.cached,
        a.max_fresh, 0, (float*)a.Y, a.L, a.status);
    return cudaGetLastError();
}

}  // namespace relation
