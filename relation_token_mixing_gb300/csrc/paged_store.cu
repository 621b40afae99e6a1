// The input prologue of packed new tokens with the rows of the Relation Cache
// written straight into their pages ("Ask Self, Ask Others", Sec. 3.1 below
// eq.(1) and Appendix B.3: RoPE of the relation coordinates; Sec. 3.2 eq.(4) and
// Appendix A.2.2: Givens mixing of the information states; Sec. 5.3 and Appendix
// A.5.3: the cache update):
//   P1 = RoPE(X1),  P2_pages[slot] = RoPE(X2),  I_pages[slot] = Givens(I).
// One pass: every element is read once and written once, 2 (H + 2 G) d elements
// a token, and the pass is bound by that traffic.  A block takes a few tokens,
// forms their d/2 sines and cosines once in shared memory (H + G heads use them)
// and then moves pairs of vectors, each pair turned by one angle per column: for
// X1 and X2 columns c and c + d/2 of a head, for I the same columns of a head
// pair.
#include <math.h>

#include <algorithm>

#include "paged.h"
#include "vec_io.cuh"

namespace relation {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 8;  // of one block

// HALF: d/2.  VC: columns of one access; HALF is a multiple of it.  BATCH: pairs of vectors that a
// thread has in flight.
template <typename T, int HALF, int VC, int BATCH>
__global__ void __launch_bounds__(kThreads)
    paged_store_kernel(PagedProblem pp, const T* __restrict__ X1, const T* __restrict__ X2, const T* __restrict__ I,
                       const float* __restrict__ theta, int pairing, const __grid_constant__ RopeTable tab,
                       const int* __restrict__ positions, const int64_t* __restrict__ slots, T* __restrict__ P1,
                       T* __restrict__ P2_pages, T* __restrict__ I_pages, unsigned int* status, int tokens, FastDiv by_heads) {
    constexpr int D = 2 * HALF, PER = HALF / VC;
    extern __shared__ float2 sh[];  // (cos, sin) [tokens][HALF], then [G/2] of the head pairs
    __shared__ int64_t s_slot[kMaxTokens];
    __shared__ float2 same;  // no mixing
    float2* turn = sh;
    float2* mix = sh + kMaxTokens * HALF;
    const int n0 = blockIdx.x * tokens, count = min(tokens, pp.N - n0);
    if (threadIdx.x < count) {
        int64_t slot = slots[n0 + threadIdx.x];
        if (slot >= ((int64_t)pp.pages << pp.page_shift)) {
            record_status(status, kDevBadPosition);
            slot = -1;
        }
        s_slot[threadIdx.x] = slot;
    }
    for (int k = threadIdx.x; k < count * HALF; k += kThreads) {
        const int t = k / HALF, c = k - t * HALF;
        float sn = 0.f, cs = 1.f;
        if (tab.enabled) rope_sincos((float)positions[n0 + t], tab.hi[c], tab.lo[c], &sn, &cs);
        turn[k] = make_float2(cs, sn);
    }
    if (threadIdx.x == 0) same = make_float2(1.f, 0.f);
    if (theta != nullptr)
        for (int k = threadIdx.x; k < pp.G / 2; k += kThreads) {
            float sn, cs;
            sincosf(theta[k], &sn, &cs);
            mix[k] = make_float2(cs, sn);
        }
    __syncthreads();
    // Items of one token: H heads of X1, G of X2, G of I (pairs of heads, each half
    // the columns: the same number of items), PER vector pairs each.
    const int heads = pp.H + 2 * pp.G, items = count * heads * PER;
    for (int k0 = threadIdx.x; k0 < items; k0 += kThreads * BATCH) {
        Vec<T, VC> va[BATCH], vb[BATCH];
        T *a_dst[BATCH], *b_dst[BATCH];
        const float2* cs[BATCH];
        bool each[BATCH];  // an angle per column (RoPE) or one for all (Givens)
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const int k = k0 + i * kThreads;
            a_dst[i] = nullptr;
            if (k >= items) continue;
            const int v = k % PER, u = k / PER;
            const int t = (int)by_heads.div((uint32_t)u), hd = u - t * heads, c = v * VC;
            const int64_t n = n0 + t, slot = s_slot[t];
            const int64_t page = slot >> pp.page_shift;
            const int off = (int)(slot & pp.page_mask);
            const T *a_src, *b_src;
            cs[i] = turn + t * HALF + c;
            each[i] = true;
            if (hd < pp.H) {
                a_src = X1 + ((size_t)n * pp.H + hd) * D + c;
                b_src = a_src + HALF;
                a_dst[i] = P1 + ((size_t)n * pp.H + hd) * D + c;
                b_dst[i] = a_dst[i] + HALF;
            } else if (slot < 0) {
                continue;
            } else if (hd < pp.H + pp.G) {
                const int g = hd - pp.H;
                a_src = X2 + ((size_t)n * pp.G + g) * D + c;
                b_src = a_src + HALF;
                a_dst[i] = P2_pages + page_row_offset(pp, page, off, g) + c;
                b_dst[i] = a_dst[i] + HALF;
            } else {
                const int g = hd - pp.H - pp.G;
                int ga = g, gb = g, ca = c, cb = c + HALF;
                each[i] = false;
                cs[i] = &same;
                if (theta != nullptr) {  // item g: pair g/2, the first or second half of its columns
                    const int pair = g >> 1;
                    cs[i] = mix + pair;
                    ga = 2 * pair + pairing;
                    gb = ga + 1 == pp.G ? 0 : ga + 1;
                    ca = cb = c + (g & 1) * HALF;
                }
                a_src = I + ((size_t)n * pp.G + ga) * D + ca;
                b_src = I + ((size_t)n * pp.G + gb) * D + cb;
                a_dst[i] = I_pages + page_row_offset(pp, page, off, ga) + ca;
                b_dst[i] = I_pages + page_row_offset(pp, page, off, gb) + cb;
            }
            va[i].load(a_src);
            vb[i].load(b_src);
        }
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            if (a_dst[i] == nullptr) continue;
            float a[VC], b[VC], ra[VC], rb[VC];
            va[i].unpack(a);
            vb[i].unpack(b);
#pragma unroll
            for (int e = 0; e < VC; ++e) {
                const float2 w = cs[i][each[i] ? e : 0];
                ra[e] = w.x * a[e] - w.y * b[e];
                rb[e] = w.y * a[e] + w.x * b[e];
            }
            va[i].pack(ra);
            vb[i].pack(rb);
            va[i].store(a_dst[i]);
            vb[i].store(b_dst[i]);
        }
    }
}

template <typename T, int HALF, int VC>
cudaError_t launch_store(const PagedProblem& pp, const void* X1, const void* X2, const void* I, const float* theta,
                         int pairing, const RopeTable& tab, const int* positions, const int64_t* slots, void* P1,
                         void* P2_pages, void* I_pages, unsigned int* status, int num_sms, cudaStream_t s) {
    constexpr int kBatch = VC * sizeof(T) >= 16 ? 2 : 4;
    // A few blocks per SM first, then more tokens to a block.
    const int tokens = (int)std::min<int64_t>(kMaxTokens, std::max<int64_t>(1, (int64_t)pp.N / (4 * num_sms)));
    const unsigned blocks = (unsigned)(((int64_t)pp.N + tokens - 1) / tokens);
    const size_t sh = (size_t)(kMaxTokens * HALF + pp.G / 2) * sizeof(float2);
    paged_store_kernel<T, HALF, VC, kBatch><<<blocks, kThreads, sh, s>>>(
        pp, (const T*)X1, (const T*)X2, (const T*)I, theta, pairing, tab, positions, slots, (T*)P1, (T*)P2_pages,
        (T*)I_pages, status, tokens, FastDiv((uint32_t)(pp.H + 2 * pp.G)));
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_store(const PagedProblem& pp, bool bf16, const void* X1, const void* X2, const void* I,
                               const float* theta, int pairing, const RopeTable& tab, const int* positions,
                               const int64_t* slots, void* P1, void* P2_pages, void* I_pages, unsigned int* status,
                               int num_sms, cudaStream_t s) {
#define STORE(T, HALF, VC) \
    return launch_store<T, HALF, VC>(pp, X1, X2, I, theta, pairing, tab, positions, slots, P1, P2_pages, I_pages, \
                                     status, num_sms, s)
    // The widest access that d/2 columns and the rows' alignment allow.
    if (bf16) {
        switch (pp.d) {
            case 48: STORE(__nv_bfloat16, 24, 8);
            case 60: STORE(__nv_bfloat16, 30, 2);
            case 64: STORE(__nv_bfloat16, 32, 8);
            case 80: STORE(__nv_bfloat16, 40, 8);
            case 128: STORE(__nv_bfloat16, 64, 8);
        }
    } else {
        switch (pp.d) {
            case 48: STORE(float, 24, 4);
            case 60: STORE(float, 30, 2);
            case 64: STORE(float, 32, 4);
            case 80: STORE(float, 40, 4);
            case 128: STORE(float, 64, 4);
        }
    }
#undef STORE
    return cudaErrorInvalidValue;
}

}  // namespace relation
