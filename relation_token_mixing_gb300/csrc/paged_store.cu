// The input prologue of packed new tokens with the rows of the Relation Cache
// written straight into their pages ("Ask Self, Ask Others", Sec. 3.1 below
// eq.(1) and Appendix B.3: RoPE of the relation coordinates; Sec. 3.2 eq.(4) and
// Appendix A.2.2: Givens mixing of the information states; Sec. 5.3 and Appendix
// A.5.3: the cache update):
//   P1 = RoPE(X1),  P2_pages[slot] = RoPE(X2),  I_pages[slot] = Givens(I).
// One pass: every element is read once and written once, 2 (H + 2 G) d elements
// a token, and the pass is bound by that traffic.  A block takes up to four tokens
// and forms their d/2 sines and cosines once in shared memory (H + G heads use
// them).  A thread keeps one pair of vectors of the token, turned by one angle per
// column (X1, X2: columns c and c + d/2 of a head) or by one for all (I: the same
// columns of a head pair), through all the block's tokens, two to four in flight: what is
// where is worked out once a thread and not once a vector.  That matters where the
// vectors are short: rows of 60 halves are 4-byte pairs (d/2 = 30).
// Measured: 16384 tokens, 32 heads over 8 of 128: 73 us, 403 MB, 5.5 TB/s (8 tokens a block
// 76, 2 tokens 72; two rounds of vectors worked out singly 72); 4999 tokens, 8 heads over
// 8 of 60: 9.9 us (singly 14.4); 64 tokens, 16 heads of 64: 3.0 us.
#include <math.h>

#include <algorithm>

#include "paged.h"
#include "paged_rope.cuh"
#include "vec_io.cuh"

namespace relation {
namespace {

constexpr int kMaxThreads = 256;
constexpr int kMaxTokens = 4;  // of one block

// HALF: d/2.  VC: columns of one access; HALF is a multiple of it.  BATCH: tokens whose
// vectors a thread has in flight.
template <typename T, int HALF, int VC, int BATCH>
__global__ void __launch_bounds__(kMaxThreads)
    paged_store_kernel(PagedProblem pp, const T* __restrict__ X1, const T* __restrict__ X2, const T* __restrict__ I,
                       const float* __restrict__ theta, int pairing, const __grid_constant__ RopeTable tab,
                       const int* __restrict__ positions, const int64_t* __restrict__ slots, T* __restrict__ P1,
                       T* __restrict__ P2_pages, T* __restrict__ I_pages, unsigned int* status, int tokens) {
    constexpr int D = 2 * HALF, PER = HALF / VC;
    extern __shared__ float2 sh[];  // (cos, sin) [tokens][HALF], then [G/2] of the head pairs
    __shared__ int64_t s_row[kMaxTokens];  // where the token's row of cache head 0 begins, or -1
    __shared__ float2 same;                // no mixing
    float2* turn = sh;
    float2* mix = sh + kMaxTokens * HALF;
    const int threads = (int)blockDim.x, n0 = blockIdx.x * tokens, count = min(tokens, pp.N - n0);
    if ((int)threadIdx.x < count) {
        const int64_t slot = slots[n0 + threadIdx.x];
        const bool in = slot >= 0 && slot < ((int64_t)pp.pages << pp.page_shift);
        if (slot >= 0 && !in) record_status(status, kDevBadPosition);
        s_row[threadIdx.x] =
            in ? (int64_t)page_row_offset(pp, slot >> pp.page_shift, (int)(slot & pp.page_mask), 0) : -1;
    }
    for (int k = threadIdx.x; k < count * HALF; k += threads) {
        const int t = k / HALF, c = k - t * HALF;
        float sn = 0.f, cs = 1.f;
        if (tab.enabled) position_sincos(positions[n0 + t], tab.hi[c], tab.lo[c], &sn, &cs);
        turn[k] = make_float2(cs, sn);
    }
    if (threadIdx.x == 0) same = make_float2(1.f, 0.f);
    if (theta != nullptr)
        for (int k = threadIdx.x; k < pp.G / 2; k += threads) {
            float sn, cs;
            sincosf(theta[k], &sn, &cs);
            mix[k] = make_float2(cs, sn);
        }
    __syncthreads();
    const size_t head = page_row_offset(pp, 0, 0, 1);  // from one cache head's row to the next
    // Items: H heads of X1, G of X2, G of I (pairs of heads, each half the columns: the same
    // number of items), PER vector pairs each.  A thread keeps an item through all tokens.
    const int items = (pp.H + 2 * pp.G) * PER;
    for (int k = threadIdx.x; k < items; k += threads) {
        const int hd = k / PER, c = (k - hd * PER) * VC;
        const T *a_src, *b_src;
        T *a_dst, *b_dst;
        size_t step = (size_t)pp.G * D;            // of the source, from token to token
        const float2* angle = turn + c;
        bool each = true, paged = true;  // an angle per column (RoPE) or one for all (Givens); into pages or P1
        if (hd < pp.H) {
            step = (size_t)pp.H * D;
            const size_t at = ((size_t)n0 * pp.H + hd) * D + c;
            a_src = X1 + at;
            b_src = a_src + HALF;
            a_dst = P1 + at;
            b_dst = a_dst + HALF;
            paged = false;
        } else if (hd < pp.H + pp.G) {
            const int g = hd - pp.H;
            a_src = X2 + ((size_t)n0 * pp.G + g) * D + c;
            b_src = a_src + HALF;
            a_dst = P2_pages + g * head + c;
            b_dst = a_dst + HALF;
        } else {
            const int g = hd - pp.H - pp.G;
            int ga = g, gb = g, ca = c, cb = c + HALF;
            each = false;
            angle = &same;
            if (theta != nullptr) {  // item g: pair g/2, the first or second half of its columns
                const int pair = g >> 1;
                angle = mix + pair;
                ga = 2 * pair + pairing;
                gb = ga + 1 == pp.G ? 0 : ga + 1;
                ca = cb = c + (g & 1) * HALF;
            }
            a_src = I + ((size_t)n0 * pp.G + ga) * D + ca;
            b_src = I + ((size_t)n0 * pp.G + gb) * D + cb;
            a_dst = I_pages + ga * head + ca;
            b_dst = I_pages + gb * head + cb;
        }
        for (int t0 = 0; t0 < count; t0 += BATCH) {
            Vec<T, VC> va[BATCH], vb[BATCH];
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                if (t0 + i >= count) break;
                va[i].load(a_src + (t0 + i) * step);
                vb[i].load(b_src + (t0 + i) * step);
            }
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                const int t = t0 + i;
                if (t >= count) break;
                const int64_t at = paged ? s_row[t] : (int64_t)(t * step);
                if (at < 0) continue;
                const float2* cs = each ? angle + t * HALF : angle;
                float a[VC], b[VC], ra[VC], rb[VC];
                va[i].unpack(a);
                vb[i].unpack(b);
#pragma unroll
                for (int e = 0; e < VC; ++e) {
                    const float2 w = cs[each ? e : 0];
                    ra[e] = w.x * a[e] - w.y * b[e];
                    rb[e] = w.y * a[e] + w.x * b[e];
                }
                va[i].pack(ra);
                vb[i].pack(rb);
                va[i].store(a_dst + at);
                vb[i].store(b_dst + at);
            }
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
    // As many threads as share the items evenly.
    const int items = (pp.H + 2 * pp.G) * (HALF / VC), rounds = (items + kMaxThreads - 1) / kMaxThreads;
    const int threads = std::min(kMaxThreads, ((items + rounds - 1) / rounds + 31) / 32 * 32);
    const size_t sh = (size_t)(kMaxTokens * HALF + pp.G / 2) * sizeof(float2);
    paged_store_kernel<T, HALF, VC, kBatch><<<blocks, threads, sh, s>>>(
        pp, (const T*)X1, (const T*)X2, (const T*)I, theta, pairing, tab, positions, slots, (T*)P1, (T*)P2_pages,
        (T*)I_pages, status, tokens);
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
