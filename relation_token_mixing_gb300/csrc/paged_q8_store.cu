// The paged Relation Cache in 8 bits: the input prologue of packed new tokens with
// the rows that the cache keeps quantised as they are written, and the rows of some
// slots read back ("Ask Self, Ask Others: Relation Is All You Need", Sec. 3.1 and
// Appendix B.3: RoPE; Sec. 3.2 eq.(4) and Appendix A.2.2: Givens mixing; Sec. 5.3 and
// Appendix A.5.3: the cache).
//
// A row x of d float32 values is kept as q_c = round(x_c / s), |q_c| <= 127, and one scale
// s = 2^k, the least power of two (2^-126 at least) with max |x_c| <= 127 s.  Whole numbers of
// 8 bits times a power of two are bf16 values, so the cache holds exactly what a reader forms:
// nothing is rounded a second time.  The error is half of s, at most max |x| / 127; a
// scale that is no power of two would halve that at best and cost a rounding on every read.
// e4m3 in place of whole numbers keeps 2^-4 of each value, three to four times as much
// in the norm of a Gaussian row.  A row with an infinity or a NaN gets a NaN scale and reads as NaN.
//
// One pass, as paged_store.cu: every element is read once and written once.  4, 8 or 16 lanes have a
// row (columns c and c + d/2 together, as RoPE turns them) and find its largest value among
// themselves, so a row never leaves its registers between the prologue and its pages.  Both kernels
// move bytes.  Measured, 16384 tokens, 32 heads over 8 of 128: the store 70 us (370 MB, 5.3 TB/s), the rows
// read back right after it 15 us (101 MB, 6.6 TB/s, the pages still in L2; from memory 18); 4999 tokens, 8 heads of 60: 14 and
// 4.2 us (6.3).
#include <math.h>

#include <algorithm>

#include "paged.h"
#include "paged_rope.cuh"
#include "vec_io.cuh"

namespace relation {
namespace {

constexpr int kThreads = 256;
// Tokens of one block (16384 tokens, 32 heads over 8 of 128: 2: 70.9 us, 4: 70.0, 8: 66.6; 4999 tokens, 8 heads of 60:
// 13.4, 14.3, 16.1).
constexpr int kMaxTokens = 4;

// The scale's bits as a float: of the bits of max |x|, m 2^e, it takes the exponent e - 6, or e - 5
// where m is above 127 / 64.
__device__ __forceinline__ uint32_t scale_exponent(uint32_t top) {
    return (uint32_t)max(1, (int)((top + 0x1FFFFu) >> 23) - 6);
}

// Rounded to the nearest whole number, in the low byte (1.5 2^23 leaves no room for fractions).
__device__ __forceinline__ uint32_t rounded(float x, float inv) { return __float_as_uint(fmaf(x, inv, 12582912.f)); }

template <int VC>
__device__ __forceinline__ void store_q8(int8_t* p, const float (&x)[VC], float inv) {
    if constexpr (VC == 2) {
        *reinterpret_cast<uint16_t*>(p) = (uint16_t)__byte_perm(rounded(x[0], inv), rounded(x[1], inv), 0x0040);
    } else {
        static_assert(VC == 8, "8 columns or 2");
        uint32_t w[2];
#pragma unroll
        for (int k = 0; k < 2; ++k)
            w[k] = __byte_perm(__byte_perm(rounded(x[4 * k], inv), rounded(x[4 * k + 1], inv), 0x0040),
                               __byte_perm(rounded(x[4 * k + 2], inv), rounded(x[4 * k + 3], inv), 0x0040), 0x5410);
        *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    }
}

// HALF: d/2.  VC: columns of one access.  LANES: lanes of a row, HALF / VC of them at work.
template <int HALF, int VC, int LANES>
__global__ void __launch_bounds__(kThreads)
    paged_store_q8_kernel(PagedProblem pp, const __nv_bfloat16* __restrict__ X1, const __nv_bfloat16* __restrict__ X2,
                          const __nv_bfloat16* __restrict__ I, const float* __restrict__ theta, int pairing,
                          const __grid_constant__ RopeTable tab, const int* __restrict__ positions,
                          const int64_t* __restrict__ slots, __nv_bfloat16* __restrict__ P1, int8_t* __restrict__ P2_pages,
                          int8_t* __restrict__ I_pages, __nv_bfloat16* __restrict__ scales, unsigned int* status,
                          int tokens, FastDiv by_rows) {
    constexpr int D = 2 * HALF, PER = HALF / VC;
    extern __shared__ float2 sh[];  // (cos, sin) [tokens][VC][PER]: a row's lanes side by side, then [G/2] of the head pairs
    __shared__ int64_t s_row[kMaxTokens];  // the token's row of cache head 0, counted in rows, or -1
    float2* turn = sh;
    float2* mix = sh + kMaxTokens * HALF;
    const int n0 = blockIdx.x * tokens, count = min(tokens, pp.N - n0);
    if ((int)threadIdx.x < count) {
        const int64_t slot = slots[n0 + threadIdx.x];
        const bool in = slot >= 0 && slot < ((int64_t)pp.pages << pp.page_shift);
        if (slot >= 0 && !in) record_status(status, kDevBadPosition);
        s_row[threadIdx.x] =
            in ? (int64_t)page_row_index(pp, slot >> pp.page_shift, (int)(slot & pp.page_mask), 0) : -1;
    }
    for (int k = threadIdx.x; k < count * HALF; k += kThreads) {
        const int t = k / HALF, c = k - t * HALF;
        float sn = 0.f, cs = 1.f;
        if (tab.enabled) position_sincos_fine(positions[n0 + t], tab.hi[c], tab.lo[c], &sn, &cs);
        turn[t * HALF + c % VC * PER + c / VC] = make_float2(cs, sn);
    }
    if (theta != nullptr)
        for (int k = threadIdx.x; k < pp.G / 2; k += kThreads) {
            float sn, cs;
            sincosf(theta[k], &sn, &cs);
            mix[k] = make_float2(cs, sn);
        }
    __syncthreads();
    const int64_t head = (int64_t)page_row_index(pp, 0, 0, 1);  // rows from one cache head to the next
    const int lane = threadIdx.x % LANES, c = lane * VC;
    // The block's rows of all its tokens, one after another: H of X1, G of X2, G of I.
    const int rows = pp.H + 2 * pp.G, total = rows * count;
    for (int k0 = threadIdx.x / 32 * (32 / LANES); k0 < total; k0 += kThreads / LANES) {
        const int k = k0 + (int)(threadIdx.x % 32) / LANES, t = by_rows.div(k), j = k - t * rows, n = n0 + t;
        const bool in = k < total && lane < PER, key = j < pp.H + pp.G;
        const int g = key ? j - pp.H : j - pp.H - pp.G;  // (of a row of X2 or I)
        float a[VC], b[VC];  // columns c and c + d/2
        uint32_t top = 0;
        if (in) {
            Vec<__nv_bfloat16, VC> va, vb;
            const __nv_bfloat16* src = (j < pp.H ? X1 + ((size_t)n * pp.H + j) * D : (key ? X2 : I) + ((size_t)n * pp.G + g) * D) + c;
            va.load(src);
            vb.load(src + HALF);
            if (key) {
                float x[VC], y[VC];
                va.unpack(x);
                vb.unpack(y);
#pragma unroll
                for (int e = 0; e < VC; ++e) {
                    const float2 w = turn[t * HALF + e * PER + lane];
                    a[e] = w.x * x[e] - w.y * y[e];
                    b[e] = w.y * x[e] + w.x * y[e];
                }
            } else {
                va.unpack(a);
                vb.unpack(b);
                if (theta != nullptr) {  // the first of a pair: cos a - sin b, the second: sin a + cos b
                    int pair;
                    bool first;
                    const int other = givens_partner(g, pp.G, pairing, &pair, &first);
                    const float2 w = mix[pair];
                    const float sn = first ? -w.y : w.y;
                    const __nv_bfloat16* mate = I + ((size_t)n * pp.G + other) * D + c;
                    va.load(mate);
                    vb.load(mate + HALF);
                    float x[VC], y[VC];
                    va.unpack(x);
                    vb.unpack(y);
#pragma unroll
                    for (int e = 0; e < VC; ++e) {
                        a[e] = w.x * a[e] + sn * x[e];
                        b[e] = w.x * b[e] + sn * y[e];
                    }
                }
            }
            if (j < pp.H) {
                va.pack(a);
                vb.pack(b);
                __nv_bfloat16* dst = P1 + ((size_t)n * pp.H + j) * D + c;
                va.store(dst);
                vb.store(dst + HALF);
            } else {
#pragma unroll
                for (int e = 0; e < VC; ++e)  // as whole numbers, so that a NaN is above all
                    top = max(top, max(__float_as_uint(a[e]) & 0x7fffffffu, __float_as_uint(b[e]) & 0x7fffffffu));
            }
        }
#pragma unroll
        for (int o = 1; o < LANES; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (!in || j < pp.H || s_row[t] < 0) continue;
        const bool finite = top < 0x7f800000u;
        const uint32_t ex = scale_exponent(top);
        const float inv = finite ? __uint_as_float((254u - ex) << 23) : 0.f;
        const int64_t row = s_row[t] + g * head;
        int8_t* dst = (key ? P2_pages : I_pages) + (size_t)row * pp.row + c;
        if (!finite)
#pragma unroll
            for (int e = 0; e < VC; ++e) a[e] = b[e] = 0.f;
        store_q8<VC>(dst, a, inv);
        store_q8<VC>(dst + HALF, b, inv);
        if (lane == 0)
            scales[2 * row + (key ? 0 : 1)] = __ushort_as_bfloat16(finite ? (unsigned short)(ex << 7) : (unsigned short)0x7fc0);
    }
}

// Rows [N, G, d] of some slots, as the values they stand for (exact in bf16): VC columns a thread, PER = d / VC threads
// a row, `tokens` tokens a block.
template <int VC, int PER>
__global__ void __launch_bounds__(kThreads)
    paged_read_q8_kernel(PagedProblem pp, const int64_t* __restrict__ slots, const int8_t* __restrict__ P2_pages,
                         const int8_t* __restrict__ I_pages, const __nv_bfloat16* __restrict__ scales,
                         __nv_bfloat16* __restrict__ P2, __nv_bfloat16* __restrict__ I, unsigned int* status, int tokens) {
    const int n0 = blockIdx.x * tokens, count = min(tokens, pp.N - n0), items = count * pp.G * PER;
    for (int k = threadIdx.x; k < items; k += kThreads) {
        const int row_of = k / PER, c = (k - row_of * PER) * VC, t = pp.by_G.div(row_of), g = row_of - t * pp.G, n = n0 + t;
        const int64_t slot = slots[n];
        const bool in = slot >= 0 && slot < ((int64_t)pp.pages << pp.page_shift);
        if (slot >= 0 && !in) record_status(status, kDevBadPosition);
        const size_t row = in ? page_row_index(pp, slot >> pp.page_shift, (int)(slot & pp.page_mask), g) : 0;
        const __nv_bfloat162 sc = *reinterpret_cast<const __nv_bfloat162*>(scales + 2 * row);
        uint32_t x[2][VC / 4] = {};
        if (in) {
#pragma unroll
            for (int w = 0; w < VC / 4; ++w) {
                x[0][w] = __ldg(reinterpret_cast<const uint32_t*>(P2_pages + row * pp.row + c + 4 * w));
                x[1][w] = __ldg(reinterpret_cast<const uint32_t*>(I_pages + row * pp.row + c + 4 * w));
            }
        }
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            const float s = in ? __bfloat162float(which ? sc.y : sc.x) : 0.f;
            float v[VC];
#pragma unroll
            for (int e = 0; e < VC; ++e) v[e] = s * (float)(int8_t)(x[which][e / 4] >> (8 * (e % 4)));
            Vec<__nv_bfloat16, VC> out;
            out.pack(v);
            out.store((which ? I : P2) + ((size_t)n * pp.G + g) * pp.d + c);
        }
    }
}

}  // namespace

cudaError_t launch_paged_store_q8(const PagedProblem& pp, const void* X1, const void* X2, const void* I,
                                  const float* theta, int pairing, const RopeTable& tab, const int* positions,
                                  const int64_t* slots, void* P1, void* P2_pages, void* I_pages, void* scales,
                                  unsigned int* status, int num_sms, cudaStream_t s) {
    using B = __nv_bfloat16;
    // A few blocks per SM first, then more tokens to a block.
    const int tokens = (int)std::min<int64_t>(kMaxTokens, std::max<int64_t>(1, (int64_t)pp.N / (4 * num_sms)));
    const unsigned blocks = (unsigned)(((int64_t)pp.N + tokens - 1) / tokens);
    const size_t sh = (size_t)(kMaxTokens * (pp.d / 2) + pp.G / 2) * sizeof(float2);
#define STORE(HALF, VC, LANES)                                                                                      \
    paged_store_q8_kernel<HALF, VC, LANES><<<blocks, kThreads, sh, s>>>(                                             \
        pp, (const B*)X1, (const B*)X2, (const B*)I, theta, pairing, tab, positions, slots, (B*)P1, (int8_t*)P2_pages, \
        (int8_t*)I_pages, (B*)scales, status, tokens, FastDiv((uint32_t)(pp.H + 2 * pp.G)));                          \
    return cudaGetLastError()
    switch (pp.d) {  // the widest access that d/2 columns and the rows' alignment allow
        case 48: STORE(24, 8, 4);
        case 60: STORE(30, 2, 16);
        case 64: STORE(32, 8, 4);
        case 80: STORE(40, 8, 8);
        case 128: STORE(64, 8, 8);
    }
#undef STORE
    return cudaErrorInvalidValue;
}

cudaError_t launch_paged_read_q8(const PagedProblem& pp, const int64_t* slots, const void* P2_pages, const void* I_pages,
                                 const void* scales, void* P2, void* I, unsigned int* status, int num_sms,
                                 cudaStream_t s) {
    using B = __nv_bfloat16;
    // Two rounds of a block's threads, as long as that leaves some blocks for every SM.
    const int vc = pp.d % 8 == 0 ? 8 : 4, per_token = pp.G * (pp.d / vc);
    const int tokens = (int)std::max<int64_t>(1, std::min<int64_t>(2 * kThreads / per_token, (int64_t)pp.N / (4 * num_sms)));
    const unsigned blocks = (unsigned)(((int64_t)pp.N + tokens - 1) / tokens);
    auto run = [&](auto kern) {
        kern<<<blocks, kThreads, 0, s>>>(pp, slots, (const int8_t*)P2_pages, (const int8_t*)I_pages, (const B*)scales,
                                         (B*)P2, (B*)I, status, tokens);
        return cudaGetLastError();
    };
    switch (pp.d) {
        case 48: return run(paged_read_q8_kernel<8, 6>);
        case 60: return run(paged_read_q8_kernel<4, 15>);
        case 64: return run(paged_read_q8_kernel<8, 8>);
        case 80: return run(paged_read_q8_kernel<8, 10>);
        case 128: return run(paged_read_q8_kernel<8, 16>);
    }
    return cudaErrorInvalidValue;
}

}  // namespace relation
