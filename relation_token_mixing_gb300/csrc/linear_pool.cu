// Linear Relation of packed new tokens over a pool of states: serving ("Ask
// Self, Ask Others", Sec. 5.2 eq.(15)-(17), Appendix A.4).  Per request and head,
// from the state C that its slot of the pool holds, token by token
//     C-_t = Diag(exp g_t) C_{t-1},  Y_t = I~_t + S_t (C-_t)^T p^1_t,
//     C_t  = C-_t + S_t p^2_t I~_t^T,  S_t = sigmoid(p1_t . p2_t / (tau_S sqrt d)),
// and the last C goes to the request's other slot (the same one, if the caller
// says so).
//
// Requests of at most kFewTokens new tokens run the recurrence as it stands
// (linear_few_kernel), longer ones in chunks of 64 tokens on the tensor cores
// (linear_chunk_kernel).  Single tokens are bound by the states' bytes; chunks by the instructions and latencies of
// forming their operands (a channel of a token: two exponentials, two scales, three roundings), far above the bytes.
// Measured: one token each of 512 requests, 16 heads of 64: 44 us, 6.2 TB/s; of 16 requests, 8 heads of 60: 3.0 us, one
// launch's latency; 16 tokens each of 64 requests, 16 heads of 64: 18.6 us, 23.4 with the gate; one request of 32768
// tokens, 8 heads of 60: 124 us, 1.5 TB/s; 24 prompts of up to 2048, 25198 tokens: 125 us; 60 single tokens and 4 chunks of
// 250 to 500, 16 heads of 64: 38 us.
//
// A chunk.  With q = S p^1, k = S p^2 and the running sum of the log-retentions
// G_t (from the chunk's start, in units of log2), the retention between tokens j
// and i is 2^(G_i - G_j), so with any reference m per channel
//     q~_i = q_i 2^(G_i - m),  k~_j = k_j 2^(m - G_j):
//     Y = I~ + strictly-lower(q~ k~^T) I~ + q~ (2^m C),
//     C <- 2^(G_end - m) (2^m C + k~^T I~)
// is the recurrence in four products of 64 x 64 x 64, all from the same two operands.
// m is half of what the chunk loses, G_end / 2: a chunk may then lose up to 2^(2 kRange) of
// a channel before a factor leaves the range of bf16.  A chunk that loses more in some
// channel, or has an |I~| above kLargest, takes another way to the same sums (strong_chunk below) whose factors
// are all retentions between two of its own tokens.
//
// Roundings: q~, the weights and the state as an operand of the output product are
// bf16, as the outputs are (2^m C to 2^-134, so an output has its share of the state to 2^-31 in absolute terms);
// k~ enters the state's product as a sum of three
// bf16 values (2^-25; of two, 2^-17, in a strongly fading chunk), since the state is kept in float32 from call
// to call: of two everywhere, the states of 32768 tokens are off by 2e-6 in place of less than 1e-6, 4 % sooner.
// Sums and the state itself are float32.  Exponents are running sums too: behind a token that takes 2^-190 from a channel
// at once, the largest that stays with one reference, what is added to the state is off by up to 2.2e-5 (2^-120: 1.0e-5,
// 2^-30: 2.6e-6, gentle retention: 5e-7; a strongly fading chunk, summed from its end: 7e-6).
#include <cuda_bf16.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "linear_common.cuh"
#include "linear_cut.h"
#include "linear_pool.h"
#include "once_per_device.h"
#include "ptx_sm100.cuh"
#include "tile_copy.cuh"

namespace relation {
namespace lin {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ void dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void dependency_release() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// softplus of two to a relative 2e-7 (softplus_f is exact to 1e-7 absolute, which a float32 state of
// weak retention would show): log(1 + y) = 2 artanh(s), s = y / (2 + y), y <= 1, with artanh(s) / s by a polynomial of
// degree 4 in s^2 <= 1/9 (fitted at Chebyshev nodes: 4e-9).
__device__ __forceinline__ float2 softplus_rel(float2 x) {
    const auto two = [](float c) { return make_float2(c, c); };
    const float2 y = make_float2(__expf(-fabsf(x.x)), __expf(-fabsf(x.y))), d = ptx::add2(y, two(2.f));
    const float2 s = make_float2(__fdividef(y.x, d.x), __fdividef(y.y, d.y)), z = ptx::mul2(s, s);
    float2 t = ptx::fma2(z, two(0.140873283f), two(0.139807090f));
    t = ptx::fma2(z, t, two(0.200124264f));
    t = ptx::fma2(z, t, two(0.333331585f));
    t = ptx::fma2(z, t, two(1.f));
    return ptx::fma2(ptx::add2(s, s), t, make_float2(fmaxf(x.x, 0.f), fmaxf(x.y, 0.f)));
}

// log2 of the retention of one thread's channels c, c + 1 of head h from what G holds.
struct Gate {
    float2 na, db;  // -exp(A_log) log2(e) and dt_bias, or log2(e) and nothing
};
template <bool kGate>
__device__ __forceinline__ Gate gate_of(const LinearPool& p, int h, int c) {
    Gate g{make_float2(kLog2e, kLog2e), make_float2(0.f, 0.f)};
    if (kGate) {
        g.na = make_float2(0.f, 0.f);
        if (c < p.d) {
            const size_t o = (size_t)h * p.d + c;
            g.na = make_float2(-expf(p.A_log[o]) * kLog2e, -expf(p.A_log[o + 1]) * kLog2e);
            g.db = make_float2(p.dt_bias[o], p.dt_bias[o + 1]);
        }
    }
    return g;
}
// The larger of two, NaN if one is (fmaxf gives the other).
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// At least -280: 2^-280 of any float32 is 0, and sums of a chunk's terms keep their fractions.
template <bool kGate>
__device__ __forceinline__ float2 log2_retention(float2 x, const Gate& g) {
    const float2 e = ptx::mul2(kGate ? softplus_rel(ptx::add2(x, g.db)) : x, g.na);
    return make_float2(max_nan(e.x, -280.f), max_nan(e.y, -280.f));
}

// A request's tokens; ones that cannot be followed give count = -1 and are reported.
__device__ __forceinline__ Span span_of(const LinearPool& p, int r) {
    if (p.starts == nullptr) return Span{r, 1};
    const Span sp = span_between(__ldg(p.starts + r), __ldg(p.starts + r + 1), p.N, p.max_fresh);
    if (sp.count < 0) record_status(p.status, kDevBadPosition);
    return sp;
}
// The state a slot names, or nullptr (negative: none; past the pool: reported).
__device__ __forceinline__ float* state_of(const LinearPool& p, int slot, int h) {
    if (slot >= p.slots) record_status(p.status, kDevBadPosition);
    if (slot < 0 || slot >= p.slots) return nullptr;
    return p.states + ((size_t)slot * p.H + h) * p.d * p.d;
}

// A stretch of a request for one block of the chunked kernels: segment `seg` of `segs`.
struct Item {
    int r, first, count;
    int seg_segs;  // seg | segs << 16 (segs = 0: no such item)
};
// What block 0 of the first kernel leaves for the others (items = nullptr: every request is one segment).
struct Plan {
    Item* items;
    int *order, *joins;
    int most_items, most_joins, seg_tokens;
    bool beside;  // the requests of few tokens run beside the others, which were launched before them
};

// ------------------------------------------------------------ the recurrence
// One block per request and head: thread (rg, cg) has rows rg + 8 i and columns 4 cg ..
// 4 cg + 3 of the state, in registers over all the request's tokens, so that the state
// is read and written once, 8 d d bytes, which bounds it.  The first kFewTokens tokens'
// vectors are made by the warps in turn while the state is on its way.
constexpr int kFewThreads = 128;

// A token's vectors in shared memory, of as many tokens as a request may have.
constexpr int few_smem(int max_fresh) { return std::min(max_fresh, kFewTokens) * 4 * kDp * (int)sizeof(float); }

// Block 0 of a packed call with items: the longer requests' segments, a request's side by side and equal but for whole
// chunks; where the requests of more than one begin; and the order in which blocks take the segments, the longest
// first (those of one length in any order), so that the last to start are short. A request with rows before the end
// of an earlier one is reported and has none: the list has places for each row once.
__device__ void make_items(const LinearPool& p, const Plan& plan) {
    constexpr int kBins = 64;  // of segments by their chunks, 63 and more together
    __shared__ int sums[kFewThreads / 32], ends[kFewThreads / 32], many, bins[kBins];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const auto bin_of = [](int tokens) { return kBins - 1 - min((tokens + kChunk - 1) / kChunk, kBins - 1); };
    if (tid == 0) many = 0;
    for (int k = tid; k < kBins; k += kFewThreads) bins[k] = 0;
    int base = 0, end = 0;  // segments of the requests before, and the end of their rows
    for (int r0 = 0; r0 < p.R; r0 += kFewThreads) {
        const int r = r0 + tid;
        Span sp{0, 0};
        if (r < p.R) sp = span_of(p, r);
        int e = sp.end();
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, e, o);
            if (lane >= o) e = max(e, y);
        }
        if (lane == 31) ends[warp] = e;
        __syncthreads();
        int before = __shfl_up_sync(0xffffffffu, e, 1);
        before = max(end, lane ? before : 0);
        for (int w = 0; w < kFewThreads / 32; ++w) {
            if (w < warp) before = max(before, ends[w]);
            end = max(end, ends[w]);
        }
        const Segments sg = segments_of(sp, before, plan.seg_tokens);
        if (sg.refused) record_status(p.status, kDevBadPosition);
        int x = sg.count;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) sums[warp] = x;
        __syncthreads();
        int at = base + x - sg.count;
        for (int w = 0; w < kFewThreads / 32; ++w) {
            if (w < warp) at += sums[w];
            base += sums[w];
        }
        const bool fits = at + sg.count <= plan.most_items;  // (always: cut_of)
        for (int k = 0; k < sg.count && at + k < plan.most_items; ++k) {
            const int count = fits ? min(sg.tokens, sp.count - k * sg.tokens) : 0;
            plan.items[at + k] = Item{r, sp.first + k * sg.tokens, count, k | sg.count << 16};
            atomicAdd(&bins[bin_of(count)], 1);
        }
        if (sg.count > 1 && fits) {  // in any order
            const int k = atomicAdd(&many, 1);
            if (k < plan.most_joins) plan.joins[k] = at;
        }
        __syncthreads();
    }
    base = min(base, plan.most_items);
    for (int k = many + tid; k < plan.most_joins; k += kFewThreads) plan.joins[k] = -1;
    if (warp == 0) {  // where each length's begin
        const int a = bins[2 * lane], b = bins[2 * lane + 1];
        int x = a + b;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        bins[2 * lane] = x - a - b, bins[2 * lane + 1] = x - b;
    }
    __syncthreads();
    for (int k = tid; k < plan.most_items; k += kFewThreads) {
        if (k < base) plan.order[atomicAdd(&bins[bin_of(plan.items[k].count)], 1)] = k;
        else plan.order[k] = -1;
    }
}

template <int D, bool kGate>
__global__ void __launch_bounds__(kFewThreads)
    linear_few_kernel(const __grid_constant__ LinearPool p, const __grid_constant__ Plan plan) {
    extern __shared__ __align__(16) float few[];
    __shared__ __align__(16) float part[2][8][kDp];
    const int most = min(p.max_fresh, kFewTokens);
    float (*const sa)[kDp] = reinterpret_cast<float (*)[kDp]>(few), (*const sq)[kDp] = sa + most, (*const sk)[kDp] = sq + most,
          (*const sv)[kDp] = sk + most;
    constexpr int kCols = D / 4, kRows = (D + 7) / 8;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // Beside the chunks' kernel only the grid's end has to wait for that kernel's: all of its blocks have waited for what
    // ran before the call when they release this one.  So it may only be launched right behind that kernel, which
    // must not release before it has waited.
    if (!plan.beside) dependency_wait();
    dependency_release();
    if (plan.beside && blockIdx.x == gridDim.x - 1) {
        dependency_wait();
        return;
    }
    int x = blockIdx.x;
    if (plan.items != nullptr) {
        if (x == 0) {
            make_items(p, plan);
            return;
        }
        --x;
    }
    const int r = x / p.H, h = x - r * p.H;
    const Span sp = span_of(p, r);
    if (sp.count < 0 || sp.count > kFewTokens) return;
    const float* in = state_of(p, __ldg(p.slots_in + r), h);
    float* out = state_of(p, __ldg(p.slots_out + r), h);
    if (sp.count == 0 && in == out) return;

    const int cg = tid % kCols, rg = tid / kCols;
    const bool active = rg < 8;
    float4 C[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int c = rg + 8 * i;
        C[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (active && c < D && in != nullptr) C[i] = *reinterpret_cast<const float4*>(in + c * D + 4 * cg);
    }
    // Tokens' vectors, a warp a token, a lane two channels.
    {
        const int c = 2 * lane;
        const bool has = c < D;
        const Gate gate = gate_of<kGate>(p, h, c);
        for (int t = warp; t < sp.count; t += kFewThreads / 32) {
            const size_t at = ((size_t)(sp.first + t) * p.H + h) * D + c;
            uint32_t w1 = 0, w2 = 0, wv = 0;
            float2 g = make_float2(0.f, 0.f);
            if (has) {
                w1 = __ldg(reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(p.P1) + at));
                w2 = __ldg(reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(p.P2) + at));
                wv = __ldg(reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(p.I) + at));
                g = __ldg(reinterpret_cast<const float2*>(p.G + at));
            }
            float n1 = lo_f(w1) * lo_f(w1) + hi_f(w1) * hi_f(w1), n2 = lo_f(w2) * lo_f(w2) + hi_f(w2) * hi_f(w2);
            float dt = lo_f(w1) * lo_f(w2) + hi_f(w1) * hi_f(w2);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                n1 += __shfl_xor_sync(0xffffffffu, n1, o);
                n2 += __shfl_xor_sync(0xffffffffu, n2, o);
                dt += __shfl_xor_sync(0xffffffffu, dt, o);
            }
            const float S = 1.f / (1.f + __expf(-dt * p.zscale));
            const float s1 = n1 > 0.f ? S * rsqrtf(n1) : 0.f, s2 = n2 > 0.f ? S * rsqrtf(n2) : 0.f;
            const float2 e = log2_retention<kGate>(g, gate);
            *reinterpret_cast<float2*>(&sa[t][c]) = make_float2(exp2f(e.x), exp2f(e.y));
            *reinterpret_cast<float2*>(&sq[t][c]) = make_float2(lo_f(w1) * s1, hi_f(w1) * s1);
            *reinterpret_cast<float2*>(&sk[t][c]) = make_float2(lo_f(w2) * s2, hi_f(w2) * s2);
            *reinterpret_cast<float2*>(&sv[t][c]) = make_float2(lo_f(wv), hi_f(wv));
        }
    }
    __syncthreads();
    __nv_bfloat16* Y = static_cast<__nv_bfloat16*>(p.Y);
    for (int t = 0; t < sp.count; ++t) {
        if (active) {
            const float4 v = *reinterpret_cast<const float4*>(&sv[t][4 * cg]);
            float4 e = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                const int c = rg + 8 * i;
                if (c >= D) break;
                const float a = sa[t][c], q = sq[t][c], k = sk[t][c];
                C[i] = make_float4(C[i].x * a, C[i].y * a, C[i].z * a, C[i].w * a);
                e = make_float4(fmaf(q, C[i].x, e.x), fmaf(q, C[i].y, e.y), fmaf(q, C[i].z, e.z), fmaf(q, C[i].w, e.w));
                C[i] = make_float4(fmaf(k, v.x, C[i].x), fmaf(k, v.y, C[i].y), fmaf(k, v.z, C[i].z),
                                   fmaf(k, v.w, C[i].w));
            }
            *reinterpret_cast<float4*>(&part[t & 1][rg][4 * cg]) = e;
        }
        __syncthreads();  // the other buffer's readers are a token behind: past the next barrier
        if (tid < D / 2) {
            float2 y = *reinterpret_cast<const float2*>(&sv[t][2 * tid]);
#pragma unroll
            for (int g = 0; g < 8; ++g) {
                const float2 e = *reinterpret_cast<const float2*>(&part[t & 1][g][2 * tid]);
                y.x += e.x, y.y += e.y;
            }
            *reinterpret_cast<uint32_t*>(Y + ((size_t)(sp.first + t) * p.H + h) * D + 2 * tid) = pack2(y.x, y.y);
        }
    }
    if (out != nullptr && active) {
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int c = rg + 8 * i;
            if (c < D) *reinterpret_cast<float4*>(out + c * D + 4 * cg) = C[i];
        }
    }
}

// ------------------------------------------------------------------- chunks
constexpr int kT = kChunk;
constexpr int kThreads = 256;
constexpr float kRange = 100.f;   // log2 of half of what a chunk may lose of a channel
constexpr float kLargest = 0x1p20f;  // of |I~|: 64 terms of 2^(kRange + 20) stay below 2^127
constexpr int kTile = kT * 128;   // a bf16 tile of 64 x 64
constexpr int kGp = kDp + 8;      // of a row of sums: eight rows' same columns on different banks
constexpr int kSegFloats = kDp * kDp + kDp;  // of a segment in the workspace: its state, the log2 of its retention

struct ChunkStage {
    uint8_t p1[kTile];  // q~ in place of p1, the larger part of k~ in place of p2, once they are made
    uint8_t p2[kTile];
    uint8_t v[kTile];
};
struct ChunkSmem {
    ChunkStage st[2];
    union {
        struct {
            uint8_t kl[kTile];  // what bf16 leaves of k~
            uint8_t c[kTile];   // the state as an operand, [value channel][key channel]
        };
        float g[kT * kGp];  // (strong_chunk)
        struct {
            uint8_t below[kTile];
            float tot[8][kDp];  // a warp's 8 tokens: sum of log2 of their retentions
        };
    };
    uint8_t w[kTile];  // the weights inside the chunk, [query][key]; before, what two bf16 leave of k~
    float c_half[kDp], c_all[kDp];  // per channel: factor of the state as an operand and of what the chunk adds; of the
                                    // state through the chunk
    float2 rs[kT];        // (S / |p1|, S / |p2|) of a token
    uint64_t c_done, o_done, drain;
    uint32_t tmem;
    int abort_flag;
};
static_assert(sizeof(ChunkStage) % 1024 == 0, "tiles on swizzle atoms");

// Accumulators of 64 rows lie in lanes 0-15 of each of the four warps' 32: row r in lane 32 (r / 16) + r % 16.
constexpr uint32_t kColW = 0, kColO = 0, kColC = 64, kTmemCols = 128;  // O overwrites the scores once they are read

// 16 rows x 32 columns of an accumulator as four fragments of m16n8: x[n][0, 1] row lane / 4, columns 8 n + 2 (lane % 4)
// and the next, x[n][2, 3] the row 8 further.
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t (&x)[4][4]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(x[0][0]), "=r"(x[0][1]), "=r"(x[0][2]), "=r"(x[0][3]), "=r"(x[1][0]), "=r"(x[1][1]), "=r"(x[1][2]),
          "=r"(x[1][3]), "=r"(x[2][0]), "=r"(x[2][1]), "=r"(x[2][2]), "=r"(x[2][3]), "=r"(x[3][0]), "=r"(x[3][1]),
          "=r"(x[3][2]), "=r"(x[3][3])
        : "r"(taddr));
    ptx::tmem_ld_wait();
#pragma unroll
    for (int n = 0; n < 4; ++n) ptx::pin_regs(x[n]);
}
// Four 8 x 8 blocks of bf16 pairs from such fragments into a tile.
__device__ __forceinline__ void stsm4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
                 "r"(d)
                 : "memory");
}

// A chunk's rows: those past the stretch's end are zero, as the columns past d stay.
struct Loader {
    int row, col;
    uint32_t dst;

    __device__ __forceinline__ explicit Loader(const LinearPool& p) {
        const int tid = threadIdx.x;
        const bool wide = (p.d & 7) == 0;  // else rows of 120 bytes, which start on 8
        row = wide ? tid >> 3 : tid >> 4;
        col = wide ? 8 * (tid & 7) : 4 * (tid & 15);
        dst = swz(row, col);
    }
    // first: the element that the chunk's first row begins at; left: tokens from this chunk on.
    template <bool kAll>
    __device__ __forceinline__ void rows(const ChunkStage& s, const LinearPool& p, size_t first, int left) const {
        const uint32_t stride = (uint32_t)(p.H * p.d);
        const size_t at = (first + (size_t)row * stride + col) * 2;
        const char* src[3] = {static_cast<const char*>(p.P1) + at, static_cast<const char*>(p.P2) + at,
                              static_cast<const char*>(p.I) + at};
        const uint32_t to = ptx::smem_u32(s.p1) + dst;
        if ((p.d & 7) == 0) {
#pragma unroll
            for (int k = 0; k < 3; ++k)
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    if (kAll || row + 32 * r < left) cp_async_16(to + k * kTile + r * 32 * 128, src[k] + (size_t)(r * 64 * stride));
                    else st_zero16(to + k * kTile + r * 32 * 128);
        } else {
#pragma unroll
            for (int k = 0; k < 3; ++k)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (kAll || row + 16 * r < left) cp_async_8(to + k * kTile + r * 16 * 128, src[k] + (size_t)(r * 32 * stride));
                    else st_shared_zero8(to + k * kTile + r * 16 * 128);
        }
    }
    __device__ __forceinline__ void chunk_into(const ChunkStage& s, const LinearPool& p, size_t first, int left) const {
        if (col < p.d) {
            if (left >= kT) rows<true>(s, p, first, left);
            else rows<false>(s, p, first, left);
        }
        cp_async_commit();
    }
};

__device__ __forceinline__ float2 add2(float2 a, float2 b) { return ptx::add2(a, b); }

// The warp's 8 tokens: |p1|^2, |p2|^2, |I~|^2 and p1 . p2 are the diagonals of 8 x 8 products of the rows with
// one another (a row's fragment is the same on both sides, and p1's and p2's stand over each other), then S / |p1| and
// S / |p2|.  Twelve products and six fetches in place of some 200 multiply-adds and shuffles.  Returns whether the lane's
// |I~| is above kLargest.
__device__ __forceinline__ bool row_scalars(ChunkSmem& sm, const ChunkStage& s, float zscale, int warp, int lane) {
    float n1_dt[4] = {}, n2[4] = {}, nv[4] = {};
    const uint32_t at = 8 * warp * 128 + swz(lane & 7, 8 * (lane >> 3)), at2 = 8 * warp * 128 + swz(lane & 7, 32 + 8 * (lane >> 3));
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        uint32_t x[4], y[4], v[4];
        ldsm4(x, ptx::smem_u32(s.p1) + (k ? at2 : at));
        ldsm4(y, ptx::smem_u32(s.p2) + (k ? at2 : at));
        ldsm4(v, ptx::smem_u32(s.v) + (k ? at2 : at));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t axy[4] = {x[2 * h], y[2 * h], x[2 * h + 1], y[2 * h + 1]};
            const uint32_t ay[4] = {y[2 * h], 0u, y[2 * h + 1], 0u}, av[4] = {v[2 * h], 0u, v[2 * h + 1], 0u};
            mma16816(n1_dt, axy, x[2 * h], x[2 * h + 1]);
            mma16816(n2, ay, y[2 * h], y[2 * h + 1]);
            mma16816(nv, av, v[2 * h], v[2 * h + 1]);
        }
    }
    const int g = lane >> 2;
    bool large = false;
    if ((lane & 3) == g >> 1) {  // the diagonal's entry of row g
        const float a = g & 1 ? n1_dt[1] : n1_dt[0], b = g & 1 ? n2[1] : n2[0], x = g & 1 ? n1_dt[3] : n1_dt[2];
        const float S = 1.f / (1.f + __expf(-x * zscale));
        sm.rs[8 * warp + g] = make_float2(a > 0.f ? S * rsqrtf(a) : 0.f, b > 0.f ? S * rsqrtf(b) : 0.f);
        large = (g & 1 ? nv[1] : nv[0]) > kLargest * kLargest;
    }
    __syncwarp();
    return large;
}

// The weights (in sm.w), q k^T with the retention between the two tokens, for a chunk whose factors from one
// reference would leave bf16's range: sm.g holds G, s.p1 and s.p2 the rows as they came.  Of each 16 queries, keys
// before them meet the queries at the block's first token, the block's first 8 keys its last 8 queries at the ninth:
// all factors are retentions.  What is left are pairs inside 8 tokens, a lane a pair.  Warps w and w + 4 share 16
// queries, 8 keys in turn.  Behind n tokens that forget everything the sums keep an exponent to 280 n 2^-24, 2^-10 at
// most: less than the weights' rounding, 2^-8.  Chunks like this are rare; one costs its block some 9 us (others: 4), most of it code that
// no other block has fetched.
__device__ __noinline__ void strong_chunk(ChunkSmem& sm, const ChunkStage& s, int warp, int lane) {
    const int g = lane >> 2, t = lane & 3, rt = warp & 3, half = warp >> 2, i0 = 16 * rt + g;
    const auto row_of = [](const uint8_t* tile, int r, int c) { return *reinterpret_cast<const uint32_t*>(tile + swz(r, c)); };
    const auto sum_of = [&](int r, int c) { return *reinterpret_cast<const float2*>(sm.g + r * kGp + c); };
    // q (or k) of row r, columns c and c + 1, times 2^(+-(G_r - B)) as a bf16 pair.
    const auto scaled = [&](bool query, int r, float2 B, int c) {
        const float2 G = sum_of(r, c);
        const uint32_t x = row_of(query ? s.p1 : s.p2, r, c);
        const float f = query ? sm.rs[r].x : sm.rs[r].y;
        const float2 e = query ? make_float2(G.x - B.x, G.y - B.y) : make_float2(B.x - G.x, B.y - G.y);
        return pack2(lo_f(x) * f * ptx::ex2_approx(e.x), hi_f(x) * f * ptx::ex2_approx(e.y));
    };
    const auto put = [&](int row, int n, float a, float b) {
        *reinterpret_cast<uint32_t*>(sm.w + swz(row, 8 * n + 2 * t)) = pack2(a, b);
    };
    float w[3][4] = {}, last[4] = {};
#pragma unroll 1
    for (int c = 2 * t; c < kDp; c += 16) {
        if (rt > 0) {
            const float2 B0 = sum_of(16 * rt - 1, c), B1 = sum_of(16 * rt - 1, c + 8);
            const uint32_t a[4] = {scaled(true, i0, B0, c), scaled(true, i0 + 8, B0, c), scaled(true, i0, B1, c + 8),
                                   scaled(true, i0 + 8, B1, c + 8)};
#pragma unroll
            for (int k = 0; k < 3; ++k)
                if (k < rt) {
                    const int j = 8 * (2 * k + half) + g;
                    mma16816(w[k], a, scaled(false, j, B0, c), scaled(false, j, B1, c + 8));
                }
        }
        if (half == 0) {
            const float2 B0 = sum_of(16 * rt + 7, c), B1 = sum_of(16 * rt + 7, c + 8);
            const uint32_t a[4] = {0u, scaled(true, i0 + 8, B0, c), 0u, scaled(true, i0 + 8, B1, c + 8)};
            mma16816(last, a, scaled(false, i0, B0, c), scaled(false, i0, B1, c + 8));
        }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int n = 2 * k + half;
        if (k != rt) {
            const bool before = k < rt;
            put(i0, n, before ? w[k < 3 ? k : 0][0] : 0.f, before ? w[k < 3 ? k : 0][1] : 0.f);
            put(i0 + 8, n, before ? w[k < 3 ? k : 0][2] : 0.f, before ? w[k < 3 ? k : 0][3] : 0.f);
        } else if (half == 0) {
            put(i0 + 8, n, last[2], last[3]);
        } else {
            put(i0, n, 0.f, 0.f);
        }
    }
    // The 28 pairs of the warp's own 8 tokens; zeros on and above the diagonal.
    put(8 * warp + g, warp, 0.f, 0.f);
    __syncwarp();
    if (lane < 28) {
        int i = 1, j = lane;
        while (j >= i) j -= i++;
        i += 8 * warp, j += 8 * warp;
        float2 x = make_float2(0.f, 0.f);
#pragma unroll 2
        for (int c = 0; c < kDp; c += 2) {
            const float2 Gi = sum_of(i, c), Gj = sum_of(j, c);
            const uint32_t q = row_of(s.p1, i, c), k = row_of(s.p2, j, c);
            x.x += lo_f(q) * lo_f(k) * ptx::ex2_approx(Gi.x - Gj.x);
            x.y += hi_f(q) * hi_f(k) * ptx::ex2_approx(Gi.y - Gj.y);
        }
        *reinterpret_cast<__nv_bfloat16*>(sm.w + swz(i, j)) = __float2bfloat16_rn((x.x + x.y) * (sm.rs[i].x * sm.rs[j].y));
    }
}

// One block a segment of a request and head: the output pass (kOut) from the state that
// enters it, or the state pass, which leaves the segment's own contribution and retention.
//
// The chunk's elements are the threads' (warp w has tokens 8 w .. 8 w + 7, a lane two channels; the retention comes
// straight to their registers, a chunk ahead), its four products tcgen05's: scores q~ k~^T and the state's addition
// I~^T k~ as soon as the operands are there, then O = w I~ + q~ C into the scores' columns once those are read.  Of the
// accumulators' 64 rows, a warp reads the 16 of its quarter (w % 4), columns 32 (w / 4) and on, as fragments of
// m16n8: of the weights, of O and of the state's addition, whose rows are value channels and whose columns key
// channels; the state itself stays in such fragments, from chunk to chunk.
template <bool kOut, bool kGate>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    linear_chunk_kernel(const __grid_constant__ LinearPool p, const __grid_constant__ Plan plan, float* __restrict__ segments) {
    extern __shared__ uint8_t smem_raw[];
    ChunkSmem& sm =
        *reinterpret_cast<ChunkSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int x = blockIdx.x / p.H;
    const int h = blockIdx.x - x * p.H;
    dependency_wait();
    dependency_release();
    Item it{x, 0, 0, 1 << 16};
    if (plan.items != nullptr) {
        x = plan.order[x];
        if (x < 0) return;
        it = plan.items[x];
    } else {
        const Span sp = span_of(p, it.r);
        it.first = sp.first, it.count = sp.count;
    }
    const int seg = it.seg_segs & 0xffff, segs = it.seg_segs >> 16;
    if (it.count <= (segs > 1 ? 0 : kFewTokens) || (!kOut && seg + 1 == segs)) return;
    if (tid == 0) {
        for (uint64_t* bar : {&sm.c_done, &sm.o_done, &sm.drain}) ptx::mbar_init(bar, 1);
        sm.abort_flag = 0;
        ptx::fence_barrier_init();
    }
    // Zeros for the columns past d, which no copy writes.
    if (p.d < kDp)
        for (int k = tid; k < 6 * kT; k += kThreads) {
            uint8_t* tile = sm.st[k / (3 * kT)].p1 + k / kT % 3 * kTile;
            for (int c = p.d & ~7; c < kDp; c += 8) *reinterpret_cast<uint4*>(tile + swz(k % kT, c)) = make_uint4(0, 0, 0, 0);
        }
    if (warp == 0) {
        ptx::tmem_alloc(&sm.tmem, kTmemCols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = sm.tmem;
    const size_t row = ((size_t)it.first * p.H + h) * p.d;
    const int chunks = (it.count + kT - 1) / kT;
    const uint32_t stride = (uint32_t)(p.H * p.d);
    const Loader load(p);
    load.chunk_into(sm.st[0], p, row, it.count);
    // The lane's channels of the warp's 8 tokens: what G holds of them, then its running sums.
    const int c2 = 2 * lane;
    float2 G[8];
    auto load_g = [&](size_t first, int left) {
        const float* src = p.G + first + (size_t)(8 * warp) * stride + c2;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            G[i] = make_float2(0.f, 0.f);
            if (c2 < p.d && 8 * warp + i < left)
                asm volatile("ld.global.nc.v2.f32 {%0, %1}, [%2];" : "=f"(G[i].x), "=f"(G[i].y) : "l"(src + i * stride));
        }
    };
    load_g(row, it.count);

    const int g = lane >> 2, t = lane & 3, quarter = warp & 3, r0 = 16 * quarter + g, col0 = 32 * (warp >> 2);
    const uint32_t lane_addr = tmem + ((uint32_t)(32 * quarter) << 16) + col0;
    // Where a lane's row of stsm4's (and ldsm4's) four blocks begins: rows 16 quarter .. + 15, columns col0 .. + 15; the
    // next 16 columns are two chunks further, which the permutation turns into an exclusive-or.
    const uint32_t frag_at = swz(16 * quarter + (lane & 15), col0 + 8 * (lane >> 4)), frag_next = frag_at ^ 32;
    // Rows r0, r0 + 8 of the state C^T, columns col0 + 8 n + 2 t and the next.
    float2 C[4][2];
    float* mine = segments == nullptr ? nullptr : segments + ((size_t)x * p.H + h) * kSegFloats;
    {
        const float* in = nullptr;
        int ld = p.d;
        if (kOut) {
            if (segs > 1) in = mine, ld = kDp;
            else in = state_of(p, __ldg(p.slots_in + it.r), h);
        }
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int v = r0 + 8 * e, c = col0 + 8 * n + 2 * t;  // (widths are even)
                C[n][e] = in != nullptr && v < ld && c < ld ? make_float2(in[(size_t)c * ld + v], in[(size_t)(c + 1) * ld + v])
                                                            : make_float2(0.f, 0.f);
            }
    }
    const uint32_t own = 8 * warp * 128 + ((c2 & 7) << 1);  // the lane's channels in its tokens' rows, see `at`
    const Gate gate = gate_of<kGate>(p, h, c2);
    // log2 of the retention of the warp's token i, `left` tokens from the chunk's first one on, from what G holds.
    auto retention = [&](float2 g, int i, int left) {
        const float2 e = log2_retention<kGate>(g, gate);
        return kGate && (8 * warp + i >= left || c2 >= p.d) ? make_float2(0.f, 0.f) : e;  // (a gate opens at zero)
    };
    auto retention_of = [&](int n, int i, int left) {
        float2 g = make_float2(0.f, 0.f);
        if (c2 < p.d && 8 * warp + i < left)
            g = __ldg(reinterpret_cast<const float2*>(p.G + row + ((size_t)n * kT + 8 * warp + i) * stride + c2));
        return retention(g, i, left);
    };
    float2 lost = make_float2(0.f, 0.f);  // log2 of the segment's retention
    // Operands along a row (K) or across rows (M).
    constexpr uint32_t kKK = ptx::idesc_bf16(64, 64, false, false), kKM = ptx::idesc_bf16(64, 64, false, true),
                       kMM = ptx::idesc_bf16(64, 64, true, true);
    constexpr uint32_t kStepK = 32 >> 4, kStepM = 2048 >> 4;  // 16 columns, 16 rows
    const uint64_t desc0 = ptx::smem_desc(0, kTile, 1024, ptx::kSwizzle128B);
    const uint32_t desc_high = ptx::desc_hi(desc0);
    auto desc = [&](const uint8_t* tile) { return ptx::desc_lo(desc0) | ((ptx::smem_u32(tile) & 0x3FFFFu) >> 4); };
    volatile int* abort_flag = &sm.abort_flag;
    bool ok = true;
    // One warp asks for the products' end, the others wait for that warp: eight that ask took two fifths of the
    // instructions.
    auto wait = [&](uint64_t* bar, int n) {
        if (warp == 0 && ok) ok = ptx::mbar_wait_warp(bar, n & 1, abort_flag, p.status, kDevTimeoutMma);
        __syncthreads();
        ptx::tc_fence_after();
    };
    // The same code twice: without the strong chunks' way, and with it for the chunks that turn out to need it, which
    // start over. In one, what that way needs takes registers from every chunk (mixed step of 64 requests, 16 heads of
    // 64: 46 us against 42).
    enum { kNext, kStop };
    auto chunk = [&](int n, auto rare) {
        constexpr bool kRare = decltype(rare)::value;
        ChunkStage& s = sm.st[n & 1];
        const int left = it.count - n * kT;  // tokens from this chunk on
        cp_async_wait<0>();
        // The chunk is there, and nothing reads the one before any more.
        if (!__syncthreads_and(ok)) {
            ok = false;
            return kStop;
        }
        if (n + 1 < chunks) load.chunk_into(sm.st[(n + 1) & 1], p, row + (size_t)(n + 1) * kT * stride, left - kT);
        const bool large = row_scalars(sm, s, p.zscale, warp, lane);
        // The running sums inside the warp's 8 tokens.
        float2 sum = make_float2(0.f, 0.f);
        float most = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 e = retention(G[i], i, left);
            if (!kGate) most = ptx::max3(most, e.x, e.y);
            sum = add2(sum, e);
            G[i] = sum;
        }
        *reinterpret_cast<float2*>(&sm.tot[warp][c2]) = sum;
        // A state that grows may do so at one token and fade at others: the sums say nothing then.  Nor may a large I~
        // meet k~, which is up to 2^kRange: their sum would pass float32 before 2^m takes that back.
        const bool grows = __syncthreads_or(large || most > 0.f);
        float2 base = make_float2(0.f, 0.f), all = base;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            if (w == warp) base = all;
            all = add2(all, *reinterpret_cast<const float2*>(&sm.tot[w][c2]));
        }
        const float2 half = mul2(all, make_float2(0.5f, 0.5f));
        // The same for every warp.
        const bool is_strong = grows || __any_sync(0xffffffffu, !(fminf(half.x, half.y) >= -kRange));
        if (!kRare && is_strong) return kStop;
        const bool strong = kRare && is_strong;
        lost = add2(lost, all);
        float2 later = make_float2(0.f, 0.f);  // (strong) from the warp's tokens to the chunk's end
        if (strong) {
#pragma unroll
            for (int x = 0; x < 8; ++x)
                if (x > warp) later = add2(later, *reinterpret_cast<const float2*>(&sm.tot[x][c2]));
            if (kOut) {
                __syncthreads();  // before the sums are overwritten
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    *reinterpret_cast<float2*>(sm.g + (8 * warp + i) * kGp + c2) = add2(base, G[i]);
                __syncthreads();
                strong_chunk(sm, s, warp, lane);
                __syncthreads();  // before the rows are overwritten
            }
        }
        // The operands, in the rows' places: a warp's own tokens, a lane's own channels.  Exponents: of a query
        // G - m and of a key its negative; in a strong chunk from the chunk's start, and to its end.
        const bool third = !kOut || !strong;  // of k~, in the weights' place until those are there
        auto operands = [&](int i, float2 eq, float2 ek) {
            const uint32_t at = own + i * 128 + (((lane >> 2) ^ i) << 4);  // swz(8 warp + i, c2)
            const float2 f = sm.rs[8 * warp + i];
            if (kOut) {
                const uint32_t x = *reinterpret_cast<const uint32_t*>(s.p1 + at);
                const float2 q = mul2(mul2(make_float2(lo_f(x), hi_f(x)), make_float2(f.x, f.x)),
                                      make_float2(ptx::ex2_approx(eq.x), ptx::ex2_approx(eq.y)));
                *reinterpret_cast<uint32_t*>(s.p1 + at) = pack2(q.x, q.y);
            }
            const uint32_t y = *reinterpret_cast<const uint32_t*>(s.p2 + at);
            const float2 k = mul2(mul2(make_float2(lo_f(y), hi_f(y)), make_float2(f.y, f.y)),
                                  make_float2(ptx::ex2_approx(ek.x), ptx::ex2_approx(ek.y)));
            const uint32_t hi = pack2(k.x, k.y);
            *reinterpret_cast<uint32_t*>(s.p2 + at) = hi;
            const float2 lo = add2(k, make_float2(-lo_f(hi), -hi_f(hi)));
            const uint32_t l = pack2(lo.x, lo.y);
            *reinterpret_cast<uint32_t*>(sm.kl + at) = l;
            if (third) {
                const float2 least = add2(lo, make_float2(-lo_f(l), -hi_f(l)));
                *reinterpret_cast<uint32_t*>(sm.w + at) = pack2(least.x, least.y);
            }
        };
        if (!strong) {
            const float2 from = make_float2(base.x - half.x, base.y - half.y);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 eq = add2(from, G[i]);
                operands(i, eq, make_float2(-eq.x, -eq.y));
            }
        } else {
            // A key's retention to the end is summed from the end: as a difference of sums from the start, a token
            // that forgets everything between takes the fraction of what is left with it (the states of four such tokens
            // in a row were off by 5e-5 of their sums of magnitudes, so by 7e-6).  What G held is read again: a
            // loop, one copy of the code in the state pass; unrolled, 2 us of 122 (one request of 32768 tokens).
#pragma unroll 1
            for (int i = 7; i >= 0; --i) {
                float2 prefix = G[0];
#pragma unroll
                for (int j = 1; j < 8; ++j)
                    if (j == i) prefix = G[j];
                operands(i, add2(base, prefix), later);
                later = add2(later, retention_of(n, i, left));
            }
        }
        if (warp == 1) {
            const float2 one = make_float2(1.f, 1.f);
            *reinterpret_cast<float2*>(&sm.c_all[c2]) = make_float2(ptx::ex2_approx(all.x), ptx::ex2_approx(all.y));
            *reinterpret_cast<float2*>(&sm.c_half[c2]) =
                strong ? one : make_float2(ptx::ex2_approx(half.x), ptx::ex2_approx(half.y));
        }
        load_g(row + (size_t)(n + 1) * kT * stride, left - kT);  // the next chunk's
        ptx::fence_proxy_async_smem();
        ptx::tc_fence_before();
        __syncthreads();
        if (warp == 0) {
            ptx::tc_fence_after();
            const uint32_t q = desc(s.p1), kh = desc(s.p2), kl = desc(sm.kl), v = desc(s.v);
            if (kOut) {  // (a strong chunk's are not used)
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    ptx::mma_ss_elect(tmem + kColW, q + ks * kStepK, desc_high, kh + ks * kStepK, desc_high, kKK, ks > 0);
            }
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
                ptx::mma_ss_elect(tmem + kColC, v + (ks & 3) * kStepM, desc_high, (ks < 4 ? kh : kl) + (ks & 3) * kStepM,
                                  desc_high, kMM, ks > 0);
            if (third) {
                const uint32_t kz = desc(sm.w);
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    ptx::mma_ss_elect(tmem + kColC, v + ks * kStepM, desc_high, kz + ks * kStepM, desc_high, kMM, 1);
            }
            ptx::mma_commit_elect(&sm.c_done);
        }
        if (kOut) {
            // The state as an operand: 2^m C, and C itself in a strong chunk.
            uint32_t w[4][2];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const float2 f = *reinterpret_cast<const float2*>(&sm.c_half[col0 + 8 * x + 2 * t]);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float2 a = mul2(C[x][e], f);
                    w[x][e] = pack2(a.x, a.y);
                }
            }
            stsm4(ptx::smem_u32(sm.c) + frag_at, w[0][0], w[0][1], w[1][0], w[1][1]);
            stsm4(ptx::smem_u32(sm.c) + frag_next, w[2][0], w[2][1], w[3][0], w[3][1]);
        }
        wait(&sm.c_done, n);
        if (kOut) {
            // The weights, in a strong chunk there already.
            if (!strong) {
                uint32_t x[4][4];
                tmem_ld_frag(lane_addr + kColW, x);
                uint32_t w[4][2];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int first = col0 + 8 * c - 16 * quarter;  // key 0 of the block from the warp's first row
                    if (first > -8) {                               // strictly earlier keys only
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (first + 2 * t + (e & 1) >= g + 8 * (e >> 1)) x[c][e] = 0u;
                    }
                    w[c][0] = pack2(__uint_as_float(x[c][0]), __uint_as_float(x[c][1]));
                    w[c][1] = pack2(__uint_as_float(x[c][2]), __uint_as_float(x[c][3]));
                }
                stsm4(ptx::smem_u32(sm.w) + frag_at, w[0][0], w[0][1], w[1][0], w[1][1]);
                stsm4(ptx::smem_u32(sm.w) + frag_next, w[2][0], w[2][1], w[3][0], w[3][1]);
            }
            ptx::fence_proxy_async_smem();
            ptx::tc_fence_before();
            __syncthreads();
            if (warp == 0) {
                ptx::tc_fence_after();
                const uint32_t q = desc(s.p1), v = desc(s.v), w = desc(sm.w), c = desc(sm.c);
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    ptx::mma_ss_elect(tmem + kColO, q + ks * kStepK, desc_high, c + ks * kStepK, desc_high, kKK, ks > 0);
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    ptx::mma_ss_elect(tmem + kColO, w + ks * kStepK, desc_high, v + ks * kStepM, desc_high, kKM, 1);
                ptx::mma_commit_elect(&sm.o_done);
            }
        }
        // The state through the chunk.
        {
            uint32_t x[4][4];
            tmem_ld_frag(lane_addr + kColC, x);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float2 a = *reinterpret_cast<const float2*>(&sm.c_all[col0 + 8 * c + 2 * t]);
                const float2 f = *reinterpret_cast<const float2*>(&sm.c_half[col0 + 8 * c + 2 * t]);
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    C[c][e] = fma2(make_float2(__uint_as_float(x[c][2 * e]), __uint_as_float(x[c][2 * e + 1])), f,
                                   mul2(C[c][e], a));
            }
        }
        if (kOut) {
            uint32_t v[4][2];  // the tokens' own states, as fragments
            {
                uint32_t x[4];
                ldsm4(x, ptx::smem_u32(s.v) + frag_at);
                v[0][0] = x[0], v[0][1] = x[1], v[1][0] = x[2], v[1][1] = x[3];
                ldsm4(x, ptx::smem_u32(s.v) + frag_next);
                v[2][0] = x[0], v[2][1] = x[1], v[3][0] = x[2], v[3][1] = x[3];
            }
            wait(&sm.o_done, n);
            uint32_t x[4][4];
            tmem_ld_frag(lane_addr + kColO, x);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (r0 + 8 * e >= left || !ok) continue;
                __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.Y) + row + ((size_t)n * kT + r0 + 8 * e) * stride + col0 + 2 * t;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float2 o = add2(make_float2(lo_f(v[c][e]), hi_f(v[c][e])),
                                          make_float2(__uint_as_float(x[c][2 * e]), __uint_as_float(x[c][2 * e + 1])));
                    if (col0 + 8 * c + 2 * t < p.d) *reinterpret_cast<uint32_t*>(y + 8 * c) = pack2(o.x, o.y);
                }
            }
        }
        ptx::tc_fence_before();
        return kNext;
    };
    for (int n = 0; n < chunks && ok; ++n) {
        if (kOut) {
            if (chunk(n, std::false_type()) == kNext) continue;
            if (!ok) break;
            load_g(row + (size_t)n * kT * stride, it.count - n * kT);
        }
        chunk(n, std::true_type());
    }
    if (warp == 0 && *abort_flag) {  // let what is in flight end before its memory goes
        ptx::mma_commit_elect(&sm.drain);
        ptx::mbar_drain(&sm.drain, 0, p.status);
    }
    cp_async_wait<0>();
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, kTmemCols);
    }
    float* out = mine;
    int ld = kDp;
    if (kOut) {
        out = seg + 1 == segs ? state_of(p, __ldg(p.slots_out + it.r), h) : nullptr;
        ld = p.d;
    } else if (warp == 0) {
        *reinterpret_cast<float2*>(mine + kDp * kDp + c2) = lost;
    }
    if (out != nullptr) {
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int v = r0 + 8 * e, c = col0 + 8 * n + 2 * t;
                if (v < ld && c < ld) out[(size_t)c * ld + v] = C[n][e].x, out[(size_t)(c + 1) * ld + v] = C[n][e].y;
            }
    }
}

// Every segment's entering state in the place of its own contribution, from the pool's
// state on.  A thread has one entry, the next 16 segments' on their way: what it takes are the rounds of
// loads, not the bytes.
constexpr int kScanThreads = 128;
__global__ void __launch_bounds__(kScanThreads)
    linear_join_kernel(const __grid_constant__ LinearPool p, const __grid_constant__ Plan plan, float* __restrict__ segments) {
    dependency_wait();
    dependency_release();
    const int at = plan.joins[blockIdx.x];
    if (at < 0) return;
    const Item it = plan.items[at];
    const int segs = it.seg_segs >> 16, h = blockIdx.y;
    if (at + segs > plan.most_items) return;  // (never: make_items)
    const int e = blockIdx.z * kScanThreads + threadIdx.x, c = e >> 6, v = e & 63;
    const float* in = state_of(p, __ldg(p.slots_in + it.r), h);
    float C = in != nullptr && c < p.d && v < p.d ? in[(size_t)c * p.d + v] : 0.f;
    const size_t step = (size_t)p.H * kSegFloats;
    float* H = segments + ((size_t)at * p.H + h) * kSegFloats;
    constexpr int kAhead = 16;
    for (int s0 = 0; s0 < segs; s0 += kAhead) {
        float x[kAhead], a[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int s = s0 + k;
            const bool there = s + 1 < segs;  // the last one leaves none
            x[k] = there ? H[s * step + e] : 0.f;
            a[k] = there ? H[s * step + kDp * kDp + c] : 0.f;
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int s = s0 + k;
            if (s < segs) H[s * step + e] = C;
            C = fmaf(exp2f(a[k]), C, x[k]);
        }
    }
}

// The list of segments, their order, the list of joins.
size_t items_bytes(const Cut& c) {
    return ((size_t)c.items * (sizeof(Item) + sizeof(int)) + (size_t)c.joins * sizeof(int) + 255) / 256 * 256;
}

template <typename... P, typename... A>
cudaError_t launch(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, A... args) {
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

template <bool kGate>
cudaError_t launch_few(const LinearPool& p, const Plan& plan, cudaStream_t s) {
    const dim3 grid((unsigned)((int64_t)p.R * p.H + (plan.items != nullptr || plan.beside)));
    switch (p.d) {
        case 48: return launch(linear_few_kernel<48, kGate>, grid, kFewThreads, few_smem(p.max_fresh), s, p, plan);
        case 60: return launch(linear_few_kernel<60, kGate>, grid, kFewThreads, few_smem(p.max_fresh), s, p, plan);
        case 64: return launch(linear_few_kernel<64, kGate>, grid, kFewThreads, few_smem(p.max_fresh), s, p, plan);
    }
    return cudaErrorInvalidValue;
}

template <bool kGate>
cudaError_t launch_pool(const LinearPool& p, void* workspace, const Cut& cut, int* launches, cudaStream_t s) {
    Plan plan{};
    float* segments = nullptr;
    if (cut.segmented) {
        plan.items = static_cast<Item*>(workspace);
        plan.order = reinterpret_cast<int*>(plan.items + cut.items);
        plan.joins = plan.order + cut.items;
        plan.most_items = cut.items, plan.most_joins = cut.joins, plan.seg_tokens = cut.seg_tokens;
        segments = reinterpret_cast<float*>(static_cast<char*>(workspace) + items_bytes(cut));
    }
    cudaError_t e;
    if (!cut.chunked) {
        *launches = 1;
        return launch_few<kGate>(p, plan, s);
    }
    constexpr int smem = (int)sizeof(ChunkSmem) + 1024;
    static OncePerDevice once_out, once_state, split_out, split_state;
    if ((e = prefer_shared(split_out, linear_chunk_kernel<true, kGate>, kBlocksPerSm, smem)) != cudaSuccess) return e;
    if ((e = prefer_shared(split_state, linear_chunk_kernel<false, kGate>, kBlocksPerSm, smem)) != cudaSuccess) return e;
    if ((e = allow_dynamic_smem(once_out, linear_chunk_kernel<true, kGate>, smem)) != cudaSuccess) return e;
    if ((e = allow_dynamic_smem(once_state, linear_chunk_kernel<false, kGate>, smem)) != cudaSuccess) return e;
    const dim3 grid((unsigned)((int64_t)cut.items * p.H));
    if (!cut.segmented) {
        // The longer requests first, the others in the room beside them (60 single tokens and 4 chunks of 250 to 500,
        // 16 heads of 64: 40 us; the other way round 43).
        *launches = 2;
        plan.beside = true;
        e = launch(linear_chunk_kernel<true, kGate>, grid, kThreads, smem, s, p, plan, segments);
        return e != cudaSuccess ? e : launch_few<kGate>(p, plan, s);
    }
    *launches = 4;
    if ((e = launch_few<kGate>(p, plan, s)) != cudaSuccess) return e;
    if ((e = launch(linear_chunk_kernel<false, kGate>, grid, kThreads, smem, s, p, plan, segments)) != cudaSuccess) return e;
    e = launch(linear_join_kernel, dim3((unsigned)cut.joins, (unsigned)p.H, kDp * kDp / kScanThreads), kScanThreads, 0, s, p,
               plan, segments);
    if (e != cudaSuccess) return e;
    return launch(linear_chunk_kernel<true, kGate>, grid, kThreads, smem, s, p, plan, segments);
}

}  // namespace
}  // namespace lin

size_t linear_pool_workspace(int R, int N, int H, int max_fresh, int num_sms) {
    const lin::Cut c = lin::cut_of(R, N, H, max_fresh, num_sms);
    return c.segmented ? lin::items_bytes(c) + (size_t)c.items * H * lin::kSegFloats * sizeof(float) : 0;
}

cudaError_t launch_linear_pool(const LinearPool& p, void* workspace, int num_sms, int* launches, cudaStream_t s) {
    const lin::Cut c = lin::cut_of(p.R, p.N, p.H, p.max_fresh, num_sms);
    return p.A_log != nullptr ? lin::launch_pool<true>(p, workspace, c, launches, s)
                              : lin::launch_pool<false>(p, workspace, c, launches, s);
}

}  // namespace relation
