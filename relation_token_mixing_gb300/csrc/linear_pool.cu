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
// (linear_chunk_kernel).
//
// A chunk.  With q = S p^1, k = S p^2 and the running sum of the log-retentions
// G_t (from the chunk's start, in units of log2), the retention between tokens j
// and i is 2^(G_i - G_j), so with any reference m per channel
//     q~_i = q_i 2^(G_i - m),  k~_j = k_j 2^(m - G_j):
//     Y = I~ + strictly-lower(q~ k~^T) I~ + q~ (2^m C),
//     C <- 2^(G_end - m) (2^m C + k~^T I~)
// is the recurrence in four products of 64 x 64 x 64, all from the same two operands.
// m is the sum at the chunk's middle: half a chunk may then lose up to 2^kRange of
// a channel before a factor leaves the range of bf16.  A chunk that loses more in some
// channel takes another way to the same sums (strong_chunk below) whose factors
// are all retentions between two of its own tokens.
//
// Roundings: q~, the weights and the state as an operand of the output product are
// bf16, as the outputs are; k~ enters the state's product as a sum of two
// bf16 values (2^-17), since the state is kept in float32 from call to call; sums and the
// state itself are float32.
#include <cuda_bf16.h>
#include <stdint.h>

#include <algorithm>

#include "common.cuh"
#include "linear_common.cuh"
#include "linear_pool.h"
#include "once_per_device.h"
#include "ptx_sm100.cuh"
#include "tile_copy.cuh"

namespace relation {
namespace lin {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kFewTokens = 16;

__device__ __forceinline__ void dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void dependency_release() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// softplus to a relative 3e-7 (softplus_f is exact to 1e-7 absolute, which a float32 state of
// weak retention would show): log(1 + y) = 2 artanh(y / (2 + y)), y <= 1, by its Taylor series
// up to the 13th power of an argument of at most 1/3.
__device__ __forceinline__ float softplus_rel(float x) {
    const float y = __expf(-fabsf(x)), s = __fdividef(y, 2.f + y), z = s * s;
    float t = fmaf(z, 1.f / 13.f, 1.f / 11.f);
    t = fmaf(z, t, 1.f / 9.f);
    t = fmaf(z, t, 1.f / 7.f);
    t = fmaf(z, t, 1.f / 5.f);
    t = fmaf(z, t, 1.f / 3.f);
    t = fmaf(z, t, 1.f);
    return fmaf(2.f * s, t, fmaxf(x, 0.f));
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
// At least -280: 2^-280 of any float32 is 0, and sums of a chunk's terms keep their fractions.
template <bool kGate>
__device__ __forceinline__ float2 log2_retention(float2 x, const Gate& g) {
    const float2 e = kGate ? make_float2(g.na.x * softplus_rel(x.x + g.db.x), g.na.y * softplus_rel(x.y + g.db.y))
                           : make_float2(x.x * g.na.x, x.y * g.na.y);
    return make_float2(fmaxf(e.x, -280.f), fmaxf(e.y, -280.f));
}

// A request's tokens; ones that cannot be followed give count = -1 and are reported.
struct Span {
    int first, count;
};
__device__ __forceinline__ Span span_of(const LinearPool& p, int r) {
    if (p.starts == nullptr) return Span{r, 1};
    const int first = __ldg(p.starts + r);
    const int64_t n = (int64_t)__ldg(p.starts + r + 1) - first;
    if (first < 0 || n < 0 || first + n > p.N || n > p.max_fresh) {
        record_status(p.status, kDevBadPosition);
        return Span{0, -1};
    }
    return Span{first, (int)n};
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
constexpr int kMaxSegs = 1 << 15;

// ------------------------------------------------------------ the recurrence
// One block per request and head: thread (rg, cg) has rows rg + 8 i and columns 4 cg ..
// 4 cg + 3 of the state, in registers over all the request's tokens, so that the state
// is read and written once, 8 d d bytes, which bounds it.  The first kFewTokens tokens'
// vectors are made by the warps in turn while the state is on its way.
constexpr int kFewThreads = 128;

struct FewSmem {
    float a[kFewTokens][kDp], q[kFewTokens][kDp], k[kFewTokens][kDp], v[kFewTokens][kDp];
    float part[2][8][kDp];
};

// Block 0 of a packed call with items: the list of the longer requests' segments.
__device__ void make_items(const LinearPool& p, Item* items, int most, int seg_tokens) {
    __shared__ int sums[kFewThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int base = 0;
    for (int r0 = 0; r0 < p.R; r0 += kFewThreads) {
        const int r = r0 + tid;
        Span sp{0, 0};
        if (r < p.R) sp = span_of(p, r);
        const int segs = sp.count > kFewTokens ? (sp.count + seg_tokens - 1) / seg_tokens : 0;
        int x = segs;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) sums[warp] = x;
        __syncthreads();
        int at = base + x - segs;
        for (int w = 0; w < kFewThreads / 32; ++w) {
            if (w < warp) at += sums[w];
            base += sums[w];
        }
        for (int k = 0; k < segs && at + k < most; ++k)
            items[at + k] = Item{r, sp.first + k * seg_tokens, min(seg_tokens, sp.count - k * seg_tokens), k | segs << 16};
        __syncthreads();
    }
    for (int k = base + tid; k < most; k += kFewThreads) items[k] = Item{0, 0, 0, 0};
}

template <int D, bool kGate>
__global__ void __launch_bounds__(kFewThreads)
    linear_few_kernel(const __grid_constant__ LinearPool p, Item* items, int most_items, int seg_tokens) {
    __shared__ __align__(16) FewSmem sm;
    constexpr int kCols = D / 4, kRows = (D + 7) / 8;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    dependency_wait();
    dependency_release();
    int x = blockIdx.x;
    if (items != nullptr) {
        if (x == 0) {
            make_items(p, items, most_items, seg_tokens);
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
            *reinterpret_cast<float2*>(&sm.a[t][c]) = make_float2(exp2f(e.x), exp2f(e.y));
            *reinterpret_cast<float2*>(&sm.q[t][c]) = make_float2(lo_f(w1) * s1, hi_f(w1) * s1);
            *reinterpret_cast<float2*>(&sm.k[t][c]) = make_float2(lo_f(w2) * s2, hi_f(w2) * s2);
            *reinterpret_cast<float2*>(&sm.v[t][c]) = make_float2(lo_f(wv), hi_f(wv));
        }
    }
    __syncthreads();
    __nv_bfloat16* Y = static_cast<__nv_bfloat16*>(p.Y);
    for (int t = 0; t < sp.count; ++t) {
        if (active) {
            const float4 v = *reinterpret_cast<const float4*>(&sm.v[t][4 * cg]);
            float4 e = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                const int c = rg + 8 * i;
                if (c >= D) break;
                const float a = sm.a[t][c], q = sm.q[t][c], k = sm.k[t][c];
                C[i] = make_float4(C[i].x * a, C[i].y * a, C[i].z * a, C[i].w * a);
                e = make_float4(fmaf(q, C[i].x, e.x), fmaf(q, C[i].y, e.y), fmaf(q, C[i].z, e.z), fmaf(q, C[i].w, e.w));
                C[i] = make_float4(fmaf(k, v.x, C[i].x), fmaf(k, v.y, C[i].y), fmaf(k, v.z, C[i].z),
                                   fmaf(k, v.w, C[i].w));
            }
            *reinterpret_cast<float4*>(&sm.part[t & 1][rg][4 * cg]) = e;
        }
        __syncthreads();  // the other buffer's readers are a token behind: past the next barrier
        if (tid < D / 2) {
            float2 y = *reinterpret_cast<const float2*>(&sm.v[t][2 * tid]);
#pragma unroll
            for (int g = 0; g < 8; ++g) {
                const float2 e = *reinterpret_cast<const float2*>(&sm.part[t & 1][g][2 * tid]);
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
constexpr int kT = 64;            // tokens of a chunk
constexpr int kThreads = 256;
constexpr float kRange = 100.f;   // log2 of what half a chunk may lose of a channel
constexpr int kTile = kT * 128;   // a bf16 tile of 64 x 64
constexpr int kSegFloats = kDp * kDp + kDp;  // of a segment in the workspace: its state, the log2 of its retention

struct ChunkStage {
    uint8_t p1[kTile];  // q~ in place of p1, the larger part of k~ in place of p2, once they are made
    uint8_t p2[kTile];
    uint8_t v[kTile];
    float g[kT * kDp];
};
struct ChunkSmem {
    ChunkStage st[2];
    uint8_t kl[kTile];    // what bf16 leaves of k~
    uint8_t c[kTile];     // the state as an operand, [value channel][key channel]
    float tot[8][kDp];    // a warp's 8 tokens: sum of log2 of their retentions
    float c_op[kDp], c_pre[kDp];  // per channel: the state's factor as an operand and before the update
    float2 rs[kT];        // (S / |p1|, S / |p2|) of a token
};

// The rows of a stretch of `count` tokens, 64 at a time: a thread's sources go on from chunk to
// chunk.  Rows past the end are zero, as the columns past d stay.
struct Loader {
    const char *p1, *p2, *v, *g;
    size_t half;    // bytes from a row to the thread's next one
    size_t g_step;
    size_t chunk;   // and from a chunk to the next
    int row, g_row, col, g_col;
    uint32_t dst, g_dst;

    __device__ __forceinline__ Loader(const LinearPool& p, size_t first) {
        const int tid = threadIdx.x;
        const bool wide = (p.d & 7) == 0;  // else rows of 120 bytes, which start on 8
        const size_t stride = (size_t)p.H * p.d;
        row = wide ? tid >> 3 : tid >> 4;
        col = wide ? 8 * (tid & 7) : 4 * (tid & 15);
        g_row = tid >> 4, g_col = 4 * (tid & 15);
        const size_t at = (first + row * stride + col) * 2;
        p1 = static_cast<const char*>(p.P1) + at;
        p2 = static_cast<const char*>(p.P2) + at;
        v = static_cast<const char*>(p.I) + at;
        g = reinterpret_cast<const char*>(p.G) + (first + g_row * stride + g_col) * 4;
        half = stride * 2 * (wide ? 32 : 16);
        g_step = stride * 4 * 16;
        chunk = stride * 2 * kT;
        dst = swz(row, col);
        g_dst = (g_row * kDp + g_col) * 4;
    }
    // left: tokens from this chunk on.
    __device__ __forceinline__ void chunk_into(ChunkStage& s, int d, int left) {
        const char* src[3] = {p1, p2, v};
        const uint32_t to[3] = {ptx::smem_u32(s.p1) + dst, ptx::smem_u32(s.p2) + dst, ptx::smem_u32(s.v) + dst};
        if (col < d) {
            if ((d & 7) == 0) {
#pragma unroll
                for (int k = 0; k < 3; ++k)
#pragma unroll
                    for (int r = 0; r < 2; ++r)
                        if (row + 32 * r < left) cp_async_16(to[k] + r * 32 * 128, src[k] + r * half);
                        else st_zero16(to[k] + r * 32 * 128);
            } else {
#pragma unroll
                for (int k = 0; k < 3; ++k)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (row + 16 * r < left) cp_async_8(to[k] + r * 16 * 128, src[k] + r * half);
                        else st_shared_zero8(to[k] + r * 16 * 128);
            }
        }
        if (g_col < d)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const uint32_t at = ptx::smem_u32(s.g) + g_dst + r * 16 * kDp * 4;
                if (g_row + 16 * r < left) cp_async_16(at, g + r * g_step);
                else st_zero16(at);
            }
        cp_async_commit();
        p1 += chunk, p2 += chunk, v += chunk, g += 2 * chunk;
    }
};

__device__ __forceinline__ float2 add2(float2 a, float2 b) { return ptx::add2(a, b); }

// The warp's 8 tokens: |p1|^2, |p2|^2 and p1 . p2 are the diagonals of three 8 x 8 products of the rows with
// one another (a row's fragment is the same on both sides), then S / |p1| and S / |p2|.  Twelve products and
// four fetches in place of some 150 multiply-adds and shuffles.
__device__ __forceinline__ void row_scalars(ChunkSmem& sm, const ChunkStage& s, float zscale, int warp, int lane) {
    float n1[4] = {}, n2[4] = {}, dt[4] = {};
    const uint32_t at = 8 * warp * 128 + swz(lane & 7, 8 * (lane >> 3)), at2 = 8 * warp * 128 + swz(lane & 7, 32 + 8 * (lane >> 3));
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        uint32_t x[4], y[4];
        ldsm4(x, ptx::smem_u32(s.p1) + (k ? at2 : at));
        ldsm4(y, ptx::smem_u32(s.p2) + (k ? at2 : at));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t ax[4] = {x[2 * h], 0u, x[2 * h + 1], 0u}, ay[4] = {y[2 * h], 0u, y[2 * h + 1], 0u};
            mma16816(n1, ax, x[2 * h], x[2 * h + 1]);
            mma16816(dt, ax, y[2 * h], y[2 * h + 1]);
            mma16816(n2, ay, y[2 * h], y[2 * h + 1]);
        }
    }
    const int g = lane >> 2;
    if ((lane & 3) == g >> 1) {  // the diagonal's entry of row g
        const float a = g & 1 ? n1[1] : n1[0], b = g & 1 ? n2[1] : n2[0], x = g & 1 ? dt[1] : dt[0];
        const float S = 1.f / (1.f + __expf(-x * zscale));
        sm.rs[8 * warp + g] = make_float2(a > 0.f ? S * rsqrtf(a) : 0.f, b > 0.f ? S * rsqrtf(b) : 0.f);
    }
    __syncwarp();
}

// Entries (16 rt + lane / 4 (+ 8), 8 n + 2 (lane % 4) (+ 1)) of q k^T with the retention between
// the two tokens, n < 2 rt + 2, for a chunk whose factors from one reference would leave
// bf16's range: s.g holds G, s.p1 and s.p2 the rows as they came.  Keys before the 16 tokens
// meet the queries at the block's first token, the block's first 8 keys its last 8 queries at the ninth:
// all factors are retentions.  What is left are pairs inside 8 tokens, one by one.
__device__ __noinline__ void strong_chunk(float (&w)[8][4], const ChunkSmem& sm, const ChunkStage& s, int rt, int lane) {
    const int g = lane >> 2, t = lane & 3;
    const auto row_of = [](const uint8_t* tile, int r, int c) { return *reinterpret_cast<const uint32_t*>(tile + swz(r, c)); };
    // q (or k) of row r, columns c and c + 1, times 2^(+-(G_r - G_b)) as a bf16 pair; b < 0: from the chunk's start.
    const auto scaled = [&](bool query, int r, int b, int c) {
        const float2 G = *reinterpret_cast<const float2*>(s.g + r * kDp + c);
        const float2 B = b < 0 ? make_float2(0.f, 0.f) : *reinterpret_cast<const float2*>(s.g + b * kDp + c);
        const uint32_t x = row_of(query ? s.p1 : s.p2, r, c);
        const float f = query ? sm.rs[r].x : sm.rs[r].y;
        const float2 e = query ? make_float2(G.x - B.x, G.y - B.y) : make_float2(B.x - G.x, B.y - G.y);
        return pack2(lo_f(x) * f * ptx::ex2_approx(e.x), hi_f(x) * f * ptx::ex2_approx(e.y));
    };
    const int i0 = 16 * rt + g;
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) w[n][e] = 0.f;
#pragma unroll 1
    for (int c0 = 0; c0 < kDp; c0 += 16) {
        const int c = c0 + 2 * t;
        uint32_t a[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) a[x] = scaled(true, i0 + 8 * (x & 1), 16 * rt - 1, c + 8 * (x >> 1));
#pragma unroll
        for (int n = 0; n < 6; ++n)
            if (n < 2 * rt) mma16816(w[n], a, scaled(false, 8 * n + g, 16 * rt - 1, c), scaled(false, 8 * n + g, 16 * rt - 1, c + 8));
        a[0] = a[2] = 0u;
        a[1] = scaled(true, i0 + 8, 16 * rt + 7, c);
        a[3] = scaled(true, i0 + 8, 16 * rt + 7, c + 8);
        const uint32_t b0 = scaled(false, i0, 16 * rt + 7, c), b1 = scaled(false, i0, 16 * rt + 7, c + 8);
#pragma unroll
        for (int n = 0; n < 8; n += 2)
            if (n == 2 * rt) mma16816(w[n], a, b0, b1);
    }
    // Rows lane / 4 against columns 2 (lane % 4) of the two triangles on the diagonal.
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
        const int base = 16 * rt + 8 * half, i = base + g, j = base + 2 * t;
        float x0 = 0.f, x1 = 0.f;
#pragma unroll 1
        for (int c = 0; c < kDp; c += 2) {
            const float2 Gi = *reinterpret_cast<const float2*>(s.g + i * kDp + c);
            const float2 Gj = *reinterpret_cast<const float2*>(s.g + j * kDp + c);
            const float2 Gk = *reinterpret_cast<const float2*>(s.g + (j + 1) * kDp + c);
            const uint32_t q = row_of(s.p1, i, c), k0 = row_of(s.p2, j, c), k1 = row_of(s.p2, j + 1, c);
            if (j < i)
                x0 += lo_f(q) * lo_f(k0) * ptx::ex2_approx(Gi.x - Gj.x) + hi_f(q) * hi_f(k0) * ptx::ex2_approx(Gi.y - Gj.y);
            if (j + 1 < i)
                x1 += lo_f(q) * lo_f(k1) * ptx::ex2_approx(Gi.x - Gk.x) + hi_f(q) * hi_f(k1) * ptx::ex2_approx(Gi.y - Gk.y);
        }
        x0 *= sm.rs[i].x * sm.rs[j].y;
        x1 *= sm.rs[i].x * sm.rs[j + 1].y;
#pragma unroll
        for (int n = 0; n < 8; ++n)
            if (n == 2 * rt + half) w[n][2 * half] = x0, w[n][2 * half + 1] = x1;
    }
}

// One block a segment of a request and head: the output pass (kOut) from the state that
// enters it, or the state pass, which leaves the segment's own contribution and retention.
// Warps 0-3 have the query rows 16 w and value channels 0-31, warps 4-7 the rows
// 16 (7 - w), so that a scheduler's two warps have five of the eight triangle's parts, and
// channels 32-63; of the state C^T, warp w has rows (value channels) 16 (w % 4) and columns (key
// channels) 32 (w / 4), as accumulators, from chunk to chunk.
template <bool kOut, bool kGate>
__global__ void __launch_bounds__(kThreads, 2)
    linear_chunk_kernel(const __grid_constant__ LinearPool p, const Item* __restrict__ items, float* __restrict__ segments) {
    extern __shared__ __align__(128) uint8_t smem_raw[];
    ChunkSmem& sm = *reinterpret_cast<ChunkSmem*>(smem_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, h = blockIdx.y;
    for (int k = tid; k < (int)(sizeof(sm.st) / 16); k += kThreads)
        reinterpret_cast<uint4*>(sm.st)[k] = make_uint4(0, 0, 0, 0);
    // The kernel before waited for what ran before it, and leaves the items.
    if (items != nullptr) dependency_wait();
    dependency_release();
    Item it{(int)blockIdx.x, 0, 0, 1 << 16};
    if (items != nullptr) {
        it = items[blockIdx.x];
    } else {
        const Span sp = span_of(p, it.r);
        it.first = sp.first, it.count = sp.count;
    }
    const int seg = it.seg_segs & 0xffff, segs = it.seg_segs >> 16;
    const bool none = segs == 0 || it.count <= (segs > 1 ? 0 : kFewTokens) || (!kOut && seg + 1 >= segs);
    if (none) {
        if (items == nullptr && tid == 0) dependency_wait();
        return;
    }
    const size_t row = ((size_t)it.first * p.H + h) * p.d;
    const int chunks = (it.count + kT - 1) / kT;
    __syncthreads();
    Loader load(p, row);
    load.chunk_into(sm.st[0], p.d, it.count);

    // The state C^T.
    const int g = lane >> 2, t = lane & 3, vt = 16 * (warp & 3), ct = 32 * (warp >> 2);
    float C[4][4];
    float* mine = segments == nullptr ? nullptr : segments + ((size_t)blockIdx.x * p.H + h) * kSegFloats;
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
            for (int e = 0; e < 4; ++e) {
                const int v = vt + g + 8 * (e >> 1), c = ct + 8 * n + 2 * t + (e & 1);
                C[n][e] = in != nullptr && v < ld && c < ld ? in[(size_t)c * ld + v] : 0.f;
            }
    }
    const int rt = warp < 4 ? warp : 7 - warp, v0 = 32 * (warp >> 2);
    const int c2 = 2 * lane;
    const uint32_t own = 8 * warp * 128 + ((c2 & 7) << 1);  // the lane's channels in its tokens' rows, see `at`
    const Gate gate = gate_of<kGate>(p, h, c2);
    const size_t ystride = (size_t)p.H * p.d;
    __nv_bfloat16* Y = static_cast<__nv_bfloat16*>(p.Y) + row + (16 * rt + g) * ystride + v0 + 2 * t;
    float2 lost = make_float2(0.f, 0.f);  // log2 of the segment's retention
    // The accumulators hold the state over 2^owed (per channel): the factor after a chunk's update and the one before
    // the next are applied as one.
    float2 owed = make_float2(0.f, 0.f);
    for (int n = 0; n < chunks; ++n) {
        ChunkStage& s = sm.st[n & 1];
        const int left = it.count - n * kT;  // tokens from this chunk on
        cp_async_wait<0>();
        __syncthreads();  // the chunk is there, and nothing reads the one before any more
        if (n + 1 < chunks) load.chunk_into(sm.st[(n + 1) & 1], p.d, left - kT);
        row_scalars(sm, s, p.zscale, warp, lane);
        // G inside the warp's 8 tokens.
        float2 G[8], sum = make_float2(0.f, 0.f);
        float most = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float2 e = log2_retention<kGate>(*reinterpret_cast<const float2*>(s.g + (8 * warp + i) * kDp + c2), gate);
            if (kGate && 8 * warp + i >= left) e = make_float2(0.f, 0.f);  // (else the row is zero)
            if (!kGate) most = ptx::max3(most, e.x, e.y);
            sum = add2(sum, e);
            G[i] = sum;
        }
        *reinterpret_cast<float2*>(&sm.tot[warp][c2]) = sum;
        // A state that grows may do so at one token and fade at others: the sums of half a chunk say nothing then.
        const bool grows = kGate ? (__syncthreads(), false) : __syncthreads_or(most > 0.f);
        float2 base = make_float2(0.f, 0.f), mid = base, rest = base;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            const float2 x = *reinterpret_cast<const float2*>(&sm.tot[w][c2]);
            if (w == warp) base = add2(mid, rest);
            if (w < 4) mid = add2(mid, x);
            else rest = add2(rest, x);
        }
        const float2 all = add2(mid, rest);
        lost = add2(lost, all);
        const float least = fminf(fminf(mid.x, mid.y), fminf(rest.x, rest.y));
        const bool strong = grows || __any_sync(0xffffffffu, !(least >= -kRange));  // the same for every warp
        float w[8][4];
        if (strong) {
            if (kOut) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    *reinterpret_cast<float2*>(s.g + (8 * warp + i) * kDp + c2) = add2(base, G[i]);
                __syncthreads();
                float there[8][4];
                strong_chunk(there, sm, s, rt, lane);
#pragma unroll
                for (int x = 0; x < 8; ++x)
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[x][e] = there[x][e];
                __syncthreads();  // before the rows are overwritten
            }
        }
        // The operands, in the rows' places: a warp's own tokens, a lane's own channels.  Exponents: of a query
        // G - mid and of a key its negative; in a strong chunk from the chunk's start, and to its end.
        const float2 from = strong ? base : make_float2(base.x - mid.x, base.y - mid.y);
        float2 to_end = sum;
        if (strong)
#pragma unroll
            for (int x = 0; x < 8; ++x)
                if (x > warp) to_end = add2(to_end, *reinterpret_cast<const float2*>(&sm.tot[x][c2]));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t at = own + i * 128 + (((lane >> 2) ^ i) << 4);  // swz(8 warp + i, c2)
            const float2 f = sm.rs[8 * warp + i], eq = add2(from, G[i]);
            const float2 ek = strong ? make_float2(to_end.x - G[i].x, to_end.y - G[i].y) : make_float2(-eq.x, -eq.y);
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
            *reinterpret_cast<uint32_t*>(sm.kl + at) = pack2(lo.x, lo.y);
        }
        // What is owed goes with 2^mid, or before it: always in a strong chunk, and where both together would be
        // too small for a float32 factor, though the accumulators, which hold 2^-owed times the state, are not.
        const float2 both = add2(owed, mid);
        const bool apart = strong || __any_sync(0xffffffffu, !(fminf(both.x, both.y) >= -120.f));
        if (warp == 0) {
            const float2 to = strong ? all : apart ? mid : both;
            *reinterpret_cast<float2*>(&sm.c_pre[c2]) = make_float2(ptx::ex2_approx(to.x), ptx::ex2_approx(to.y));
            *reinterpret_cast<float2*>(&sm.c_op[c2]) = make_float2(ptx::ex2_approx(owed.x), ptx::ex2_approx(owed.y));
        }
        owed = strong ? make_float2(0.f, 0.f) : rest;
        __syncthreads();
        // The state as the output's operand (2^mid C; of a strong chunk C) and as the update finds it (the same; all's
        // retention applied).
        const uint32_t c_row = (vt + g) * 128;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int c = ct + 8 * x + 2 * t;
            const uint32_t at = c_row + ((((c >> 3) ^ g) & 7) << 4) + 4 * t;  // rows vt + g and 8 further
            float2 lo = make_float2(C[x][0], C[x][1]), hi = make_float2(C[x][2], C[x][3]);
            if (apart) {
                const float2 f = *reinterpret_cast<const float2*>(&sm.c_op[c]);
                lo = mul2(lo, f), hi = mul2(hi, f);
                if (kOut && strong) {
                    *reinterpret_cast<uint32_t*>(sm.c + at) = pack2(lo.x, lo.y);
                    *reinterpret_cast<uint32_t*>(sm.c + at + 8 * 128) = pack2(hi.x, hi.y);
                }
            }
            const float2 f = *reinterpret_cast<const float2*>(&sm.c_pre[c]);
            lo = mul2(lo, f), hi = mul2(hi, f);
            C[x][0] = lo.x, C[x][1] = lo.y, C[x][2] = hi.x, C[x][3] = hi.y;
            if (kOut && !strong) {
                *reinterpret_cast<uint32_t*>(sm.c + at) = pack2(lo.x, lo.y);
                *reinterpret_cast<uint32_t*>(sm.c + at + 8 * 128) = pack2(hi.x, hi.y);
            }
        }
        if (kOut) {
            uint32_t aq[4][4];
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) ldsm4(aq[ks], addr_a(s.p1 + rt * 16 * 128, 16 * ks, lane));
            float E[4][4];
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int e = 0; e < 4; ++e) E[x][e] = 0.f;
#pragma unroll
            for (int kb = 0; kb < 4; ++kb) {
                if (kb > rt) break;
                if (!strong) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[2 * kb][e] = w[2 * kb + 1][e] = 0.f;
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) {
                        uint32_t b[4];  // (keys 0-7, k 0-7), (0-7, 8-15), (8-15, 0-7), (8-15, 8-15)
                        ldsm4(b, addr_at(s.p2 + kb * 16 * 128, 16 * ks, lane));
                        mma16816(w[2 * kb], aq[ks], b[0], b[1]);
                        mma16816(w[2 * kb + 1], aq[ks], b[2], b[3]);
                    }
                }
                if (kb == rt) {  // strictly earlier keys only
#pragma unroll
                    for (int y = 0; y < 2; ++y)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (8 * y + 2 * t + (e & 1) >= g + 8 * (e >> 1)) w[2 * kb + y][e] = 0.f;
                }
                const uint32_t a[4] = {pack2(w[2 * kb][0], w[2 * kb][1]), pack2(w[2 * kb][2], w[2 * kb][3]),
                                       pack2(w[2 * kb + 1][0], w[2 * kb + 1][1]), pack2(w[2 * kb + 1][2], w[2 * kb + 1][3])};
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    uint32_t b[4];
                    ldsm4t(b, addr_bt(s.v + kb * 16 * 128, v0 + 16 * x, lane));
                    mma16816(E[2 * x], a, b[0], b[1]);
                    mma16816(E[2 * x + 1], a, b[2], b[3]);
                }
            }
            __syncthreads();  // the state's operand is there
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    uint32_t b[4];
                    ldsm4(b, addr_at(sm.c + (v0 + 16 * x) * 128, 16 * ks, lane));
                    mma16816(E[2 * x], aq[ks], b[0], b[1]);
                    mma16816(E[2 * x + 1], aq[ks], b[2], b[3]);
                }
            const uint32_t v_at = (16 * rt + g) * 128 + 4 * t;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                if (16 * rt + g + 8 * half >= left) continue;
                __nv_bfloat16* y = Y + 8 * half * ystride;
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    if (v0 + 8 * x + 2 * t >= p.d) continue;
                    const uint32_t i = *reinterpret_cast<const uint32_t*>(
                        s.v + v_at + 8 * half * 128 + ((((v0 >> 3) + x) ^ g) << 4));  // swz(16 rt + g + 8 half, v)
                    const float2 o = add2(make_float2(lo_f(i), hi_f(i)), make_float2(E[x][2 * half], E[x][2 * half + 1]));
                    *reinterpret_cast<uint32_t*>(y + 8 * x) = pack2(o.x, o.y);
                }
            }
            Y += kT * ystride;
        }
        // C^T += I~^T k~.
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            uint32_t a[4];
            ldsm4t(a, addr_at(s.v + ks * 16 * 128, vt, lane));
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                uint32_t b[4];
                ldsm4t(b, addr_bt(s.p2 + ks * 16 * 128, ct + 16 * x, lane));
                mma16816(C[2 * x], a, b[0], b[1]);
                mma16816(C[2 * x + 1], a, b[2], b[3]);
                ldsm4t(b, addr_bt(sm.kl + ks * 16 * 128, ct + 16 * x, lane));
                mma16816(C[2 * x], a, b[0], b[1]);
                mma16816(C[2 * x + 1], a, b[2], b[3]);
            }
        }
    }
    if (warp == 0) *reinterpret_cast<float2*>(&sm.c_op[c2]) = make_float2(ptx::ex2_approx(owed.x), ptx::ex2_approx(owed.y));
    __syncthreads();
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
        for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int v = vt + g + 8 * (e >> 1), c = ct + 8 * x + 2 * t + (e & 1);
                if (v < ld && c < ld) out[(size_t)c * ld + v] = C[x][e] * sm.c_op[c];
            }
    }
    // (few calls: the whole chain ends with this kernel's end)
    if (items == nullptr && tid == 0) dependency_wait();
}

// Every segment's entering state in the place of its own contribution, from the pool's
// state on.  A thread has one entry, the next 16 segments' on their way: what it takes are the rounds of
// loads, not the bytes.
constexpr int kScanThreads = 128;
__global__ void __launch_bounds__(kScanThreads)
    linear_join_kernel(const __grid_constant__ LinearPool p, const Item* __restrict__ items, float* __restrict__ segments) {
    dependency_wait();
    dependency_release();
    const Item it = items[blockIdx.x];
    const int seg = it.seg_segs & 0xffff, segs = it.seg_segs >> 16, h = blockIdx.y;
    if (seg != 0 || segs < 2) return;
    const int e = blockIdx.z * kScanThreads + threadIdx.x, c = e >> 6, v = e & 63;
    const float* in = state_of(p, __ldg(p.slots_in + it.r), h);
    float C = in != nullptr && c < p.d && v < p.d ? in[(size_t)c * p.d + v] : 0.f;
    const size_t step = (size_t)p.H * kSegFloats;
    float* H = segments + ((size_t)blockIdx.x * p.H + h) * kSegFloats;
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

// How a packed call is cut: requests longer than `seg_tokens` in segments of that many.
struct Cut {
    bool chunked;     // a request may have more than kFewTokens new tokens
    bool segmented;   // and more than seg_tokens
    int seg_tokens, items;
};
Cut cut_of(int R, int N, int H, int max_fresh, int num_sms) {
    Cut c{};
    c.chunked = max_fresh > kFewTokens;
    if (!c.chunked) return c;
    // A segment as long as a block's equal share of all tokens, 256 at least: shorter ones cost more
    // in the state pass and the join than they spread.
    const int64_t share = ((int64_t)N * H / (2 * num_sms) + kT - 1) / kT * kT;
    int64_t seg = std::max<int64_t>(256, share);
    seg = std::max<int64_t>(seg, ((int64_t)max_fresh / (kMaxSegs - 1) + kT) / kT * kT);
    c.seg_tokens = (int)std::min<int64_t>(seg, (INT32_MAX - kT) / kT * kT);
    c.segmented = max_fresh > c.seg_tokens;
    c.items = c.segmented ? (int)std::min<int64_t>((int64_t)N / c.seg_tokens + std::min(R, N / (kFewTokens + 1)), INT32_MAX) : R;
    return c;
}
size_t items_bytes(const Cut& c) { return ((size_t)c.items * sizeof(Item) + 255) / 256 * 256; }

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
cudaError_t launch_few(const LinearPool& p, Item* items, const Cut& cut, cudaStream_t s) {
    const dim3 grid((unsigned)((int64_t)p.R * p.H + (items != nullptr)));
    switch (p.d) {
        case 48: return launch(linear_few_kernel<48, kGate>, grid, kFewThreads, 0, s, p, items, cut.items, cut.seg_tokens);
        case 60: return launch(linear_few_kernel<60, kGate>, grid, kFewThreads, 0, s, p, items, cut.items, cut.seg_tokens);
        case 64: return launch(linear_few_kernel<64, kGate>, grid, kFewThreads, 0, s, p, items, cut.items, cut.seg_tokens);
    }
    return cudaErrorInvalidValue;
}

template <bool kGate>
cudaError_t launch_pool(const LinearPool& p, void* workspace, const Cut& cut, int* launches, cudaStream_t s) {
    Item* items = cut.segmented ? static_cast<Item*>(workspace) : nullptr;
    float* segments = cut.segmented ? reinterpret_cast<float*>(static_cast<char*>(workspace) + items_bytes(cut)) : nullptr;
    cudaError_t e = launch_few<kGate>(p, items, cut, s);
    *launches = 1;
    if (e != cudaSuccess || !cut.chunked) return e;
    constexpr int smem = (int)sizeof(ChunkSmem);
    static OncePerDevice once_out, once_state;
    if ((e = allow_dynamic_smem(once_out, linear_chunk_kernel<true, kGate>, smem)) != cudaSuccess) return e;
    if ((e = allow_dynamic_smem(once_state, linear_chunk_kernel<false, kGate>, smem)) != cudaSuccess) return e;
    const dim3 grid((unsigned)cut.items, (unsigned)p.H);
    if (cut.segmented) {
        *launches = 4;
        e = launch(linear_chunk_kernel<false, kGate>, grid, kThreads, smem, s, p, items, segments);
        if (e != cudaSuccess) return e;
        e = launch(linear_join_kernel, dim3(grid.x, grid.y, kDp * kDp / kScanThreads), kScanThreads, 0, s, p, items,
                   segments);
        if (e != cudaSuccess) return e;
    } else {
        *launches = 2;
    }
    return launch(linear_chunk_kernel<true, kGate>, grid, kThreads, smem, s, p, items, segments);
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
