// Relation of new tokens over a paged cache in float32 on the CUDA cores ("Ask
// Self, Ask Others", Sec. 3.1 eq.(1)-(3), Sec. 5.3 eq.(18), Appendix A.5), for any
// number of new tokens: U_j = p1 . p2_j / sqrt(d), R_j = SiLU(U_j) for j < i, R_i =
// sigmoid(U_i / tau_S) + lambda log(i + 1), Y = softmax(R) I~.
//
// Thread (ty, tx), tx of 8, owns kPer rows (row = token * group + head in the group), the
// keys tx + 8 n of a tile of 64, and four columns in every 32 of the output.  Both products use
// the packed fp32 multiply-add with a key's value for both halves: of two rows in the scores
// (the queries are held column by column), of two columns in the output.  With pairs of
// columns in the scores too, the operand that is not shared is read anew each time, and that
// product took twice the output's time.  P2 of the next tile is copied while the weights are
// applied, I~ while the scores are formed, so one buffer of each and two barriers a tile are
// enough.  Two shapes: kPer = 4 (64 rows, three
// blocks an SM; 128 columns: 128 rows and one), bound by the fp32 pipes, and kPer = 1 for
// requests of at most 16 rows, whose time is mostly the copies'.  Measured at 4 requests of
// 100 to 500 new tokens over up to 2048, 16 heads over 8 of 64: 0.192 ms, 0.41 of the fp32 pipes
// (a 16 x 16 grid of threads with pairs of columns 0.218; this grid with them 0.200; two
// blocks an SM and more in flight a warp 0.22); 16 decoding requests of 100 to 16384, 16 heads
// over 8 of 64: 0.165 ms, 3.1 TB/s (warps without a row of the unit skip the products: 0.29 if
// they do not).  Work is cut as in the bf16 kernels
// (paged_schedule.cuh).
//
// Exponentials use ex2 and the sigmoid's quotient a reciprocal, both within 2^-22;
// the argument's own rounding (|R| 2^-24) is of that size.
#include <algorithm>

#include "once_per_device.h"
#include "paged_fwd.cuh"

namespace relation {
namespace paged {
namespace {

constexpr int kKeys = 64, kTx = 8;
constexpr int kSmallRows = 16;  // requests of at most this many rows take kPer = 1
constexpr int kMinTiles = 2;  // of a worker (kPer = 1: 1, the tile's latency is the time)
constexpr int kLong = 4;      // and longer ones this kPer
constexpr int kPitchP = 68;  // rows start on 16 bytes; four rows on are 16 banks on

// kQuads: quads of 8 threads across the output (64, 96 or 128 wide).
template <int kQuads, int kPer>
struct F32Cfg {
    static constexpr int kWidth = 32 * kQuads;
    // 128 wide, one block fills an SM's shared memory: it has twice the threads and rows.
    static constexpr int kTy = kPer > 1 && kQuads == 4 ? 32 : 16, kThreads = kTy * kTx;
    static constexpr int kRows = kTy * kPer;
    static constexpr int kPitch = kWidth + 4;  // 4 (mod 32): eight rows' 16-byte reads cover the banks
    // Queries: rows, or (kPer > 1) columns of the rows.
    static constexpr int kPitchQ = kPer > 1 ? kRows + 4 : kPitch, kQ = kPer > 1 ? kWidth * kPitchQ : kRows * kPitch;
    static constexpr int kFloats = kQ + kKeys * kPitch + kKeys * kWidth + kRows * kPitchP;
    static int smem(int R) { return kFloats * 4 + 64 + (R * 4 + 15) / 16 * 16; }
    // Blocks an SM holds (kPer = 1: of 3, 4 and 5, three were fastest), by registers and by shared memory (the schedule's summary of R
    // requests takes little unless R is thousands).
    static constexpr int kPerSm =
        std::max(1, std::min(kPer == 1 || kQuads == 2 ? 3 : 2, 222 * 1024 / (kFloats * 4 + 2048)));
    using Line = Tiling<kRows, kKeys, 1>;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ float sigmoid_f32(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(1.f + ptx::ex2_approx(-kLog2e * x)));
    return y;
}

template <int kQuads, int kPer>
__global__ void __launch_bounds__(F32Cfg<kQuads, kPer>::kThreads, F32Cfg<kQuads, kPer>::kPerSm)
    paged_f32_kernel(const __grid_constant__ FwdView v, const float* __restrict__ P1, const float* __restrict__ P2,
                     const float* __restrict__ I, float* __restrict__ Y, float* __restrict__ L,
                     float* __restrict__ part, PieceMeta* __restrict__ meta) {
    using C = F32Cfg<kQuads, kPer>;
    using Tl = typename C::Line;
    constexpr int kRows = C::kRows, kThreads = C::kThreads;
    extern __shared__ float4 smem4[];
    float* sQ = reinterpret_cast<float*>(smem4);
    float* sK = sQ + C::kQ;
    float* sV = sK + kKeys * C::kPitch;
    float* sP = sV + kKeys * C::kWidth;
    int64_t* sums = reinterpret_cast<int64_t*>(sP + kRows * kPitchP);
    int* prefix = reinterpret_cast<int*>(sums + 8);
    const PagedProblem& pp = v.pp;
    const int tid = threadIdx.x, tx = tid % kTx, ty = tid / kTx;
    // The short requests' pass is first and waits for the inputs; the other's end waits for it.
    if (kPer == 1) dependency_wait();
    dependency_release();
    const int total = schedule_build(v, prefix, sums, [&](const Request& q) {
        return Tl::places(q.c, q.rows, pp.by_group, Tl::row_tiles(q.rows));
    });
    const int worker = blockIdx.x;
    const Share share(total, (int)gridDim.x, kPer == 1 ? 1 : kMinTiles);
    const int lo = share.begin(worker), hi = share.begin(worker + 1);
    PieceMeta mine{};
    if (lo >= hi) {
        if (tid == 0) {
            meta[worker] = mine;
            dependency_wait();
        }
        return;
    }
    Cursor k;
    cursor_seek<Tl>(k, v, prefix, lo);
    const int quads = pp.d / 4;
    const float inv_diag = pp.inv_sqrt_d / pp.tau_S;
    const uint32_t k_u = ptx::smem_u32(sK), v_u = ptx::smem_u32(sV);
    // Key tile j of the unit in hand, a few threads a row.  The page is asked for a tile ahead.
    // Keys past the end are zero (whatever their page holds), as are those of a page outside
    // the pool.
    constexpr int kPerRow = kThreads / kKeys;
    const int key = tid / kPerRow;
    auto page_of = [&](int j, int len) {
        const int tok = j * kKeys + key;
        return tok < len ? __ldg(v.table + (size_t)k.r * pp.width + (tok >> pp.page_shift)) : -1;
    };
    auto copy = [&](const float* pool, uint32_t dst, int pitch, int j, int page, int len) {
        const int tok = j * kKeys + key;
        const uint32_t row = dst + key * pitch * 4;
        if (tok < len && (page < 0 || page >= pp.pages)) {
            record_status(v.status, kDevBadPosition);
            page = -1;
        }
        if (page >= 0) {
            const float* src = pool + page_row_offset(pp, page, tok & pp.page_mask, k.g);
            for (int c = tid % kPerRow; c < quads; c += kPerRow) cp_async16(row + c * 16, src + c * 4);
        } else {
            for (int c = tid % kPerRow; c < quads; c += kPerRow)
                asm volatile("st.shared.v4.f32 [%0], {%1, %1, %1, %1};" ::"r"(row + c * 16), "f"(0.f) : "memory");
        }
        cp_commit();
    };
    while (k.f < hi) {
        const int j0 = k.j, j1 = min(k.n, k.j + (hi - k.f));
        const int len = k.rq.c + pp.by_group.div(k.rq.rows);
        __syncthreads();  // the unit before has been read
        const bool live = k.q * kRows + kPer * (ty & ~3) < k.rq.rows;  // some row of the warp is the unit's
        int page = page_of(j0, len);
        copy(P2, k_u, C::kPitch, j0, page, len);
        int pos[kPer];
        float corr[kPer], m[kPer], l[kPer];
        size_t yr[kPer];
        float2 o[kPer][2 * kQuads];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int rho = min(k.q * kRows + kPer * ty + i, k.rq.rows - 1), t = pp.by_group.div(rho);
            pos[i] = k.rq.c + t;
            yr[i] = (size_t)(k.rq.first + t) * pp.H + k.g * pp.group + (rho - t * pp.group);
            corr[i] = pp.lambda * logf((float)(pos[i] + 1));
            m[i] = -INFINITY;
            l[i] = 0.f;
            for (int c = tx; c < quads; c += kTx) {
                const float4 x = *reinterpret_cast<const float4*>(P1 + yr[i] * pp.d + 4 * c);
                if constexpr (kPer > 1) {
                    float* q = sQ + 4 * c * C::kPitchQ + kPer * ty + i;
                    q[0] = x.x, q[C::kPitchQ] = x.y, q[2 * C::kPitchQ] = x.z, q[3 * C::kPitchQ] = x.w;
                } else {
                    *reinterpret_cast<float4*>(sQ + ty * C::kPitchQ + 4 * c) = x;
                }
            }
#pragma unroll
            for (int e = 0; e < 2 * kQuads; ++e) o[i][e] = make_float2(0.f, 0.f);
        }
        for (int j = j0; j < j1; ++j) {
            cp_wait<0>();  // P2 of this tile
            __syncthreads();  // and I~ of the one before has been read
            copy(I, v_u, C::kWidth, j, page, len);
            if (j + 1 < j1) page = page_of(j + 1, len);
            if (live) {
                float sc[kPer][8];
                if constexpr (kPer > 1) {  // pairs of rows, a key's column for both
                    float2 s2[kPer / 2][8] = {};
#pragma unroll 1
                    for (int c = 0; c < quads; ++c) {
                        float4 q[4];
                        static_assert(kPer == 4, "a row's four");
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            q[x] = *reinterpret_cast<const float4*>(sQ + (4 * c + x) * C::kPitchQ + 4 * ty);
#pragma unroll
                        for (int n = 0; n < 8; ++n) {
                            const float4 kk = *reinterpret_cast<const float4*>(sK + (tx + kTx * n) * C::kPitch + 4 * c);
#pragma unroll
                            for (int x = 0; x < 4; ++x) {
                                const float w = x == 0 ? kk.x : x == 1 ? kk.y : x == 2 ? kk.z : kk.w;
                                s2[0][n] = ptx::fma2(make_float2(w, w), make_float2(q[x].x, q[x].y), s2[0][n]);
                                s2[1][n] = ptx::fma2(make_float2(w, w), make_float2(q[x].z, q[x].w), s2[1][n]);
                            }
                        }
                    }
#pragma unroll
                    for (int i = 0; i < kPer; ++i)
#pragma unroll
                        for (int n = 0; n < 8; ++n) sc[i][n] = (i & 1) ? s2[i / 2][n].y : s2[i / 2][n].x;
                } else {  // pairs of columns
                    float2 s2[8] = {};
#pragma unroll 4
                    for (int c = 0; c < quads; ++c) {
                        const float4 q = *reinterpret_cast<const float4*>(sQ + ty * C::kPitchQ + 4 * c);
#pragma unroll
                        for (int n = 0; n < 8; ++n) {
                            const float4 kk = *reinterpret_cast<const float4*>(sK + (tx + kTx * n) * C::kPitch + 4 * c);
                            s2[n] = ptx::fma2(make_float2(q.x, q.y), make_float2(kk.x, kk.y), s2[n]);
                            s2[n] = ptx::fma2(make_float2(q.z, q.w), make_float2(kk.z, kk.w), s2[n]);
                        }
                    }
#pragma unroll
                    for (int n = 0; n < 8; ++n) sc[0][n] = s2[n].x + s2[n].y;
                }
                const int col = j * kKeys + tx;
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    float r[8], mt = -INFINITY;
#pragma unroll
                    for (int n = 0; n < 8; ++n) {
                        const float u = sc[i][n] * pp.inv_sqrt_d;
                        r[n] = u * sigmoid_f32(u);
                    }
                    if (j * kKeys > pos[i] - kKeys) {  // the row's own token is in this tile (whose end may be 2^31) or before it
#pragma unroll
                        for (int n = 0; n < 8; ++n) {
                            if (col + kTx * n == pos[i])
                                r[n] = sigmoid_f32(sc[i][n] * inv_diag) + corr[i];
                            if (col + kTx * n > pos[i]) r[n] = -INFINITY;
                        }
                    }
#pragma unroll
                    for (int n = 0; n < 8; ++n) mt = fmaxf(mt, r[n]);
#pragma unroll
                    for (int x = kTx / 2; x > 0; x >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, x));
                    const float mn = fmaxf(m[i], mt);
                    // A row that has seen nothing yet (a piece that begins past its token) stays at -inf.
                    const float f = mn == -INFINITY ? 1.f : ptx::ex2_approx((m[i] - mn) * kLog2e);
                    const float ref = mn == -INFINITY ? 0.f : mn;
                    m[i] = mn;
                    float sum = 0.f;
#pragma unroll
                    for (int n = 0; n < 8; ++n) {
                        const float p = ptx::ex2_approx((r[n] - ref) * kLog2e);
                        sum += p;
                        sP[(kPer * ty + i) * kPitchP + tx + kTx * n] = p;
                    }
                    l[i] = l[i] * f + sum;  // this thread's keys; summed over tx at the end
#pragma unroll
                    for (int e = 0; e < 2 * kQuads; ++e) o[i][e].x *= f, o[i][e].y *= f;
                }
            }
            cp_wait<0>();  // I~ of this tile
            __syncthreads();  // and P2 has been read
            if (j + 1 < j1) copy(P2, k_u, C::kPitch, j + 1, page, len);
            if (live) {
#pragma unroll (kPer == 1 ? 4 : 1)
                for (int c = 0; c < kKeys / 4; ++c) {
                    float4 p[kPer];
#pragma unroll
                    for (int i = 0; i < kPer; ++i)
                        p[i] = *reinterpret_cast<const float4*>(sP + (kPer * ty + i) * kPitchP + 4 * c);
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
#pragma unroll
                        for (int e = 0; e < kQuads; ++e) {
                            const float4 vv =
                                *reinterpret_cast<const float4*>(sV + (4 * c + n) * C::kWidth + 4 * tx + 32 * e);
#pragma unroll
                            for (int i = 0; i < kPer; ++i) {
                                const float w = n == 0 ? p[i].x : n == 1 ? p[i].y : n == 2 ? p[i].z : p[i].w;
                                o[i][2 * e] = ptx::fma2(make_float2(w, w), make_float2(vv.x, vv.y), o[i][2 * e]);
                                o[i][2 * e + 1] = ptx::fma2(make_float2(w, w), make_float2(vv.z, vv.w), o[i][2 * e + 1]);
                            }
                        }
                    }
                }
            }
        }
        const bool direct = j0 == 0 && j1 == k.n;
        float* slot = part + ((size_t)worker * 2 + (j0 == 0 ? 1 : 0)) * slot_floats(kRows, C::kWidth);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            float ls = l[i];
#pragma unroll
            for (int x = kTx / 2; x > 0; x >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, x);
            const int row = kPer * ty + i;
            if (k.q * kRows + row >= k.rq.rows) continue;
            const float inv = 1.f / ls;
#pragma unroll
            for (int e = 0; e < kQuads; ++e) {
                const int c = 4 * tx + 32 * e;
                const float4 y = make_float4(o[i][2 * e].x, o[i][2 * e].y, o[i][2 * e + 1].x, o[i][2 * e + 1].y);
                if (direct && c < pp.d)
                    *reinterpret_cast<float4*>(Y + yr[i] * pp.d + c) =
                        make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv);
                if (!direct) *reinterpret_cast<float4*>(slot + row * C::kWidth + c) = y;
            }
            if (tx == 0) {
                if (direct) {
                    if (L != nullptr) L[yr[i]] = m[i] + logf(ls) - corr[i];
                } else {
                    store_pair(slot + kRows * C::kWidth + 2 * row, piece_max(j0 * kKeys <= pos[i], m[i] * kLog2e), ls);
                }
            }
        }
        if (j0 == 0 && !direct) 
            mine = PieceMeta{share.owner(k.f + k.n - 1) - worker + 1, k.rq.first, k.rq.c, k.rq.rows, k.g, k.q};
        k.f += j1 - j0;
        cursor_next_unit<Tl>(k, v, prefix, hi);
    }
    if (tid == 0) {
        meta[worker] = mine;
        dependency_wait();
    }
}

template <int kQuads, int kPer>
size_t f32_bytes(int num_sms) {
    using C = F32Cfg<kQuads, kPer>;
    return (size_t)num_sms * C::kPerSm *
           (sizeof(PieceMeta) + 8 + 2 * slot_floats(C::kRows, C::kWidth) * sizeof(float));
}

template <int kQuads, int kPer>
cudaError_t launch_f32(const PagedProblem& pp, const PagedFwdArgs& a, void* ws, MergeSide* small, bool last,
                       cudaStream_t s) {
    using C = F32Cfg<kQuads, kPer>;
    static_assert(C::kFloats * 4 + 64 + kPagedMaxRequests * 4 <= 232448, "shared memory of a block");
    auto kern = paged_f32_kernel<kQuads, kPer>;
    static OncePerDevice once;
    cudaError_t e = allow_dynamic_smem(once, kern, C::smem(kPagedMaxRequests));
    if (e != cudaSuccess) return e;
    const FwdView v{pp, a.table, a.starts, a.cached, a.max_fresh, kPer == 1 ? 0 : kSmallRows,
                    kPer == 1 ? kSmallRows : INT32_MAX, a.status};
    const int workers = a.num_sms * C::kPerSm;
    float* part = static_cast<float*>(ws);
    PieceMeta* meta = reinterpret_cast<PieceMeta*>(part + (size_t)workers * 2 * slot_floats(C::kRows, C::kWidth));
    e = launch_chained(kern, dim3((unsigned)workers), C::kThreads, C::smem(pp.R), s, v, (const float*)a.P1,
                       (const float*)a.P2_pages, (const float*)a.I_pages, (float*)a.Y, a.L, part, meta);
    if (e != cudaSuccess) return e;
    const MergeSide side{part, meta, workers};
    if constexpr (kPer == 1) {
        *small = side;
        return last ? launch_merge<float, C::kRows, 0, C::kWidth>(v, side, MergeSide{}, a.Y, a.L, s) : cudaSuccess;
    } else {
        return launch_merge<float, kSmallRows, C::kRows, C::kWidth>(v, *small, side, a.Y, a.L, s);
    }
}

template <int kQuads>
cudaError_t launch_f32_width(const PagedProblem& pp, const PagedFwdArgs& a, void* ws, int* launches, cudaStream_t s) {
    const bool last = (int64_t)a.max_fresh * pp.group <= kSmallRows;
    MergeSide small;
    const cudaError_t e = launch_f32<kQuads, 1>(pp, a, ws, &small, last, s);
    *launches = last ? 2 : 3;
    if (e != cudaSuccess || last) return e;
    return launch_f32<kQuads, kLong>(pp, a, static_cast<char*>(ws) + f32_bytes<kQuads, 1>(a.num_sms), &small, true, s);
}

template <int kQuads>
size_t f32_width_bytes(const PagedProblem& pp, int max_fresh, int num_sms) {
    const size_t small = f32_bytes<kQuads, 1>(num_sms);  // the two passes overlap: a part each
    return (int64_t)max_fresh * pp.group <= kSmallRows ? small : small + f32_bytes<kQuads, kLong>(num_sms);
}

}  // namespace
}  // namespace paged

size_t paged_f32_workspace(const PagedProblem& pp, int max_fresh, int num_sms) {
    using namespace paged;
    if (pp.d <= 64) return f32_width_bytes<2>(pp, max_fresh, num_sms);
    if (pp.d <= 96) return f32_width_bytes<3>(pp, max_fresh, num_sms);
    return f32_width_bytes<4>(pp, max_fresh, num_sms);
}

cudaError_t launch_paged_f32(const PagedProblem& pp, const PagedFwdArgs& a, void* ws, int* launches, cudaStream_t s) {
    using namespace paged;
    if (pp.d <= 64) return launch_f32_width<2>(pp, a, ws, launches, s);
    if (pp.d <= 96) return launch_f32_width<3>(pp, a, ws, launches, s);
    return launch_f32_width<4>(pp, a, ws, launches, s);
}

}  // namespace relation
