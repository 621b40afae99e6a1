// Relation of a few new tokens per request over a paged cache (bf16): decoding and
// the verification of drafted tokens ("Ask Self, Ask Others", Sec. 5.3 eq.(18),
// Appendix A.5).  For the token at zero-based position i, per head,
//   U_j = p1 . p2_j / sqrt(d), R_j = SiLU(U_j) for j < i, R_i = sigmoid(U_i / tau_S)
//   + lambda log(i + 1) (the count correction moved to the diagonal: softmax does
//   not see a shift of the whole row), Y = sum_j softmax(R)_j I~_j.
//
// Bound: the history is read once, 4 d bytes a cached token and cache head, and
// every byte serves at most 16 rows (the new tokens times the heads of a group), so
// memory bandwidth is the limit, and what matters is that every SM always has
// enough loads in flight.  Hence
//  - a worker is one warp with a ring of its own: TMA brings 32 keys (P2 and I~) a
//    stage, no warp waits for another, and at least two stages a warp (128 KB an SM)
//    are in flight while one is used;
//  - the workers cut all requests' key tiles into equal parts (paged_schedule.cuh),
//    so ragged lengths cost nothing; pieces of cut units are merged by a second
//    kernel that is already resident when the first one ends;
//  - the products run on mma.sync m16n8k16 with the rows as M: it needs no TMEM
//    round trip for 16 rows, and at 4 of 11.6 cycles of the memory's time per key
//    (d = 64) it is not what bounds the kernel, which is why the 128-row tcgen05
//    tile is left to the kernel for longer chunks.
// The scores' exponentials and the sigmoid use ex2 and a reciprocal (relative error
// 2^-22); the weights are rounded to bf16 for the second product (the same rounding
// as the operands'), their sum is not.
#include <cuda_bf16.h>

#include <algorithm>
#include <mutex>

#include "paged_fwd.cuh"
#include "tmap.h"

namespace relation {

cudaError_t make_page_map(CUtensorMap* map, const void* base, const PagedProblem& pp, int box_rows) {
    PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    if (encode == nullptr) return cudaErrorNotSupported;
    const cuuint64_t row = (cuuint64_t)pp.row * 2;
    const cuuint64_t dims[4] = {(cuuint64_t)pp.d, (cuuint64_t)pp.page, (cuuint64_t)pp.G, (cuuint64_t)pp.pages};
    const cuuint64_t strides[3] = {pp.layout == 0 ? row : row * pp.G, pp.layout == 0 ? row * pp.page : row,
                                   row * pp.G * pp.page};
    const cuuint32_t box[4] = {64, (cuuint32_t)box_rows, 1, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box,
                              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

namespace paged {
namespace {

constexpr int kRows = 16;   // packed rows of a unit: M of the MMA
constexpr int kKeys = 32;   // keys of a stage
using FewTiling = Tiling<kRows, kKeys>;
constexpr int kMinTiles = 2;  // a worker's least: below that the merge costs more than it spreads

// DK: 16-column steps of the head width (d = 60 reads its last 4 columns as zero).
template <int DK>
struct FewCfg {
    static constexpr int kPanels = DK > 4 ? 2 : 1;             // 64-column panels
    static constexpr int kWarps = kPanels == 1 ? 8 : 4;        // workers of a block
    static constexpr int kStages = 3;
    static constexpr int kPanelBytes = kKeys * 128;
    static constexpr int kTensorBytes = kPanels * kPanelBytes;  // P2 or I~ of a stage
    static constexpr int kStageBytes = 2 * kTensorBytes;
    static constexpr int kRingBytes = kWarps * kStages * kStageBytes;
    static constexpr int kWidth = kPanels * 64;                // floats of a partial row
    static int smem(int R) { return 1024 + kRingBytes + 1024 + (R * 4 + 15) / 16 * 16; }
};

struct FewBars {
    uint64_t full[8][4];
    int sums[8];
    int abort_flag;
};
static_assert(sizeof(FewBars) <= 1024, "the barriers' region");

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// kHalf: no unit has more than 8 rows, so the lower half of the MMA's M is unused.
template <int DK, bool kHalf>
__global__ void __launch_bounds__(FewCfg<DK>::kWarps * 32, 1)
    paged_few_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const __grid_constant__ FwdView v, const __nv_bfloat16* __restrict__ P1,
                     __nv_bfloat16* __restrict__ Y, float* __restrict__ L, float* __restrict__ part,
                     PieceMeta* __restrict__ meta) {
    using C = FewCfg<DK>;
    constexpr int kHalves = kHalf ? 1 : 2;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    FewBars* bars = reinterpret_cast<FewBars*>(smem + C::kRingBytes);
    int* prefix = reinterpret_cast<int*>(smem + C::kRingBytes + 1024);
    const PagedProblem& pp = v.pp;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (threadIdx.x == 0) {
        for (int w = 0; w < C::kWarps; ++w)
            for (int s = 0; s < C::kStages; ++s) ptx::mbar_init(&bars->full[w][s], 1);
        bars->abort_flag = 0;
        ptx::fence_barrier_init();
        ptx::tma_prefetch_desc(&tm_k);
        ptx::tma_prefetch_desc(&tm_v);
    }
    const int64_t total = (int64_t)schedule_build<FewTiling>(v, prefix, bars->sums) * pp.G;
    const int worker = blockIdx.x * C::kWarps + warp, workers = gridDim.x * C::kWarps;
    int64_t lo, hi;
    worker_range(total, workers, kMinTiles, worker, &lo, &hi);
    PieceMeta mine{-1, -1, 0, 0, 0, 0, 0, 0};
    if (lo >= hi) {
        if (lane == 0) meta[worker] = mine;
        return;
    }
    volatile int* abort_flag = &bars->abort_flag;
    uint64_t* full = bars->full[warp];
    uint8_t* ring = smem + warp * C::kStages * C::kStageBytes;
    const int box = min(pp.page, kKeys);

    // ---- loads: lane b of the first boxes issues one of a stage's copies.
    Cursor ld;
    cursor_seek<FewTiling>(ld, v, prefix, lo);
    int tb0 = -1, tb_r = -1, tb = 0;  // 32 block-table entries, one per lane
    auto issue = [&](int s) {
        const int len = ld.rq.c + ld.rq.rows / pp.group;
        const int need = (len + pp.page_mask) >> pp.page_shift;
        const int tok = ld.j * kKeys, k0 = tok >> pp.page_shift;
        if (ld.r != tb_r || k0 < tb0 || k0 + (kKeys >> 4) > tb0 + 32) {
            tb_r = ld.r;
            tb0 = k0;
            const int k = tb0 + lane;
            tb = 0;
            if (k < need) {
                tb = v.table[(size_t)ld.r * pp.width + k];
                // Out of range reads as zeros (the map's bound), and is reported.
                if (tb < 0 || tb >= pp.pages) {
                    record_status(v.status, kDevBadPosition);
                    tb = pp.pages;
                }
            }
        }
        const int parts = min(kKeys / box, need - k0);  // pages of 16 tokens: two to a stage
        const int copies = 2 * C::kPanels * parts;
        if (lane == 0) ptx::mbar_arrive_expect_tx(&full[s], copies * box * 128);
        __syncwarp();
        const int part_i = lane / (2 * C::kPanels), which = lane % (2 * C::kPanels);
        const int page = __shfl_sync(0xffffffffu, tb, (k0 - tb0 + part_i) & 31);
        if (lane < copies) {
            const int tensor = which / C::kPanels, panel = which % C::kPanels;
            ptx::tma_load_4d(ring + s * C::kStageBytes + tensor * C::kTensorBytes + panel * C::kPanelBytes +
                                 part_i * box * 128,
                             tensor ? &tm_v : &tm_k, &full[s], panel * 64, part_i ? 0 : (tok & pp.page_mask), ld.g, page);
        }
        ++ld.f;
        if (++ld.j == ld.n) cursor_next_unit<FewTiling>(ld, v, prefix, hi);
    };
    const int64_t tiles = hi - lo;
    int64_t issued = 0;
    for (; issued < tiles && issued < C::kStages - 1; ++issued) issue((int)issued);

    // ---- the unit in hand
    Cursor k;
    cursor_seek<FewTiling>(k, v, prefix, lo);
    int j_begin = k.j;
    uint32_t qf[DK][4];
    float o[2 * DK][4], m[2], l[2];
    int pos[2];
    float corr[2];
    const int row0 = lane >> 2, col0 = 2 * (lane & 3);
    auto begin_unit = [&]() {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            m[h] = -INFINITY;
            l[h] = 0.f;
            const int rho = min(k.q * kRows + row0 + 8 * h, k.rq.rows - 1);
            const int t = rho / pp.group, hd = k.g * pp.group + (rho - t * pp.group);
            pos[h] = k.rq.c + t;
            corr[h] = pp.lambda * __logf((float)(pos[h] + 1));
            const __nv_bfloat16* q = P1 + ((size_t)(k.rq.first + t) * pp.H + hd) * pp.d;
#pragma unroll
            for (int ks = 0; ks < DK; ++ks)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int c = ks * 16 + e * 8 + col0;
                    qf[ks][e * 2 + h] =
                        (h < kHalves && c < pp.d) ? __ldg(reinterpret_cast<const uint32_t*>(q + c)) : 0u;
                }
        }
#pragma unroll
        for (int n = 0; n < 2 * DK; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
    };
    auto end_unit = [&](int j_end) {
        const bool direct = j_begin == 0 && j_end == k.n;
        float* slot = part + ((size_t)worker * 2 + (j_begin == 0 ? 1 : 0)) * slot_floats(kRows, C::kWidth);
        if (!direct) {
            if (j_begin > 0) {
                mine.head = k.f - j_end;
            } else {
                mine.tail = k.f - j_end;
                mine.first = k.rq.first;
                mine.c = k.rq.c;
                mine.g = k.g;
                mine.q = k.q;
                mine.rows = k.rq.rows;
            }
        }
#pragma unroll
        for (int h = 0; h < kHalves; ++h) {
            float ls = l[h];
            ls += __shfl_xor_sync(0xffffffffu, ls, 1);
            ls += __shfl_xor_sync(0xffffffffu, ls, 2);
            const int row = row0 + 8 * h, rho = k.q * kRows + row;
            if (rho >= k.rq.rows) continue;
            if (direct) {
                const int t = rho / pp.group, hd = k.g * pp.group + (rho - t * pp.group);
                const size_t yr = (size_t)(k.rq.first + t) * pp.H + hd;
                const float inv = 1.f / ls;
#pragma unroll
                for (int n = 0; n < 2 * DK; ++n)
                    if (8 * n + col0 < pp.d)
                        *reinterpret_cast<uint32_t*>(Y + yr * pp.d + 8 * n + col0) =
                            ptx::pack_bf16x2(o[n][2 * h] * inv, o[n][2 * h + 1] * inv);
                if (L != nullptr && (lane & 3) == 0) L[yr] = (m[h] + __log2f(ls)) * kLn2 - corr[h];
            } else {
#pragma unroll
                for (int n = 0; n < 2 * DK; ++n)
                    *reinterpret_cast<float2*>(slot + row * C::kWidth + 8 * n + col0) =
                        make_float2(o[n][2 * h], o[n][2 * h + 1]);
                if ((lane & 3) == 0)
                    *reinterpret_cast<float2*>(slot + kRows * C::kWidth + 2 * row) = make_float2(m[h], ls);
            }
        }
    };
    begin_unit();

    const uint32_t ring_u = ptx::smem_u32(ring);
    const int sw = lane & 7;
    const uint32_t k_row = ((lane & 7) + ((lane >> 4) & 1) * 8) * 128, k_chunk = (lane >> 3) & 1;
    const uint32_t v_row = ((lane & 7) + ((lane >> 3) & 1) * 8) * 128, v_chunk = (lane >> 4) & 1;
    const float scale = pp.inv_sqrt_d;
    int s = 0, s_issue = C::kStages - 1;
    uint32_t phase = 0;
    bool ok = true;
    for (int64_t it = 0; it < tiles; ++it) {
        if (issued < tiles) {
            // The stage freed a step ago: its readers are this warp's lanes.
            __syncwarp();
            issue(s_issue);
            ++issued;
        }
        if (++s_issue == C::kStages) s_issue = 0;
        if (!ptx::mbar_wait_warp(&full[s], phase, abort_flag, v.status, kDevTimeoutFull)) {
            ok = false;
            // What was issued lands before the block's memory is given back.
            for (int64_t x = it; x < issued; ++x) {
                ptx::mbar_drain(&full[s], phase, v.status);
                if (++s == C::kStages) s = 0, phase ^= 1;
            }
            break;
        }
        const uint32_t sk = ring_u + s * C::kStageBytes, sv = sk + C::kTensorBytes;
        float sc[4][4];
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[n][e] = 0.f;
#pragma unroll
        for (int ks = 0; ks < DK; ++ks)
#pragma unroll
            for (int np = 0; np < 2; ++np) {
                uint32_t b[4];
                ldsm4(b, sk + (ks / 4) * C::kPanelBytes + np * 2048 + k_row + (((2 * (ks % 4) + k_chunk) ^ sw) << 4));
                mma16816(sc[2 * np], qf[ks], b[0], b[1]);
                mma16816(sc[2 * np + 1], qf[ks], b[2], b[3]);
            }
        const int tok = k.j * kKeys;
        const bool edge = tok + kKeys > k.rq.c;  // new tokens or the history's end in this tile
        float mt[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int e = 0; e < 2 * kHalves; ++e) {
                const float u = sc[n][e] * scale;
                float r = u * rcp_approx(1.f + ptx::ex2_approx(-kLog2e * u));
                if (edge) {
                    const int h = e >> 1, j = tok + 8 * n + col0 + (e & 1);
                    if (j == pos[h])
                        r = rcp_approx(1.f + ptx::ex2_approx(-kLog2e * u / pp.tau_S)) + corr[h];
                    else if (j > pos[h])
                        r = -INFINITY;
                }
                sc[n][e] = r * kLog2e;
                mt[e >> 1] = fmaxf(mt[e >> 1], sc[n][e]);
            }
        bool raise = false;
#pragma unroll
        for (int h = 0; h < kHalves; ++h) raise |= mt[h] > m[h] + kRaise;
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
            for (int h = 0; h < kHalves; ++h) {
                float x = mt[h];
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
                x = fmaxf(x, m[h]);
                const float f = x == -INFINITY ? 1.f : ptx::ex2_approx(m[h] - x);
                m[h] = x;
                l[h] *= f;
#pragma unroll
                for (int n = 0; n < 2 * DK; ++n) o[n][2 * h] *= f, o[n][2 * h + 1] *= f;
            }
        }
#pragma unroll
        for (int h = 0; h < kHalves; ++h) {
            const float base = m[h] == -INFINITY ? 0.f : m[h];  // nothing seen yet: every weight is 0
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                sc[n][2 * h] = ptx::ex2_approx(sc[n][2 * h] - base);
                sc[n][2 * h + 1] = ptx::ex2_approx(sc[n][2 * h + 1] - base);
                l[h] += sc[n][2 * h] + sc[n][2 * h + 1];
            }
        }
        const int len = k.rq.c + k.rq.rows / pp.group;
        if (tok + kKeys > len) {
            // Keys past the request's end hold whatever their page holds: weight 0 times
            // a NaN is a NaN, so they are cleared.
            if (lane >= len - tok) {
                uint8_t* row = ring + s * C::kStageBytes + C::kTensorBytes + lane * 128;
#pragma unroll
                for (int p = 0; p < C::kPanels; ++p)
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        *reinterpret_cast<uint4*>(row + p * C::kPanelBytes + c * 16) = make_uint4(0, 0, 0, 0);
                ptx::fence_proxy_async_smem();  // before the copy that reuses the stage
            }
            __syncwarp();
        }
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            const uint32_t a[4] = {ptx::pack_bf16x2(sc[2 * kk][0], sc[2 * kk][1]),
                                   kHalf ? 0u : ptx::pack_bf16x2(sc[2 * kk][2], sc[2 * kk][3]),
                                   ptx::pack_bf16x2(sc[2 * kk + 1][0], sc[2 * kk + 1][1]),
                                   kHalf ? 0u : ptx::pack_bf16x2(sc[2 * kk + 1][2], sc[2 * kk + 1][3])};
#pragma unroll
            for (int np = 0; np < DK; ++np) {
                uint32_t b[4];
                ldsm4t(b, sv + (np / 4) * C::kPanelBytes + kk * 2048 + v_row + (((2 * (np % 4) + v_chunk) ^ sw) << 4));
                mma16816(o[2 * np], a, b[0], b[1]);
                mma16816(o[2 * np + 1], a, b[2], b[3]);
            }
        }
        if (++s == C::kStages) s = 0, phase ^= 1;
        ++k.f;
        if (++k.j == k.n || it + 1 == tiles) {
            end_unit(k.j);
            if (it + 1 < tiles) {
                cursor_next_unit<FewTiling>(k, v, prefix, hi);
                j_begin = 0;
                begin_unit();
            }
        }
    }
    if (!ok) mine.head = mine.tail = -1;
    if (lane == 0) meta[worker] = mine;
}

template <int DK>
int few_workers(int num_sms) { return num_sms * FewCfg<DK>::kWarps; }

template <int DK>
size_t few_bytes(int num_sms) {
    const size_t w = few_workers<DK>(num_sms);
    return w * sizeof(PieceMeta) + w * 2 * slot_floats(kRows, FewCfg<DK>::kWidth) * sizeof(float);
}

template <int DK, bool kHalf>
cudaError_t launch_few(const PagedProblem& pp, const PagedFwdArgs& a, void* ws, cudaStream_t s) {
    using C = FewCfg<DK>;
    auto kern = paged_few_kernel<DK, kHalf>;
    static std::once_flag once;
    static cudaError_t attr_err = cudaSuccess;
    std::call_once(once, [&] {
        attr_err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem(kPagedMaxRequests));
    });
    static_assert(1024 + C::kRingBytes + 1024 + kPagedMaxRequests * 4 <= 232448, "shared memory budget");
    if (attr_err != cudaSuccess) return attr_err;
    const FwdView v{pp, a.table, a.starts, a.cached, a.max_fresh, 0, kPagedFewRows, a.status};
    const int workers = few_workers<DK>(a.num_sms);
    PieceMeta* meta = static_cast<PieceMeta*>(ws);
    float* part = reinterpret_cast<float*>(meta + workers);
    CUtensorMap mk, mv;
    cudaError_t e;
    const int box = std::min(pp.page, kKeys);
    if ((e = make_page_map(&mk, a.P2_pages, pp, box)) != cudaSuccess) return e;
    if ((e = make_page_map(&mv, a.I_pages, pp, box)) != cudaSuccess) return e;
    kern<<<a.num_sms, C::kWarps * 32, C::smem(pp.R), s>>>(mk, mv, v, (const __nv_bfloat16*)a.P1, (__nv_bfloat16*)a.Y,
                                                         a.L, part, meta);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    return launch_merge_rows<__nv_bfloat16, kRows>(v, C::kWidth, part, meta, workers, a.Y, a.L, s);
}

template <int DK>
cudaError_t launch_few_d(const PagedProblem& pp, const PagedFwdArgs& a, void* ws, cudaStream_t s) {
    // The host's bound says whether any unit can have more than 8 rows.
    return (int64_t)a.max_fresh * pp.group <= 8 ? launch_few<DK, true>(pp, a, ws, s) : launch_few<DK, false>(pp, a, ws, s);
}

}  // namespace
}  // namespace paged

size_t paged_few_workspace(const PagedProblem& pp, int num_sms) {
    using namespace paged;
    switch ((pp.d + 15) / 16) {
        case 3: return few_bytes<3>(num_sms);
        case 4: return few_bytes<4>(num_sms);
        case 5: return few_bytes<5>(num_sms);
        default: return few_bytes<8>(num_sms);
    }
}

cudaError_t launch_paged_few(const PagedProblem& pp, const PagedFwdArgs& a, void* workspace, cudaStream_t s) {
    using namespace paged;
    switch ((pp.d + 15) / 16) {
        case 3: return launch_few_d<3>(pp, a, workspace, s);
        case 4: return launch_few_d<4>(pp, a, workspace, s);
        case 5: return launch_few_d<5>(pp, a, workspace, s);
        default: return launch_few_d<8>(pp, a, workspace, s);
    }
}

}  // namespace relation
