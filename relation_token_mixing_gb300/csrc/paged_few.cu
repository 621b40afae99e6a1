// Relation of a few new tokens per request over a paged cache (bf16): decoding and
// the verification of drafted tokens ("Ask Self, Ask Others", Sec. 5.3 eq.(18),
// Appendix A.5).  For the token at zero-based position i, per head,
//   U_j = p1 . p2_j / sqrt(d), R_j = SiLU(U_j) for j < i, R_i = sigmoid(U_i / tau_S)
//   + lambda log(i + 1) (the count correction moved to the diagonal: softmax does
//   not see a shift of the whole row), Y = sum_j softmax(R)_j I~_j.
//
// Bound: the history is read once, 4 d bytes a cached token and cache head, and
// every byte serves at most 16 rows (the new tokens times the heads of a group), so
// memory bandwidth is the limit; what matters is that every SM always has enough
// loads in flight and that a key costs few instructions.  Hence
//  - a worker is one warp with a ring of its own: two stages of 32 keys (P2 and I~)
//    that it refills by TMA itself, one copy a lane, as soon as it has used one; no
//    worker waits for another, and 192 KB of an SM's shared memory are stages;
//  - the workers cut all requests' key tiles into equal parts (paged_schedule.cuh),
//    so ragged lengths cost nothing; the pieces of a unit are merged in the block, and
//    those of different blocks by a second kernel;
//  - the products run on mma.sync m16n8k16 with the keys as M and the rows as N (8 or
//    16): S^T = P2 P1^T, O^T = I~^T F^T.  The keys, which are many, then fill the
//    wide side, a key's fragment is loaded once for all rows, and the weights' 8 x 8
//    blocks are turned by movmatrix between the products.  With 16 rows at most there
//    is nothing for the 128-row tcgen05 tile and its trip through TMEM to gain.
// Measured: decoding 32 requests of 1000 to 32767, 32 heads over 8 of 128: 0.264 to 0.270 ms,
// 6.7 to 6.8 TB/s, the copy rate; 8 requests of up to 4095, 16 heads of 64: 22 us, of which 3.3 until the first
// bytes and 4 for the merge; 48 requests of up to 8192 with 0 to 5 new tokens, 10 heads over 5 of
// 64: 46 us, 4.5 TB/s.
// The sigmoid is (1 + tanh)/2 by the hardware's tanh (2^-11), below the rounding of
// the bf16 output; the weights are rounded to bf16 for the second product (as the
// operands are), their sum is not.
#include <cuda_bf16.h>

#include <algorithm>

#include "once_per_device.h"
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
    // Promotion to 128 bytes, a row's panel: with 256, token-major pages bring in the next
    // head's rows too (48 requests with drafted tokens: 46 us, with 256 50 us).
    const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box,
                              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

namespace paged {
namespace {

constexpr int kKeys = 32;     // keys of a stage
constexpr int kMinTiles = 2;  // a worker's least: below that the merge costs more than it spreads

// DK: 16-column steps of the head width (d = 60 reads its last 4 columns as zero).
// NT: groups of 8 packed rows of a unit.
template <int DK, int NT>
struct FewCfg {
    static constexpr int kPanels = DK > 4 ? 2 : 1;  // 64-column panels
    // Workers of a block and stages of each: 192 KB in all.  128 columns and 8 rows: 4 x 3
    // (decode 32 x 32k: 268 us, 6 x 2: 278 us); 16 rows, more work a key: 6 x 2 (a mixed step
    // of 80-wide heads: 84 us, 4 x 3: 89 us).
    static constexpr int kWarps = kPanels == 1 ? 12 : NT == 1 ? 4 : 6;
    static constexpr int kStages = kPanels == 2 && NT == 1 ? 3 : 2;
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kPanelBytes = kKeys * 128;
    static constexpr int kTensorBytes = kPanels * kPanelBytes;  // P2 or I~ of a stage
    static constexpr int kStageBytes = 2 * kTensorBytes;
    static constexpr int kRingBytes = kWarps * kStages * kStageBytes;
    static constexpr int kRows = 8 * NT, kWidth = kPanels * 64;  // of a partial slot
    static constexpr size_t kSlot = slot_floats(kRows, kWidth);
    static_assert(kSlot * 4 <= kStages * kStageBytes, "a worker's last piece takes its ring's place");
    static int smem(int R) { return 1024 + kRingBytes + 1024 + (R * 4 + 15) / 16 * 16; }
};

// What a worker leaves in shared memory of the unit that it begins and does not
// finish, and (the block's first worker) of the one that it continues.
struct FewPiece {
    int pieces;  // workers from this one on, its own included (0: no such unit)
    int end;     // the line's tile after the unit's last
    int first, c, rows, g;
};

struct FewBars {
    uint64_t full[24];  // a worker's stages one after another
    int64_t sums[16];
    FewPiece begun[12], continued;
    int abort_flag;
};
static_assert(sizeof(FewBars) <= 1024, "the barriers' region");

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
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
// An 8 x 8 block of 16-bit values, a lane holding columns 2 (lane % 4) and the next
// of row lane / 4, transposed.
__device__ __forceinline__ uint32_t turn8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// A stretch of a worker's: a unit's key tiles j .. n - 1.
struct FewUnit {
    int r, g, j, n;
};

__device__ __forceinline__ FewUnit few_seek(const FwdView& v, const int* prefix, int f) {
    FewUnit u;
    u.r = schedule_find(v, prefix, f);
    const int before = u.r ? prefix[u.r - 1] : 0;
    u.n = prefix[u.r] - before;
    const int off = f - before * v.pp.G;
    u.g = off / u.n;
    u.j = off - u.g * u.n;
    return u;
}
__device__ __forceinline__ void few_next(FewUnit& u, const FwdView& v, const int* prefix) {
    u.j = 0;
    if (++u.g < v.pp.G) return;
    u.g = 0;
    do ++u.r; while (prefix[u.r] == prefix[u.r - 1]);
    u.n = prefix[u.r] - prefix[u.r - 1];
}
__device__ __forceinline__ Request few_request(const FwdView& v, int r) {
    Request q{__ldg(v.starts + r), __ldg(v.cached + r), 0};
    q.rows = __ldg(v.starts + r + 1) - q.first;  // new tokens; times the group below
    return q;
}

// A unit has all of a request's packed rows of one cache head.
template <int DK, int NT>
__global__ void __launch_bounds__(FewCfg<DK, NT>::kThreads, 1)
    paged_few_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const __grid_constant__ FwdView v, const __nv_bfloat16* __restrict__ P1,
                     __nv_bfloat16* __restrict__ Y, float* __restrict__ L, float* __restrict__ part,
                     PieceMeta* __restrict__ meta) {
    using C = FewCfg<DK, NT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    FewBars* bars = reinterpret_cast<FewBars*>(smem + C::kRingBytes);
    int* prefix = reinterpret_cast<int*>(smem + C::kRingBytes + 1024);
    const PagedProblem& pp = v.pp;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x < C::kWarps * C::kStages) {
        ptx::mbar_init(&bars->full[threadIdx.x], 1);
        ptx::fence_barrier_init();
        if (threadIdx.x == 0) {
            bars->abort_flag = 0;
            ptx::tma_prefetch_desc(&tm_k);
            ptx::tma_prefetch_desc(&tm_v);
        }
    }
    dependency_wait();
    dependency_release();
    const int total = schedule_build(v, prefix, bars->sums, [&](const Request& q) {
        return ((int64_t)q.c + pp.by_group.div(q.rows) + kKeys - 1) / kKeys;
    });
    volatile int* abort_flag = &bars->abort_flag;
    const int workers = gridDim.x * C::kWarps;
    const Share share(total, workers, kMinTiles);

    const int worker0 = blockIdx.x * C::kWarps, worker = worker0 + warp;
    const int lo = share.begin(worker), hi = share.begin(worker + 1);
    if (lane == 0) bars->begun[warp].pieces = 0;
    if (threadIdx.x == 0) bars->continued.pieces = 0;
    if (lo < hi) {
    uint64_t* full = bars->full + warp * C::kStages;
    uint8_t* ring = smem + warp * C::kStages * C::kStageBytes;
    FewUnit u = few_seek(v, prefix, lo);

    // ---- loads: u_ld runs ahead of the unit in hand; 32 block-table entries, one per
    // lane, are asked for as soon as the tile before has been sent for.
    FewUnit u_ld = u;
    int need, tb0 = 0, tb = 0;
    const int box = min(pp.page, kKeys);
    auto ask = [&](bool unit) {
        if (unit) {
            const Request q = few_request(v, u_ld.r);
            need = (q.c + q.rows + pp.page_mask) >> pp.page_shift;
        }
        tb0 = (u_ld.j * kKeys) >> pp.page_shift;
        tb = 0;
        if (tb0 + lane < need) tb = __ldg(v.table + (size_t)u_ld.r * pp.width + tb0 + lane);
    };
    int sent = lo;
    auto send = [&](int s) {
        const int tok = u_ld.j * kKeys, k0 = tok >> pp.page_shift;
        const int parts = box < kKeys && k0 + 1 < need ? 2 : 1;  // pages of 16 tokens: two to a stage
        const int copies = 2 * C::kPanels * parts;
        const int which = lane % (2 * C::kPanels), half = lane / (2 * C::kPanels);
        int page = __shfl_sync(0xffffffffu, tb, (k0 - tb0 + half) & 31);
        if (lane == 0) ptx::mbar_arrive_expect_tx(&full[s], copies * box * 128);
        __syncwarp();
        if (lane < copies) {
            if ((unsigned)page >= (unsigned)pp.pages) {  // reads as zeros (the map's bound), and is reported
                record_status(v.status, kDevBadPosition);
                page = pp.pages;
            }
            ptx::tma_load_4d(ring + s * C::kStageBytes + which * C::kPanelBytes + half * 2048,
                             which >= C::kPanels ? &tm_v : &tm_k, &full[s], (which % C::kPanels) * 64,
                             half ? 0 : tok & pp.page_mask & ~(box - 1), u_ld.g, page);
        }
        if (++sent < hi) {
            const bool unit = ++u_ld.j == u_ld.n;
            if (unit) few_next(u_ld, v, prefix);
            if (unit || ((u_ld.j * kKeys) >> pp.page_shift) + 1 >= tb0 + 32) ask(unit);
        }
    };
    ask(true);
    for (int s = 0; s < C::kStages && sent < hi; ++s) send(s);

    Request rq;
    int j_begin = u.j, len = 0, nt_used = NT;
    // A lane holds packed rows 8 n + 2 (lane % 4) and the next one, of keys lane / 4 (+ 8).
    uint32_t qf[NT][DK][2];
    float o[NT][DK][4], m[NT][2], l[NT][2], corr[NT][2];
    int pos[NT][2];
    const int key0 = lane >> 2, col0 = 2 * (lane & 3);
    auto begin_unit = [&]() {
        rq = few_request(v, u.r);
        len = rq.c + rq.rows;
        rq.rows *= pp.group;
        nt_used = (rq.rows + 7) >> 3;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int rho = min(8 * n + key0, rq.rows - 1), t = pp.by_group.div(rho);
            const __nv_bfloat16* q =
                P1 + ((size_t)(rq.first + t) * pp.H + u.g * pp.group + (rho - t * pp.group)) * pp.d;
#pragma unroll
            for (int ks = 0; ks < DK; ++ks)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int c = ks * 16 + e * 8 + col0;
                    qf[n][ks][e] = c < pp.d ? __ldg(reinterpret_cast<const uint32_t*>(q + c)) : 0u;
                }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                pos[n][e] = rq.c + pp.by_group.div(min(8 * n + col0 + e, rq.rows - 1));
                corr[n][e] = pp.lambda * __log2f((float)(pos[n][e] + 1));
                m[n][e] = -INFINITY;
                l[n][e] = 0.f;
            }
#pragma unroll
            for (int dt = 0; dt < DK; ++dt)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[n][dt][e] = 0.f;
        }
    };
    auto end_unit = [&](int f_end) {  // f_end: the line's tile after the last one of this piece
        const bool direct = j_begin == 0 && u.j == u.n;
        const int end = f_end - u.j + u.n;
        // The last piece of a stretch: nothing is in flight to the ring any more.
        float* slot = f_end == hi ? reinterpret_cast<float*>(ring) : part + (size_t)worker * C::kSlot;
        if (!direct && lane == 0 && (j_begin == 0 || warp == 0)) {
            FewPiece& pc = j_begin == 0 ? bars->begun[warp] : bars->continued;
            pc = FewPiece{share.owner(end - 1) - worker + 1, end, rq.first, rq.c, rq.rows, u.g};
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            if (n >= nt_used) break;
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], x);
            if (direct) {
                // Turned back to rows: a lane stores pairs of columns of row 8 n + lane / 4.
                const int rho = 8 * n + key0, t = pp.by_group.div(min(rho, rq.rows - 1));
                const size_t yr = (size_t)(rq.first + t) * pp.H + u.g * pp.group + (rho - t * pp.group);
                const float i0 = 1.f / l[n][0], i1 = 1.f / l[n][1];
#pragma unroll
                for (int dt = 0; dt < DK; ++dt)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t w =
                            turn8(ptx::pack_bf16x2(o[n][dt][2 * h] * i0, o[n][dt][2 * h + 1] * i1));
                        const int c = dt * 16 + h * 8 + col0;
                        if (rho < rq.rows && c < pp.d) *reinterpret_cast<uint32_t*>(Y + yr * pp.d + c) = w;
                    }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int rho = 8 * n + col0 + e;
                if (rho >= rq.rows) continue;
                if (!direct) {
#pragma unroll
                    for (int dt = 0; dt < DK; ++dt)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            slot[rho * C::kWidth + dt * 16 + h * 8 + key0] = o[n][dt][2 * h + e];
                    if (key0 == 0)
                        store_pair(slot + C::kRows * C::kWidth + 2 * rho,
                                   piece_max(j_begin * kKeys <= pos[n][e], m[n][e]), l[n][e]);
                } else if (L != nullptr && key0 == 0) {
                    const int t = pp.by_group.div(rho);
                    L[(size_t)(rq.first + t) * pp.H + u.g * pp.group + (rho - t * pp.group)] =
                        (m[n][e] + __log2f(l[n][e]) - corr[n][e]) * kLn2;
                }
            }
        }
    };
    begin_unit();

    const uint32_t ring_u = ptx::smem_u32(ring);
    const int sw = lane & 7;
    const uint32_t k_row = ((lane & 7) + ((lane >> 3) & 1) * 8) * 128, k_chunk = lane >> 4;
    const uint32_t v_row = ((lane & 7) + ((lane >> 4) & 1) * 8) * 128, v_chunk = (lane >> 3) & 1;
    const float c_half = 0.5f * pp.inv_sqrt_d, c_self = c_half / pp.tau_S;
    for (int it = 0; it < hi - lo; ++it) {
        const int s = it % C::kStages;
        if (!ptx::mbar_wait_warp(&full[s], (it / C::kStages) & 1, abort_flag, v.status, kDevTimeoutFull)) {
            for (int x = it; x < sent - lo; ++x)  // let what is in flight land
                ptx::mbar_drain(&full[x % C::kStages], (x / C::kStages) & 1, v.status);
            break;
        }
        const uint32_t sk = ring_u + s * C::kStageBytes, sv = sk + C::kTensorBytes;
        const int tok = u.j * kKeys;
        if (tok > len - kKeys) {  // (tok + kKeys may be 2^31)
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
        float sc[NT][2][4] = {};
#pragma unroll
        for (int ks = 0; ks < DK; ++ks)
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
                uint32_t a[4];
                ldsm4(a, sk + (ks / 4) * C::kPanelBytes + mt * 2048 + k_row + (((2 * (ks % 4) + k_chunk) ^ sw) << 4));
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    if (n < nt_used) mma16816(sc[n][mt], a, qf[n][ks][0], qf[n][ks][1]);
            }
        const bool edge = tok > rq.c - kKeys;  // new tokens or the history's end in this tile
        float mt_[NT][2];
        bool raise = false;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            if (n >= nt_used) break;
            mt_[n][0] = mt_[n][1] = -INFINITY;
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float x = sc[n][mt][e], h = x * c_half;
                    float r = fmaf(h, ptx::tanh_approx(h), h) * kLog2e;  // SiLU(U) = (U/2)(1 + tanh(U/2))
                    if (edge) {
                        const int j = tok + mt * 16 + key0 + (e >> 1) * 8;
                        if (j == pos[n][e & 1])
                            r = fmaf(0.5f * kLog2e, ptx::tanh_approx(x * c_self), 0.5f * kLog2e) + corr[n][e & 1];
                        else if (j > pos[n][e & 1])
                            r = -INFINITY;
                    }
                    sc[n][mt][e] = r;
                    mt_[n][e & 1] = fmaxf(mt_[n][e & 1], r);
                }
            raise |= mt_[n][0] > m[n][0] + kRaise || mt_[n][1] > m[n][1] + kRaise;
        }
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if (n >= nt_used) break;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float x = mt_[n][e];
#pragma unroll
                    for (int y = 4; y < 32; y <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, y));
                    x = fmaxf(x, m[n][e]);
                    const float f = x == -INFINITY ? 1.f : ptx::ex2_approx(m[n][e] - x);
                    m[n][e] = x;
                    l[n][e] *= f;
#pragma unroll
                    for (int dt = 0; dt < DK; ++dt) o[n][dt][e] *= f, o[n][dt][2 + e] *= f;
                }
            }
        }
        uint32_t pb[NT][2][2];  // F^T as the second product's B: key block, its halves
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            if (n >= nt_used) break;
            // A row that has seen nothing yet: every weight is 0.
            const float b0 = m[n][0] == -INFINITY ? 0.f : m[n][0], b1 = m[n][1] == -INFINITY ? 0.f : m[n][1];
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float p0 = ptx::ex2_approx(sc[n][mt][2 * h] - b0);
                    const float p1 = ptx::ex2_approx(sc[n][mt][2 * h + 1] - b1);
                    l[n][0] += p0;
                    l[n][1] += p1;
                    pb[n][mt][h] = turn8(ptx::pack_bf16x2(p0, p1));
                }
        }
#pragma unroll
        for (int dt = 0; dt < DK; ++dt)
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
                uint32_t a[4];
                ldsm4t(a, sv + (dt / 4) * C::kPanelBytes + mt * 2048 + v_row + (((2 * (dt % 4) + v_chunk) ^ sw) << 4));
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    if (n < nt_used) mma16816(o[n][dt], a, pb[n][mt][0], pb[n][mt][1]);
            }
        __syncwarp();  // every lane has read the stage
        if (sent < hi) send(s);
        ++u.j;
        if (u.j == u.n || it + 1 == hi - lo) {
            end_unit(lo + it + 1);
            if (it + 1 < hi - lo) {
                few_next(u, v, prefix);
                j_begin = 0;
                begin_unit();
            }
        }
    }
    }  // lo < hi
    if (threadIdx.x == 0) meta[blockIdx.x].pieces = 0;
    __syncthreads();
    // ---- merge inside the block: a worker's last piece is in its ring's place, one that
    // ended before its stretch did in the workspace.  What the block's ends cut goes to
    // the block's slots.  Eight threads a row.
    constexpr int kQuads = C::kWidth / 32;
    float* slots = part + (size_t)workers * C::kSlot + (size_t)blockIdx.x * 2 * C::kSlot;
    const int sub = threadIdx.x & 7;
    for (int job = threadIdx.x >> 3; job < (C::kWarps + 1) * C::kRows; job += C::kThreads / 8) {
        const int i = job / C::kRows, rho = job - i * C::kRows;
        const bool head = i == C::kWarps;
        const FewPiece& pc = head ? bars->continued : bars->begun[i];
        if (pc.pieces == 0 || rho >= pc.rows) continue;
        const int w0 = head ? 0 : i, n = min(pc.pieces, C::kWarps - w0);
        MergedRow<kQuads> out;
        for (int p = 0; p < n; ++p) {
            const int w = w0 + p;
            const bool last = p + 1 < pc.pieces || pc.end == share.begin(worker0 + w + 1);  // ends its stretch
            const float* src = last ? reinterpret_cast<const float*>(smem + w * C::kStages * C::kStageBytes)
                                    : part + (size_t)(worker0 + w) * C::kSlot;
            const float2 ml = *reinterpret_cast<const float2*>(src + C::kRows * C::kWidth + 2 * rho);
            float4 x[kQuads];
#pragma unroll
            for (int e = 0; e < kQuads; ++e)
                x[e] = *reinterpret_cast<const float4*>(src + rho * C::kWidth + 32 * e + 4 * sub);
            out.add(ml.x, ml.y, x);
        }
        if (!head && n == pc.pieces) {
            out.finish(pp, pc.first, pc.c, pc.g, rho, sub, Y, L);
            continue;
        }
        float* dst = slots + (head ? 0 : C::kSlot);
#pragma unroll
        for (int e = 0; e < kQuads; ++e)
            *reinterpret_cast<float4*>(dst + rho * C::kWidth + 32 * e + 4 * sub) = out.acc[e];
        if (sub == 0) store_pair(dst + C::kRows * C::kWidth + 2 * rho, out.m, out.l);
        if (!head && sub == 0 && rho == 0)
            meta[blockIdx.x] = PieceMeta{share.owner(pc.end - 1) / C::kWarps - (int)blockIdx.x + 1, pc.first, pc.c,
                                         pc.rows, pc.g, 0};
    }
}

template <int DK, int NT>
size_t few_bytes(int num_sms) {
    using C = FewCfg<DK, NT>;
    return (size_t)num_sms * (sizeof(PieceMeta) + 8 + (C::kWarps + 2) * C::kSlot * sizeof(float));
}

template <int DK, int NT>
cudaError_t launch_few(const PagedProblem& pp, const PagedFwdArgs& a, void* ws, MergeSide* left, cudaStream_t s) {
    using C = FewCfg<DK, NT>;
    auto kern = paged_few_kernel<DK, NT>;
    static OncePerDevice once;
    static_assert(1024 + C::kRingBytes + 1024 + kPagedMaxRequests * 4 <= 232448, "shared memory of a block");
    cudaError_t e = allow_dynamic_smem(once, kern, C::smem(kPagedMaxRequests));
    if (e != cudaSuccess) return e;
    const FwdView v{pp, a.table, a.starts, a.cached, a.max_fresh, 0, kPagedFewRows, a.status};
    // A piece of each worker, two of each block, the blocks' units.
    float* part = static_cast<float*>(ws);
    float* slots = part + (size_t)a.num_sms * C::kWarps * C::kSlot;
    PieceMeta* meta = reinterpret_cast<PieceMeta*>(slots + (size_t)a.num_sms * 2 * C::kSlot);
    CUtensorMap mk, mv;
    const int box = std::min(pp.page, kKeys);
    if ((e = make_page_map(&mk, a.P2_pages, pp, box)) != cudaSuccess) return e;
    if ((e = make_page_map(&mv, a.I_pages, pp, box)) != cudaSuccess) return e;
    e = launch_chained(kern, dim3((unsigned)a.num_sms), C::kThreads, C::smem(pp.R), s, mk, mv, v,
                       (const __nv_bfloat16*)a.P1, (__nv_bfloat16*)a.Y, a.L, part, meta);
    if (e != cudaSuccess) return e;
    const MergeSide side{slots, meta, a.num_sms};
    if (left != nullptr) {
        *left = side;
        return cudaSuccess;
    }
    return launch_merge<__nv_bfloat16, C::kRows, 0, C::kWidth>(v, side, MergeSide{}, a.Y, a.L, s);
}

// Whether the host's bound on the new tokens keeps every unit within 8 rows.
bool few_rows(const PagedProblem& pp, int max_fresh) { return (int64_t)max_fresh * pp.group <= 8; }

template <int DK>
cudaError_t launch_few_d(const PagedProblem& pp, const PagedFwdArgs& a, void* ws, MergeSide* left, cudaStream_t s) {
    return few_rows(pp, a.max_fresh) ? launch_few<DK, 1>(pp, a, ws, left, s) : launch_few<DK, 2>(pp, a, ws, left, s);
}

template <int DK>
size_t few_bytes_d(const PagedProblem& pp, int max_fresh, int num_sms) {
    return few_rows(pp, max_fresh) ? few_bytes<DK, 1>(num_sms) : few_bytes<DK, 2>(num_sms);
}

}  // namespace
}  // namespace paged

size_t paged_few_workspace(const PagedProblem& pp, int max_fresh, int num_sms) {
    using namespace paged;
    switch ((pp.d + 15) / 16) {
        case 3: return few_bytes_d<3>(pp, max_fresh, num_sms);
        case 4: return few_bytes_d<4>(pp, max_fresh, num_sms);
        case 5: return few_bytes_d<5>(pp, max_fresh, num_sms);
        default: return few_bytes_d<8>(pp, max_fresh, num_sms);
    }
}

cudaError_t launch_paged_few(const PagedProblem& pp, const PagedFwdArgs& a, void* workspace, paged::MergeSide* left,
                             cudaStream_t s) {
    using namespace paged;
    switch ((pp.d + 15) / 16) {
        case 3: return launch_few_d<3>(pp, a, workspace, left, s);
        case 4: return launch_few_d<4>(pp, a, workspace, left, s);
        case 5: return launch_few_d<5>(pp, a, workspace, left, s);
        default: return launch_few_d<8>(pp, a, workspace, left, s);
    }
}

}  // namespace relation
