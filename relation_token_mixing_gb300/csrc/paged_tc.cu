// Relation of a chunk of new tokens over a paged cache on the tensor cores (bf16
// in, fp32 accumulate): prompts and prompt chunks ("Ask Self, Ask Others", Sec.
// 3.1 eq.(1)-(3), Sec. 5.3 eq.(18), Appendix A.5).  Per new token at zero-based
// position i, U_j = p1 . p2_j / sqrt(d), R_j = SiLU(U_j) for j < i, R_i =
// sigmoid(U_i / tau_S) + lambda log(i + 1) (the count correction moved to the
// diagonal: softmax does not see a shift of the whole row), Y = softmax(R) I~.
//
// A unit is one request's 256 packed rows (row = token * group + head in the group,
// so grouped heads share one read of their cache head) of one cache head against
// the keys up to its last token, in tiles of 128.  The kernel is persistent: the
// blocks cut all units' key tiles into equal parts (paged_schedule.cuh), so a few
// long rows fill the GPU as well as many short ones, and a second kernel merges the
// units that the cuts divide.
//   warp 0      walks the block's stretch of the line, one piece of a unit after another,
//               hands each to the others, and loads P2: the pages of each tile by TMA, one
//               copy per lane
//   warp 1      MMA issuer and TMEM owner
//   warp 2      query rows into shared memory (d <= 64)
//   warp 3      loads I~ and clears the keys past a request's end
//   warps 4-7   softmax of rows 0-127 (one thread per row)
//   warps 8-11  softmax of rows 128-255
// Per key tile, per 128-row half: S = Q K^T (both in shared memory) -> registers: SiLU,
// mask and Self where the tile reaches the rows' own tokens, online softmax -> P as bf16
// in TMEM -> O += P V.
//  - d <= 64: P has TMEM columns of its own, and the next S is issued once the softmax has
//    read this one.  The softmax takes 32 columns at a time in a loop: its code stays in the
//    instruction caches, and the two warps of a sub-partition fill each other's waits.
//  - d 80 and 128: S and O fill TMEM, P overwrites S, and the next S waits for P V.  So
//    the softmax takes the 128 columns at once, to be done with S soon, and the two halves
//    take turns on the special-function unit: one computes while the other's products run.
//
// Bound: two special functions per score (tanh, 16 results a cycle and SM; ex2, 32)
// give 3/32 cycle a score, against 4 d / 8192 = 1/32 cycle (d = 64) or 1/16 (d =
// 128) of tensor-core time, so the special-function unit is the limit.  The packed half
// forms of both functions run at half the rate, so they gain nothing.
// Measured: nine prompts of 1 to 4096 tokens, 16 heads of 64: 0.344 ms, half of it the special
// functions' time; two chunks of 1024 tokens over 16k and 31k, 32 heads over 8 of 128: 0.81 ms,
// 1.0 PFLOP/s, 63% the special functions' time (with a pass for the maximum between the two
// functions 0.347 and 0.82).  At d <= 64 the rest is the softmax's own
// latencies, with two warps to hide them (4.2 thousand cycles a tile of both halves, 3.1 of
// them special functions), and a unit's beginning and end; at d = 128 the latencies of one
// warp in its turn.  Other shapes measured on the two: tiles of 64 keys with two score
// buffers a half and no turns 0.366 and 0.995 ms; at d <= 64, 512 rows in four streams
// 0.395 ms, and two streams of alternate 64-key tiles for each half, joined at a unit's end,
// 0.343 ms (four warps a sub-partition, each waiting for its one score buffer).
#include <cuda_bf16.h>

#include <algorithm>

#include "once_per_device.h"
#include "paged_fwd.cuh"

namespace relation {
namespace paged {
namespace {

constexpr int kBM = 128, kRows = 256, kKeys = 128;
constexpr int kThreads = 384;
// 128 * 104 + 256 * 200 = 64512 = 384 * 168 registers.
constexpr uint32_t kRegsControl = 104, kRegsSoftmax = 200;
constexpr int kPanelBytes = 128 * 128;  // 128 rows x 64 bf16
constexpr int kMinTiles = 4;
// A unit's beginning and end (queries, first scores, output: 7 to 12 thousand cycles)
// cost about two key tiles (5 thousand each).
using TcTiling = Tiling<kRows, kKeys, 2>;

template <int D>
struct TcCfg {
    static constexpr bool kSepP = D == 64;
    static constexpr uint32_t kColP = 384;
    static constexpr int kPanels = D / 64;
    static constexpr int kTileBytes = kBM * D * 2;
    static constexpr int kStages = D == 64 ? 4 : 2;
    // At d <= 64 the next unit's queries have a place of their own while this one's last
    // scores are formed.
    static constexpr int kQBufs = D == 64 ? 2 : 1;
    static constexpr int kTiles = (2 * kQBufs + 2 * kStages) * kTileBytes;
    static int smem(int R) { return 1024 + kTiles + 1024 + (R * 4 + 15) / 16 * 16; }
    static constexpr size_t kSlotFloats = slot_floats(kRows, D);
};

// A piece of a unit, as warp 0 hands it out (words of one 64-byte slot).
struct Piece {
    int first, c, rows, g;      // the request and cache head
    int q, j0, j1, n;           // row tile; its key tiles j0 .. j1 - 1 of n
    int steps[2], most, tail;   // key tiles that each half of the rows sees, the most of
                                // them (-1: no more pieces), and the one that the
                                // request ends inside (-1: not in this piece)
    int place;                  // of tile j0 on the line
    int r, pad[2];              // row of the block table
};
static_assert(sizeof(Piece) == 64, "a slot");
constexpr int kSlots = 4;  // pieces handed out and not yet done with

struct TcBars {
    uint64_t piece_full[kSlots], piece_free[kSlots];
    uint64_t q_full[2], q_free[2];
    uint64_t k_full[4], v_full[4], k_empty[4], v_empty[4];
    // In turn: up to kStages cleared tiles may be there and not yet waited for.
    uint64_t v_clean[4];
    uint64_t s_full[2], s_free[2], p_full[2], o_done[2];
    uint64_t turn[2][4];
    uint64_t drain;
    uint32_t tmem_base;
    int abort_flag;
    int64_t sums[12];
    alignas(16) Piece pieces[kSlots];
};
static_assert(sizeof(TcBars) <= 1024, "the barriers' region");

__device__ __forceinline__ float as_f(uint32_t u) { return __uint_as_float(u); }
__device__ __forceinline__ uint32_t as_u(float f) { return __float_as_uint(f); }

__device__ __forceinline__ Piece piece_of(const Cursor& k, const FastDiv& by_group, int end) {
    Piece p;
    p.first = k.rq.first;
    p.c = k.rq.c;
    p.rows = k.rq.rows;
    p.g = k.g;
    p.q = k.q;
    p.j0 = k.j;
    p.j1 = min(k.n, k.j + (end - k.f));
    p.n = k.n;
    p.most = 0;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int base = k.q * kRows + t * kBM, rows = max(0, min(kBM, k.rq.rows - base));
        const int n = rows ? (int)(((uint32_t)k.rq.c + by_group.div(base + rows - 1) + kKeys) / kKeys) : 0;
        p.steps[t] = max(0, min(p.j1, n) - p.j0);
        p.most = max(p.most, p.steps[t]);
    }
    const int len = k.rq.c + by_group.div(k.rq.rows), tail = len / kKeys;
    p.tail = (len % kKeys != 0 && tail >= p.j0 && tail < p.j0 + p.most) ? tail : -1;
    p.place = k.f;
    p.r = k.r;
    return p;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    paged_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                    const __grid_constant__ FwdView v, const __nv_bfloat16* __restrict__ P1,
                    __nv_bfloat16* __restrict__ Y, float* __restrict__ L, float* __restrict__ part,
                    PieceMeta* __restrict__ meta) {
    using C = TcCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sQ = smem;
    uint8_t* sK = sQ + 2 * C::kQBufs * C::kTileBytes;
    uint8_t* sV = sK + C::kStages * C::kTileBytes;
    TcBars* bars = reinterpret_cast<TcBars*>(smem + C::kTiles);
    int* prefix = reinterpret_cast<int*>(smem + C::kTiles + 1024);
    const PagedProblem& pp = v.pp;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // The pass before (paged_few.cu) waited for this one's inputs; this one's end waits for it.
    dependency_release();
    if (threadIdx.x == 0) {
        for (int x = 0; x < kSlots; ++x) {
            ptx::mbar_init(&bars->piece_full[x], 1);
            ptx::mbar_init(&bars->piece_free[x], 11);  // the other warps
        }
        for (int x = 0; x < 4; ++x) ptx::mbar_init(&bars->v_clean[x], 1);
        for (int t = 0; t < 2; ++t) {
            ptx::mbar_init(&bars->q_full[t], C::kSepP ? 1 : 4);  // a buffer, or a half
            ptx::mbar_init(&bars->q_free[t], 1);
            ptx::mbar_init(&bars->s_full[t], 1);
            for (int q = 0; q < 4; ++q) ptx::mbar_init(&bars->turn[t][q], 1);
            ptx::mbar_init(&bars->s_free[t], 128);
            ptx::mbar_init(&bars->p_full[t], 128);
            ptx::mbar_init(&bars->o_done[t], 1);
        }
        for (int s = 0; s < C::kStages; ++s) {
            ptx::mbar_init(&bars->k_full[s], 1);
            ptx::mbar_init(&bars->v_full[s], 1);
            ptx::mbar_init(&bars->k_empty[s], 1);
            ptx::mbar_init(&bars->v_empty[s], 1);
        }
        ptx::mbar_init(&bars->drain, 1);
        bars->abort_flag = 0;
        ptx::fence_barrier_init();
        ptx::tma_prefetch_desc(&tm_k);
        ptx::tma_prefetch_desc(&tm_v);
    }
    const int total = schedule_build(v, prefix, bars->sums, [&](const Request& q) {
        return TcTiling::places(q.c, q.rows, pp.by_group, TcTiling::row_tiles(q.rows));
    });
    const int worker = blockIdx.x;
    const Share share(total, (int)gridDim.x, kMinTiles);
    const int lo = share.begin(worker), hi = share.begin(worker + 1);
    if (lo >= hi) {
        if (threadIdx.x == 0) {
            meta[worker] = PieceMeta{};
            dependency_wait();
        }
        return;
    }
    if (warp == 1) {
        ptx::tmem_alloc(&bars->tmem_base, 512);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = bars->tmem_base;
    volatile int* abort_flag = &bars->abort_flag;
    bool ok = true;
    // The other roles' side of the pieces: the slot of piece `seg` once it is there.
    auto take = [&](int seg) -> const Piece* {
        if (!ptx::mbar_wait_warp(&bars->piece_full[seg % kSlots], (seg / kSlots) & 1, abort_flag, v.status,
                                 kDevTimeoutFull)) {
            ok = false;
            return nullptr;
        }
        return &bars->pieces[seg % kSlots];
    };
    auto give = [&](int seg) {
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bars->piece_free[seg % kSlots]);
    };
    // One tensor's tiles of a piece, tile x of the block into stage x % kStages.
    const int box = min(pp.page, kKeys), boxes = kKeys / box;
    int x = 0, tb0 = -1, tb_r = -1, tb = 0;
    auto load = [&](const Piece& pc, const CUtensorMap* map, uint8_t* ring, uint64_t* full, uint64_t* empty) {
        const int need = (pc.c + pp.by_group.div(pc.rows) + pp.page_mask) >> pp.page_shift;
        for (int j = pc.j0; j < pc.j0 + pc.most; ++j, ++x) {
            const int s = x % C::kStages;
            const int tok = j * kKeys, k0 = tok >> pp.page_shift;
            if (pc.r != tb_r || k0 < tb0 || k0 + boxes > tb0 + 32) {
                tb_r = pc.r;
                tb0 = k0;
                tb = 0;
                if (tb0 + lane < need) {
                    tb = __ldg(v.table + (size_t)pc.r * pp.width + tb0 + lane);
                    // Out of range reads as zeros (the map's bound), and is reported.
                    if ((unsigned)tb >= (unsigned)pp.pages) {
                        record_status(v.status, kDevBadPosition);
                        tb = pp.pages;
                    }
                }
            }
            if (x >= C::kStages && !ptx::mbar_wait_warp(&empty[s], ((x / C::kStages) - 1) & 1, abort_flag, v.status,
                                                        kDevTimeoutEmpty)) {
                ok = false;
                return;
            }
            const int copies = C::kPanels * min(boxes, need - k0);
            const int p = lane / C::kPanels, panel = lane % C::kPanels;
            const int page = __shfl_sync(0xffffffffu, tb, (k0 - tb0 + p) & 31);
            if (lane == 0) ptx::mbar_arrive_expect_tx(&full[s], copies * box * 128);
            __syncwarp();
            if (lane < copies)
                ptx::tma_load_4d(ring + s * C::kTileBytes + panel * kPanelBytes + p * box * 128, map, &full[s],
                                 panel * 64, boxes > 1 ? 0 : (tok & pp.page_mask), pc.g, page);
        }
    };
    auto drain = [&](uint64_t* full) {  // after an abort: let the copies already issued land
        if (*abort_flag)
            for (int y = max(0, x - C::kStages); y < x; ++y)
                ptx::mbar_drain(&full[y % C::kStages], (y / C::kStages) & 1, v.status);
    };
    // Query rows r_begin .. r_end - 1 of a piece into buffer qb, by one warp; rows past the
    // unit's are zero.  Eight steps' addresses at a time: one after the other they cost a lone
    // warp 150 cycles each.
    auto load_q = [&](const Piece& pc, int qb, int r_begin, int r_end, uint64_t* full) {
        constexpr int kChunks = D / 8, kStep = 32 / kChunks;  // 16-byte chunks of a row; rows at a time
        const int chunk = lane % kChunks, cols = max(0, min(8, pp.d - chunk * 8));
        const uint32_t q_u = ptx::smem_u32(sQ) + (chunk / 8) * kPanelBytes;
        for (int r0 = r_begin + lane / kChunks; r0 < r_end; r0 += 8 * kStep) {
            const __nv_bfloat16* src[8];
            uint32_t dst[8];
            int bytes[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = r0 + i * kStep, rho = pc.q * kRows + r, rr = r & 127;
                const bool in = rho < pc.rows;
                const int t = in ? pp.by_group.div(rho) : 0, hd = pc.g * pp.group + (in ? rho - t * pp.group : 0);
                src[i] = P1 + ((size_t)(pc.first + t) * pp.H + hd) * pp.d + (cols ? chunk * 8 : 0);
                bytes[i] = in ? cols * 2 : 0;
                dst[i] = q_u + (2 * qb + (r >> 7)) * C::kTileBytes + rr * 128 + (((chunk & 7) ^ (rr & 7)) << 4);
            }
            if ((pp.d & 7) == 0) {
#pragma unroll
                for (int i = 0; i < 8; ++i) cp_async16(dst[i], src[i], bytes[i]);
            } else {  // rows of 120 bytes start on 8
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    cp_async8(dst[i], src[i], min(bytes[i], 8));
                    cp_async8(dst[i] + 8, bytes[i] > 8 ? src[i] + 4 : src[i], max(bytes[i] - 8, 0));
                }
            }
        }
        asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(full);
    };
    if (warp == 0) {
        // --------------------------------------------------------- pieces, P2
        ptx::regs_dec<kRegsControl>();
        Cursor k;
        cursor_seek<TcTiling>(k, v, prefix, lo);
        for (int seg = 0; ok; ++seg) {
            if (seg >= kSlots && !ptx::mbar_wait_warp(&bars->piece_free[seg % kSlots], (seg / kSlots - 1) & 1,
                                                      abort_flag, v.status, kDevTimeoutEmpty))
                break;
            Piece pc{};  // no steps of either half
            pc.most = -1;
            if (k.f < hi) pc = piece_of(k, pp.by_group, hi);
            if (lane == 0) {
                bars->pieces[seg % kSlots] = pc;
                ptx::mbar_arrive(&bars->piece_full[seg % kSlots]);
            }
            __syncwarp();
            if (pc.most < 0) break;
            load(pc, &tm_k, sK, bars->k_full, bars->k_empty);
            k.f += pc.j1 - pc.j0;
            cursor_next_unit<TcTiling>(k, v, prefix, hi);
        }
        drain(bars->k_full);
    } else if (warp == 3) {
        // ------------------------------------------------------------------ I~
        ptx::regs_dec<kRegsControl>();
        int tails = 0;
        for (int seg = 0; ok; ++seg) {
            const Piece* slot = take(seg);
            if (slot == nullptr) break;
            const Piece pc = *slot;
            give(seg);
            if (pc.most < 0) break;
            load(pc, &tm_v, sV, bars->v_full, bars->v_empty);
            if (ok && pc.tail >= 0) {
                // The request ends inside the piece's last tile, the one just sent for: weight 0
                // times whatever its pages hold past the end must be 0.
                const int s = (x - 1) % C::kStages;
                if (!ptx::mbar_wait_warp(&bars->v_full[s], ((x - 1) / C::kStages) & 1, abort_flag, v.status,
                                         kDevTimeoutFull))
                    break;
                uint8_t* tile = sV + s * C::kTileBytes;
                const int len = pc.c + pp.by_group.div(pc.rows);
                for (int r = len - pc.tail * kKeys + lane / 8; r < kKeys; r += 4)
#pragma unroll
                    for (int p = 0; p < C::kPanels; ++p)
                        *reinterpret_cast<uint4*>(tile + p * kPanelBytes + r * 128 + (lane & 7) * 16) =
                            make_uint4(0, 0, 0, 0);
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&bars->v_clean[tails % 4]);
                ++tails;
            }
        }
        drain(bars->v_full);
    } else if (warp == 1) {
        // ------------------------------------------------------------ products
        ptx::regs_dec<kRegsControl>();
        const uint32_t id_s = ptx::idesc_bf16(kBM, kKeys, false, false);
        const uint32_t id_o = ptx::idesc_bf16(kBM, D, false, true);
        const uint64_t dq0 = ptx::smem_desc(ptx::smem_u32(sQ), 16, 1024, ptx::kSwizzle128B);
        const uint64_t dk0 = ptx::smem_desc(ptx::smem_u32(sK), 16, 1024, ptx::kSwizzle128B);
        const uint64_t dv0 = ptx::smem_desc(ptx::smem_u32(sV), kPanelBytes, 1024, ptx::kSwizzle128B);
        // Only a descriptor's low word (the address) changes: an add of a constant a step.
        constexpr uint32_t kTileStep = C::kTileBytes >> 4, kPanelStep = kPanelBytes >> 4;
        auto issue_s = [&](int t, int s, int qb) {
            const uint32_t q_lo = ptx::desc_lo(dq0) + (2 * qb + t) * kTileStep, q_hi = ptx::desc_hi(dq0);
            const uint32_t k_lo = ptx::desc_lo(dk0) + s * kTileStep, k_hi = ptx::desc_hi(dk0);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                const uint32_t off = (ks / 4) * kPanelStep + (ks % 4) * 2;  // 32 bytes per K-step
                ptx::mma_ss_elect(tmem + t * 128, q_lo + off, q_hi, k_lo + off, k_hi, id_s, ks > 0 ? 1u : 0u);
            }
            ptx::mma_commit_elect(&bars->s_full[t]);
        };
        auto issue_pv = [&](int t, int s, bool accumulate) {
            const uint32_t p_col = tmem + (C::kSepP ? C::kColP + 64 * t : 128 * t);
            const uint32_t v_lo = ptx::desc_lo(dv0) + s * kTileStep, v_hi = ptx::desc_hi(dv0);
#pragma unroll
            for (int ks = 0; ks < kKeys / 16; ++ks)  // 16 keys of V per K-step: 2048 bytes of the MN-major tile
                ptx::mma_ts_elect(tmem + 256 + t * D, p_col + ks * 8, v_lo + ks * 128, v_hi, id_o,
                                  (accumulate || ks > 0) ? 1u : 0u);
            ptx::mma_commit_elect(&bars->o_done[t]);
        };
        auto wait = [&](uint64_t* bar, int phase, unsigned code) {
            if (ok) ok = ptx::mbar_wait_warp(bar, phase & 1, abort_flag, v.status, code);
            return ok;
        };
        auto k_wait = [&](int x) { return wait(&bars->k_full[x % C::kStages], x / C::kStages, kDevTimeoutFull); };
        // The queries of a piece (d > 64: of its half t, in the pieces where it has steps).
        int halves[2] = {0, 0};
        auto q_wait = [&](int seg, int t) {
            return C::kSepP ? wait(&bars->q_full[seg % 2], seg / 2, kDevTimeoutFull)
                            : wait(&bars->q_full[t], halves[t]++, kDevTimeoutFull);
        };
        // What of a piece the products need.
        struct Steps {
            int steps[2], most, tail;
        };
        auto read = [&](int seg) {
            Steps x{{0, 0}, -1, -1};
            const Piece* pc = take(seg);
            if (pc != nullptr) {
                x = Steps{{pc->steps[0], pc->steps[1]}, pc->most, pc->tail < 0 ? -1 : pc->tail - pc->j0};
                give(seg);
            }
            return x;
        };
        int kt = 0, tails = 0, st[2] = {0, 0};
        bool begun[2] = {false, false};  // the next piece's first S is already issued
        Steps sg = read(0);
        for (int seg = 0; ok && sg.most >= 0; ++seg) {
            const int qb = seg % C::kQBufs;
            if (!k_wait(kt)) break;
            for (int t = 0; t < 2; ++t) {
                if (sg.steps[t] == 0 || begun[t]) continue;
                if (!q_wait(seg, t)) break;
                // S of the piece before has been read (d > 64: its P V, issued before, read it).
                if (C::kSepP && st[t] > 0 && !wait(&bars->s_free[t], st[t] - 1, kDevTimeoutFull)) break;
                ptx::tc_fence_after();
                issue_s(t, kt % C::kStages, qb);
            }
            begun[0] = begun[1] = false;
            if (!ok) break;
            ptx::mma_commit_elect(&bars->k_empty[kt % C::kStages]);
            if (C::kSepP && sg.most == 1) ptx::mma_commit_elect(&bars->q_free[qb]);
            Steps next{{0, 0}, -2, -1};  // not read yet
            for (int j = 0; ok && j < sg.most; ++j) {
                const int s = (kt + j) % C::kStages;
                bool v_ready = false;
                auto v_wait = [&]() {
                    if (v_ready) return true;
                    v_ready = j == sg.tail ? wait(&bars->v_clean[tails % 4], tails / 4, kDevTimeoutFull)
                                           : wait(&bars->v_full[s], (kt + j) / C::kStages, kDevTimeoutFull);
                    return v_ready;
                };
                if constexpr (C::kSepP) {
                    // Each half's next S once the softmax holds this one, past the piece's end too,
                    // and its P V: one half after the other, so that they settle half a step apart
                    // and neither waits for the other's.
                    for (int t = 0; t < 2 && ok; ++t) {
                        if (j >= sg.steps[t]) continue;
                        if (!wait(&bars->s_free[t], st[t] + j, kDevTimeoutFull)) break;
                        if (j + 1 < sg.steps[t]) {
                            if (!k_wait(kt + j + 1)) break;
                            ptx::tc_fence_after();
                            issue_s(t, (kt + j + 1) % C::kStages, qb);
                        } else {
                            if (next.most == -2) next = read(seg + 1);
                            if (!ok) break;
                            if (next.steps[t] > 0) {
                                if (!q_wait(seg + 1, t) || !k_wait(kt + sg.most)) break;
                                ptx::tc_fence_after();
                                issue_s(t, (kt + sg.most) % C::kStages, (seg + 1) % C::kQBufs);
                                begun[t] = true;
                            }
                        }
                        if (!wait(&bars->p_full[t], st[t] + j, kDevTimeoutFull) || !v_wait()) break;
                        ptx::tc_fence_after();
                        issue_pv(t, s, j > 0);
                    }
                    if (ok && j + 1 < sg.most) ptx::mma_commit_elect(&bars->k_empty[(kt + j + 1) % C::kStages]);
                    if (ok && j + 2 == sg.most) ptx::mma_commit_elect(&bars->q_free[qb]);
                } else {
                    for (int t = 0; t < 2 && ok; ++t) {
                        if (j >= sg.steps[t]) continue;
                        if (!wait(&bars->p_full[t], st[t] + j, kDevTimeoutFull) || !v_wait()) break;
                        ptx::tc_fence_after();
                        issue_pv(t, s, j > 0);
                        if (j + 1 < sg.steps[t]) {
                            if (!k_wait(kt + j + 1)) break;
                            ptx::tc_fence_after();
                            issue_s(t, (kt + j + 1) % C::kStages, qb);
                        }
                    }
                    if (ok && j + 1 < sg.most) ptx::mma_commit_elect(&bars->k_empty[(kt + j + 1) % C::kStages]);
                }
                if (ok) ptx::mma_commit_elect(&bars->v_empty[s]);
            }
            if (ok && next.most == -2) next = read(seg + 1);
            kt += sg.most;
            tails += sg.tail >= 0;
            st[0] += sg.steps[0];
            st[1] += sg.steps[1];
            sg = next;
        }
        ptx::mma_commit_elect(&bars->drain);
        ptx::mbar_drain(&bars->drain, 0, v.status);
    } else if (warp == 2) {
        // ------------------------------------------------------------- queries
        ptx::regs_dec<kRegsControl>();
        PieceMeta mine{};
        for (int seg = 0; ok; ++seg) {
            const Piece* slot = take(seg);
            if (slot == nullptr) break;
            const Piece pc = *slot;
            give(seg);
            if (pc.most < 0) break;
            if constexpr (C::kSepP) {
                const int qb = seg % C::kQBufs;
                if (seg >= C::kQBufs && !ptx::mbar_wait_warp(&bars->q_free[qb], (seg / C::kQBufs - 1) & 1, abort_flag,
                                                             v.status, kDevTimeoutEmpty)) {
                    ok = false;
                    break;
                }
                load_q(pc, qb, 0, pc.rows - pc.q * kRows > kBM ? 2 * kBM : kBM, &bars->q_full[qb]);
            }
            if (pc.j0 == 0 && pc.j1 < pc.n)
                mine = PieceMeta{share.owner(pc.place + pc.n - 1) - worker + 1, pc.first, pc.c, pc.rows, pc.g, pc.q};
        }
        if (lane == 0) meta[worker] = ok ? mine : PieceMeta{};
    } else {
        // ------------------------------------------------------------- softmax
        ptx::regs_inc<kRegsSoftmax>();
        const int t = (warp - 4) >> 2, quarter = warp & 3, r = quarter * 32 + lane;
        const uint32_t lane_addr = tmem + ((uint32_t)(quarter * 32) << 16);
        const uint32_t s_col = t * 128, o_col = 256 + t * D;
        const float c_half = 0.5f * pp.inv_sqrt_d;                // U/2 per raw dot product
        const float c_diag = 0.5f * pp.inv_sqrt_d / pp.tau_S;     // U/(2 tau_S)
        uint64_t* turn_mine = &bars->turn[t][quarter];
        uint64_t* turn_next = &bars->turn[t ^ 1][quarter];
        int st = 0, pairs = 0;  // steps of this half, and steps both halves took in turn
        // d > 64: this warp's 32 query rows of piece seg, once this half's last scores of the piece
        // before are there, so nothing reads its queries any more.
        auto next_q = [&](int seg) {
            if (C::kSepP || !ok) return;
            const Piece* pc = take(seg);
            if (pc != nullptr && pc->steps[t] > 0)
                load_q(*pc, 0, t * kBM + quarter * 32, t * kBM + quarter * 32 + 32, &bars->q_full[t]);
        };
        next_q(0);
        for (int seg = 0; ok; ++seg) {
            const Piece* pc = take(seg);  // the slot stays this warp's until the piece is done
            if (pc == nullptr || pc->most < 0) break;
            const int steps = pc->steps[t], n_pair = C::kSepP ? 0 : min(pc->steps[0], pc->steps[1]);
            // The row's own token (the last key it sees) as a column of the piece's first
            // tile, the warp's least and greatest.
            int own = pc->c + pp.by_group.div(min(pc->q * kRows + t * kBM + r, pc->rows - 1));
            const float corr = pp.lambda * __logf((float)(own + 1));
            own -= pc->j0 * kKeys;
            int own_lo = __shfl_sync(0xffffffffu, own, 0), own_hi = __shfl_sync(0xffffffffu, own, 31);
            // The row's reference and the sum of its weights under it.  SiLU is above -0.28, and the first
            // row's Self, which has no correction, above 0: no row's sum vanishes under the reference 0.
            // It rises when a score passes it by 2^kRaise.
            float m = 0.f, l = 0.f;
            bool o_ready = false;  // O and P are free of this tile's predecessors
            auto o_wait = [&](int j) {
                if (o_ready) return;
                o_ready = true;
                if (j == 0) return;
                if (!ptx::mbar_wait_warp(&bars->o_done[t], (st + j - 1) & 1, abort_flag, v.status, kDevTimeoutMma))
                    ok = false;
                ptx::tc_fence_after();
            };
            const uint32_t p_addr = lane_addr + (C::kSepP ? C::kColP + 64 * t : s_col);
            auto scale_pairs = [](uint32_t& w, float f) {
                const float2 x = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
                w = ptx::pack_bf16x2(x.x * f, x.y * f);
            };
            // The reference rises to m_new in block b of tile j (seldom): what has been summed under the
            // old one is scaled, in O, in l and in this tile's P so far.
            auto raise = [&](float m_new, int j, int b) {
                const float f = ptx::ex2_approx((m - m_new) * kLog2e);
                l *= f;
                m = m_new;
                o_wait(j);
                if (j > 0) {
#pragma unroll 1
                    for (int c0 = 0; c0 < D / 32; ++c0) {
                        uint32_t ov[32];
                        ptx::tmem_ld32(lane_addr + o_col + 32 * c0, ov);
                        ptx::tmem_ld_wait();
                        ptx::pin_regs(ov);
#pragma unroll
                        for (int e = 0; e < 32; ++e) ov[e] = as_u(as_f(ov[e]) * f);
                        ptx::tmem_st32(lane_addr + o_col + 32 * c0, ov);
                    }
                }
                ptx::tmem_st_wait();
#pragma unroll 1
                for (int x = 0; x < b; ++x) {
                    uint32_t pv[16];
                    ptx::tmem_ld16(p_addr + 16 * x, pv);
                    ptx::tmem_ld_wait();
                    ptx::pin_regs(pv);
#pragma unroll
                    for (int e = 0; e < 16; ++e) scale_pairs(pv[e], f);
                    ptx::tmem_st16(p_addr + 16 * x, pv);
                }
            };
            const float2 ch2 = make_float2(c_half, c_half), l2e2 = make_float2(kLog2e, kLog2e);
            // Two scores -> R (left in their place), and their weights under the reference.
            auto pair = [&](uint32_t& s0, uint32_t& s1, float2 nm2, float2& sum) {
                const float2 h = ptx::mul2(make_float2(as_f(s0), as_f(s1)), ch2);
                const float2 th = make_float2(ptx::tanh_approx(h.x), ptx::tanh_approx(h.y));
                const float2 E = ptx::fma2(h, th, h);  // SiLU(U) = (U/2)(1 + tanh(U/2))
                const float2 y = ptx::fma2(E, l2e2, nm2);
                const float2 p = make_float2(ptx::ex2_approx(y.x), ptx::ex2_approx(y.y));
                s0 = as_u(E.x), s1 = as_u(E.y);
                sum = ptx::add2(sum, p);
                return ptx::pack_bf16x2(p.x, p.y);
            };
            // 32 scores -> the weights of columns 32 b and on, and what they add to the row's sum.
            auto block = [&](uint32_t (&sv)[32], uint32_t (&pk)[16], int j, int b) {
                const int c0 = 32 * b;
                if (c0 > own_hi) {  // past every row's own token
#pragma unroll
                    for (int e = 0; e < 16; ++e) pk[e] = 0u;
                    return;
                }
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                if (c0 + 31 < own_lo) {
                    // Before every row's own token: both functions in one run, under the reference so
                    // far, with no wait for the maximum between them.
                    const float2 nm2 = make_float2(-m * kLog2e, -m * kLog2e);
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        pk[e] = pair(sv[2 * e], sv[2 * e + 1], nm2, ls[e & 1]);
                        mx[e & 3] = ptx::max3(mx[e & 3], as_f(sv[2 * e]), as_f(sv[2 * e + 1]));
                    }
                    const float m_new = fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
                    if (!__any_sync(0xffffffffu, m_new > m + kRaise * kLn2)) {
                        const float2 sum = ptx::add2(ls[0], ls[1]);
                        l += sum.x + sum.y;
                        return;
                    }
                    raise(m_new, j, b);
                } else {
                    float self = 0.f;
#pragma unroll
                    for (int c = 0; c < 32; ++c) self = c0 + c == own ? as_f(sv[c]) : self;
                    self = fmaf(0.5f, ptx::tanh_approx(self * c_diag), 0.5f) + corr;
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        const float h = as_f(sv[c]) * c_half;
                        const float x = c0 + c > own ? -INFINITY : fmaf(h, ptx::tanh_approx(h), h);
                        sv[c] = as_u(c0 + c == own ? self : x);
                    }
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        mx[e & 3] = ptx::max3(mx[e & 3], as_f(sv[2 * e]), as_f(sv[2 * e + 1]));
                    const float m_new = fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
                    if (__any_sync(0xffffffffu, m_new > m + kRaise * kLn2)) raise(m_new, j, b);
                }
                const float2 nm2 = make_float2(-m * kLog2e, -m * kLog2e);
                ls[0] = ls[1] = make_float2(0.f, 0.f);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float2 y = ptx::fma2(make_float2(as_f(sv[2 * e]), as_f(sv[2 * e + 1])), l2e2, nm2);
                    const float2 p = make_float2(ptx::ex2_approx(y.x), ptx::ex2_approx(y.y));
                    ls[e & 1] = ptx::add2(ls[e & 1], p);
                    pk[e] = ptx::pack_bf16x2(p.x, p.y);
                }
                const float2 sum = ptx::add2(ls[0], ls[1]);
                l += sum.x + sum.y;
            };
            // A tile, 32 columns at a time in a loop, not 128 in a row: its code stays in the instruction
            // caches (whole prompts, heads of 64: 0.36 ms, unrolled 0.41).
            auto blocks = [&](int j) {
#pragma unroll 1
                for (int b = 0; b < 4; ++b) {
                    uint32_t sv[32], pk[16];
                    ptx::tmem_ld32(lane_addr + s_col + 32 * b, sv);
                    ptx::tmem_ld_wait();
                    ptx::pin_regs(sv);
                    if (C::kSepP && b == 3) {  // the next S may overwrite it
                        ptx::tc_fence_before();
                        ptx::mbar_arrive(&bars->s_free[t]);
                    }
                    block(sv, pk, j, b);
                    if (C::kSepP && b == 0) o_wait(j);  // P V of the tile before has read its P
                    ptx::tmem_st16(p_addr + 16 * b, pk);
                }
            };
            for (int j = 0; ok && j < steps; ++j) {
                o_ready = false;
                if (!ptx::mbar_wait_warp(&bars->s_full[t], (st + j) & 1, abort_flag, v.status, kDevTimeoutMma)) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
                if constexpr (C::kSepP) {
                    blocks(j);
                } else {
                    // The 128 columns at once where every row's own token is past them.
                    bool whole = own_lo >= kKeys;
                    const int x = pairs + j;
                    auto take_turn = [&] {
                        return j >= n_pair || x + t == 0 ||
                               ptx::mbar_wait_warp(turn_mine, (x + t - 1) & 1, abort_flag, v.status, kDevTimeoutMma);
                    };
                    if (whole) {
                        uint32_t sv[128], pk[2][32];
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            ptx::tmem_ld32(lane_addr + s_col + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(sv + 32 * c));
                        ptx::tmem_ld_wait();
                        ptx::pin_regs(sv);
                        if (!take_turn()) {
                            ok = false;
                            break;
                        }
                        ptx::pin_regs(sv);  // the run below starts after the turn is taken
                        const float2 nm2 = make_float2(-m * kLog2e, -m * kLog2e);
                        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                        float2 ls[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                                        make_float2(0.f, 0.f)};
#pragma unroll
                        for (int e = 0; e < 64; ++e) {
                            pk[e >> 5][e & 31] = pair(sv[2 * e], sv[2 * e + 1], nm2, ls[e & 3]);
                            mx[e & 3] = ptx::max3(mx[e & 3], as_f(sv[2 * e]), as_f(sv[2 * e + 1]));
                        }
                        const float m_new = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                        whole = !__any_sync(0xffffffffu, m_new > m + kRaise * kLn2);
                        if (whole) {
                            const float2 sum = ptx::add2(ptx::add2(ls[0], ls[1]), ptx::add2(ls[2], ls[3]));
                            l += sum.x + sum.y;
                            ptx::pin_regs(pk[0]);  // and ends before it is passed on
                            ptx::pin_regs(pk[1]);
                            __syncwarp();
                            if (j < n_pair && lane == 0) ptx::mbar_arrive(turn_next);
                            ptx::tmem_st32(p_addr, pk[0]);
                            ptx::tmem_st32(p_addr + 32, pk[1]);
                        }
                    } else if (!take_turn()) {
                        ok = false;
                        break;
                    }
                    if (!whole) {  // S is still there
                        blocks(j);
                        __syncwarp();
                        if (j < n_pair && lane == 0) ptx::mbar_arrive(turn_next);
                    }
                }
                if (!ok) break;
                own -= kKeys;
                own_lo -= kKeys;
                own_hi -= kKeys;
                ptx::tmem_st_wait();
                ptx::tc_fence_before();
                ptx::mbar_arrive(&bars->p_full[t]);
            }
            next_q(seg + 1);
            if (ok && steps > 0) {
                ok = ptx::mbar_wait_warp(&bars->o_done[t], (st + steps - 1) & 1, abort_flag, v.status, kDevTimeoutMma);
                ptx::tc_fence_after();
            }
            const int row = pc->q * kRows + t * kBM + r, rows = pc->rows;  // row: of the request
            if (ok && row - r < rows) {
                const bool direct = pc->j0 == 0 && pc->j1 == pc->n, mine = row < rows;
                const int rho = min(row, rows - 1), token = pp.by_group.div(rho);
                const size_t yr = (size_t)(pc->first + token) * pp.H + pc->g * pp.group + (rho - token * pp.group);
                float* slot = part + ((size_t)worker * 2 + (pc->j0 == 0 ? 1 : 0)) * C::kSlotFloats;
                const float inv = direct ? 1.f / l : 1.f;
#pragma unroll
                for (int c0 = 0; c0 < D / 32; ++c0) {
                    if (steps == 0 || 32 * c0 >= pp.d) break;  // columns past the head width are zero padding
                    uint32_t ov[32];
                    ptx::tmem_ld32(lane_addr + o_col + 32 * c0, ov);
                    ptx::tmem_ld_wait();
                    ptx::pin_regs(ov);
                    if (direct && mine) {
                        uint32_t w[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            w[e] = ptx::pack_bf16x2(as_f(ov[2 * e]) * inv, as_f(ov[2 * e + 1]) * inv);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            store_bf16x8(Y + yr * pp.d, 32 * c0 + 8 * e, pp.d, w[4 * e], w[4 * e + 1], w[4 * e + 2],
                                         w[4 * e + 3]);
                    } else if (!direct) {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            *reinterpret_cast<float4*>(slot + (size_t)(t * kBM + r) * D + 32 * c0 + 4 * e) =
                                make_float4(as_f(ov[4 * e]), as_f(ov[4 * e + 1]), as_f(ov[4 * e + 2]),
                                            as_f(ov[4 * e + 3]));
                    }
                }
                if (!direct)
                    *reinterpret_cast<float2*>(slot + (size_t)kRows * D + 2 * (t * kBM + r)) =
                        make_float2(piece_max(pc->c + token >= pc->j0 * kKeys, m * kLog2e), l);
                else if (L != nullptr && mine)
                    L[yr] = m + __log2f(l) * kLn2 - corr;
            }
            st += steps;
            pairs += n_pair;
            give(seg);
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
    if (threadIdx.x == 0) dependency_wait();
}

template <int D>
size_t tc_bytes(int num_sms) {
    return num_sms * (sizeof(PieceMeta) + 8 + 2 * TcCfg<D>::kSlotFloats * sizeof(float));
}

template <int D>
cudaError_t launch_tc(const PagedProblem& pp, const PagedFwdArgs& a, void* ws, const MergeSide& few, cudaStream_t s) {
    using C = TcCfg<D>;
    static_assert(1024 + C::kTiles + 1024 + kPagedMaxRequests * 4 <= 232448, "shared memory of a block");
    static OncePerDevice once;
    cudaError_t e = allow_dynamic_smem(once, paged_tc_kernel<D>, C::smem(kPagedMaxRequests));
    if (e != cudaSuccess) return e;
    const FwdView v{pp, a.table, a.starts, a.cached, a.max_fresh, kPagedFewRows, INT32_MAX, a.status};
    const int workers = a.num_sms;
    float* part = static_cast<float*>(ws);
    PieceMeta* meta = reinterpret_cast<PieceMeta*>(part + (size_t)workers * 2 * C::kSlotFloats);
    CUtensorMap mk, mv;
    const int box = std::min(pp.page, kKeys);
    if ((e = make_page_map(&mk, a.P2_pages, pp, box)) != cudaSuccess) return e;
    if ((e = make_page_map(&mv, a.I_pages, pp, box)) != cudaSuccess) return e;
    e = launch_chained(paged_tc_kernel<D>, dim3((unsigned)workers), kThreads, C::smem(pp.R), s, mk, mv, v,
                       (const __nv_bfloat16*)a.P1, (__nv_bfloat16*)a.Y, a.L, part, meta);
    if (e != cudaSuccess) return e;
    return launch_merge<__nv_bfloat16, kPagedFewRows, kRows, D>(v, few, MergeSide{part, meta, workers}, a.Y, a.L, s);
}

}  // namespace
}  // namespace paged

size_t paged_tc_workspace(const PagedProblem& pp, int num_sms) {
    return pp.d <= 64 ? paged::tc_bytes<64>(num_sms) : paged::tc_bytes<128>(num_sms);
}

cudaError_t launch_paged_tc(const PagedProblem& pp, const PagedFwdArgs& a, void* workspace,
                            const paged::MergeSide& few, cudaStream_t s) {
    return pp.d <= 64 ? paged::launch_tc<64>(pp, a, workspace, few, s) : paged::launch_tc<128>(pp, a, workspace, few, s);
}

}  // namespace relation
