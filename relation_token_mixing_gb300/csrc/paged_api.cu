// Host side of the paged Relation Cache entry points (include/relation.h):
// argument checks and dispatch.
#include <math.h>
#include <stdint.h>

#include "api_internal.h"
#include "paged.h"

namespace relation {
namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

struct Span {
    const void* p;
    size_t n;
};

bool overlap(const Span& a, const Span& b) {
    if (a.p == nullptr || b.p == nullptr || a.n == 0 || b.n == 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x < y + b.n && y < x + a.n;
}

// Every output apart from every input and every other output.
bool disjoint(const Span* in, int n_in, const Span* out, int n_out) {
    for (int o = 0; o < n_out; ++o) {
        for (int i = 0; i < n_in; ++i)
            if (overlap(out[o], in[i])) return false;
        for (int q = o + 1; q < n_out; ++q)
            if (overlap(out[o], out[q])) return false;
    }
    return true;
}

size_t elem(const relation_paged_t* p) { return p->dtype == RELATION_BF16 ? 2 : 4; }

// Cached rows start on 16 bytes.
int64_t row_elems(const relation_paged_t* p) { return p->dtype == RELATION_BF16 ? (p->d_h + 7) / 8 * 8 : p->d_h; }

size_t heads_bytes(const relation_paged_t* p, int64_t heads) {
    return (size_t)p->N * (size_t)heads * (size_t)p->d_h * elem(p);
}
size_t pages_bytes(const relation_paged_t* p) {
    return (size_t)p->pages * (size_t)p->page_size * (size_t)p->G * (size_t)row_elems(p) * elem(p);
}

relation_status_t check_paged(const relation_paged_t* p) {
    if (p == nullptr) return RELATION_ERR_INVALID_ARGUMENT;
    if (p->R < 1 || p->R > (1 << 20) || p->N < 0 || p->N > (int64_t)INT32_MAX) return RELATION_ERR_INVALID_ARGUMENT;
    if (p->H < 1 || p->H > 1024 || p->G < 1 || p->G > p->H || p->H % p->G != 0) return RELATION_ERR_INVALID_ARGUMENT;
    if (p->d_h < 1 || p->d_h > 1024) return p->d_h < 1 ? RELATION_ERR_INVALID_ARGUMENT : RELATION_ERR_UNSUPPORTED;
    if (p->pages < 1 || p->pages > (int64_t)INT32_MAX || p->page_size < 1 || p->page_size > (int64_t)INT32_MAX ||
        p->table_width < 1 || p->table_width > (int64_t)INT32_MAX ||
        p->table_width * p->page_size > (int64_t)INT32_MAX)
        return RELATION_ERR_INVALID_ARGUMENT;
    if (p->dtype != RELATION_F32 && p->dtype != RELATION_BF16) return RELATION_ERR_INVALID_ARGUMENT;
    if (p->layout != RELATION_LAYOUT_BHTD && p->layout != RELATION_LAYOUT_BTHD) return RELATION_ERR_INVALID_ARGUMENT;
    if (!(p->tau_S > 0.f) || !isfinite(p->tau_S) || !isfinite(p->lambda)) return RELATION_ERR_INVALID_ARGUMENT;
    if ((double)p->N * (double)p->H * (double)p->d_h > 1e12 ||
        (double)p->pages * (double)p->page_size * (double)p->G * (double)row_elems(p) > 1e12)
        return RELATION_ERR_INVALID_ARGUMENT;
    if (p->page_size < 16 || p->page_size > 256 || (p->page_size & (p->page_size - 1)) != 0)
        return RELATION_ERR_UNSUPPORTED;
    if (p->d_h != 48 && p->d_h != 60 && p->d_h != 64 && p->d_h != 80 && p->d_h != 128) return RELATION_ERR_UNSUPPORTED;
    return RELATION_OK;
}

PagedProblem paged_problem(const relation_paged_t* p) {
    PagedProblem pp;
    pp.R = (int)p->R;
    pp.N = (int)p->N;
    pp.H = (int)p->H;
    pp.G = (int)p->G;
    pp.group = (int)(p->H / p->G);
    pp.by_group = FastDiv((uint32_t)pp.group);
    pp.by_G = FastDiv((uint32_t)pp.G);
    pp.d = (int)p->d_h;
    pp.row = (int)row_elems(p);
    pp.pages = (int)p->pages;
    pp.page = (int)p->page_size;
    pp.page_shift = 0;
    while ((1 << pp.page_shift) < pp.page) ++pp.page_shift;
    pp.page_mask = pp.page - 1;
    pp.width = (int)p->table_width;
    pp.tau_S = p->tau_S;
    pp.lambda = p->lambda;
    pp.inv_sqrt_d = (float)(1.0 / sqrt((double)p->d_h));
    pp.layout = (int)p->layout;
    return pp;
}

relation_status_t from_cuda(cudaError_t e) { return e == cudaSuccess ? RELATION_OK : RELATION_ERR_CUDA; }

// The bound the forward works with: max_fresh, or N when none is known.
int fresh_bound(const relation_paged_t* p, int max_fresh) {
    return max_fresh == 0 || (int64_t)max_fresh > p->N ? (int)p->N : max_fresh;
}

// A request's packed rows are counted in 32 bits, in row tiles of up to 256.
bool rows_fit(const relation_paged_t* p, int max_fresh) {
    return (int64_t)fresh_bound(p, max_fresh) * (p->H / p->G) <= (int64_t)INT32_MAX - 255;
}

}  // namespace
}  // namespace relation

using namespace relation;

extern "C" {

relation_status_t relation_paged_plan(const relation_paged_t* p, const int32_t* cached, const int32_t* fresh,
                                      const int32_t* free_pages, size_t free_count, int32_t* block_table,
                                      int32_t* starts, int64_t* slots, int32_t* positions, int32_t* used,
                                      void* stream) {
    relation_status_t st = check_paged(p);
    if (st != RELATION_OK) return st;
    if (free_count > (size_t)INT32_MAX) return RELATION_ERR_INVALID_ARGUMENT;
    if (cached == nullptr || fresh == nullptr || block_table == nullptr || starts == nullptr || used == nullptr ||
        (free_count > 0 && free_pages == nullptr) || (p->N > 0 && (slots == nullptr || positions == nullptr)))
        return RELATION_ERR_INVALID_ARGUMENT;
    for (const void* x : {(const void*)cached, (const void*)fresh, (const void*)free_pages, (const void*)starts,
                          (const void*)used})
        if (!aligned(x, 4)) return RELATION_ERR_MISALIGNED;
    for (const void* x : {(const void*)block_table, (const void*)slots, (const void*)positions})
        if (!aligned(x, 16)) return RELATION_ERR_MISALIGNED;
    const size_t R = (size_t)p->R, N = (size_t)p->N;
    const Span in[] = {{cached, R * 4}, {fresh, R * 4}, {free_pages, free_count * 4}};
    const Span out[] = {{block_table, R * (size_t)p->table_width * 4}, {starts, (R + 1) * 4}, {slots, N * 8},
                        {positions, N * 4}, {used, 4}};
    if (!disjoint(in, 3, out, 5)) return RELATION_ERR_INVALID_ARGUMENT;
    unsigned int* status;
    int sms;
    if ((st = api_device(&status, &sms)) != RELATION_OK) return st;
    st = from_cuda(launch_paged_plan(paged_problem(p), cached, fresh, free_pages, (int64_t)free_count, block_table,
                                     starts, slots, positions, used, status, static_cast<cudaStream_t>(stream)));
    if (st == RELATION_OK) api_set_launches(1);
    return st;
}

relation_status_t relation_paged_store(const relation_paged_t* p, const void* X1, const void* X2, const void* I,
                                       const float* theta, int pairing, float rope_base, const int32_t* positions,
                                       const int64_t* slots, void* P1, void* P2_pages, void* I_pages, void* stream) {
    relation_status_t st = check_paged(p);
    if (st != RELATION_OK) return st;
    if ((pairing != 0 && pairing != 1) || !isfinite(rope_base) || (theta != nullptr && p->G % 2 != 0))
        return RELATION_ERR_INVALID_ARGUMENT;
    if (p->N == 0) {
        api_set_launches(0);
        return RELATION_OK;
    }
    const void* ptrs[] = {X1, X2, I, positions, slots, P1, P2_pages, I_pages};
    for (const void* x : ptrs)
        if (x == nullptr) return RELATION_ERR_INVALID_ARGUMENT;
    for (const void* x : ptrs)
        if (!aligned(x, 16)) return RELATION_ERR_MISALIGNED;
    if (!aligned(theta, 4)) return RELATION_ERR_MISALIGNED;
    const size_t N = (size_t)p->N, hb = heads_bytes(p, p->H), gb = heads_bytes(p, p->G), cb = pages_bytes(p);
    const Span in[] = {{X1, hb}, {X2, gb}, {I, gb}, {positions, N * 4}, {slots, N * 8},
                       {theta, theta ? (size_t)(p->G / 2) * 4 : 0}};
    const Span out[] = {{P1, hb}, {P2_pages, cb}, {I_pages, cb}};
    if (!disjoint(in, 6, out, 3)) return RELATION_ERR_INVALID_ARGUMENT;
    unsigned int* status;
    int sms;
    if ((st = api_device(&status, &sms)) != RELATION_OK) return st;
    // The last table made on this thread is kept: a program has one (d_h, base).
    static thread_local RopeTable tab{};
    static thread_local int tab_d = 0;
    static thread_local float tab_base = 0.f;
    if (tab_d != (int)p->d_h || tab_base != rope_base) {
        tab = rope_table((int)p->d_h, rope_base);
        tab_d = (int)p->d_h;
        tab_base = rope_base;
    }
    st = from_cuda(launch_paged_store(paged_problem(p), p->dtype == RELATION_BF16, X1, X2, I, theta, pairing, tab,
                                      positions, slots, P1, P2_pages, I_pages, status, sms,
                                      static_cast<cudaStream_t>(stream)));
    if (st == RELATION_OK) api_set_launches(1);
    return st;
}

size_t relation_paged_workspace_bytes(const relation_paged_t* p, int max_fresh) {
    if (check_paged(p) != RELATION_OK || max_fresh < 0 || p->R > kPagedMaxRequests || !rows_fit(p, max_fresh)) return 0;
    unsigned int* status;
    int sms;
    if (api_device(&status, &sms) != RELATION_OK) return 0;
    return paged_fwd_workspace(paged_problem(p), p->dtype == RELATION_BF16, fresh_bound(p, max_fresh), sms);
}

relation_status_t relation_paged_fwd(const relation_paged_t* p, const void* P1, const void* P2_pages,
                                     const void* I_pages, const int32_t* block_table, const int32_t* starts,
                                     const int32_t* cached, int max_fresh, void* Y, float* L, void* workspace,
                                     size_t workspace_bytes, void* stream) {
    relation_status_t st = check_paged(p);
    if (st != RELATION_OK) return st;
    if (p->R > kPagedMaxRequests) return RELATION_ERR_UNSUPPORTED;
    if (max_fresh < 0) return RELATION_ERR_INVALID_ARGUMENT;
    if (!rows_fit(p, max_fresh)) return RELATION_ERR_UNSUPPORTED;
    if (p->N == 0) {
        api_set_launches(0);
        return RELATION_OK;
    }
    const void* ptrs[] = {P1, P2_pages, I_pages, block_table, starts, cached, Y, workspace};
    for (const void* x : ptrs)
        if (x == nullptr) return RELATION_ERR_INVALID_ARGUMENT;
    for (const void* x : {P1, P2_pages, I_pages, (const void*)block_table, (const void*)Y, (const void*)workspace})
        if (!aligned(x, 16)) return RELATION_ERR_MISALIGNED;
    for (const void* x : {(const void*)starts, (const void*)cached, (const void*)L})
        if (!aligned(x, 4)) return RELATION_ERR_MISALIGNED;
    const size_t N = (size_t)p->N, R = (size_t)p->R, hb = heads_bytes(p, p->H), cb = pages_bytes(p);
    unsigned int* status;
    int sms;
    if ((st = api_device(&status, &sms)) != RELATION_OK) return st;
    const PagedProblem pp = paged_problem(p);
    const bool bf16 = p->dtype == RELATION_BF16;
    PagedFwdArgs a{P1, P2_pages, I_pages, block_table, starts, cached, fresh_bound(p, max_fresh), Y, L, workspace,
                   status, sms};
    const size_t need = paged_fwd_workspace(pp, bf16, a.max_fresh, sms);
    if (workspace_bytes < need) return RELATION_ERR_WORKSPACE_TOO_SMALL;
    const Span in[] = {{P1, hb}, {P2_pages, cb}, {I_pages, cb}, {block_table, R * (size_t)p->table_width * 4},
                       {starts, (R + 1) * 4}, {cached, R * 4}};
    const Span out[] = {{Y, hb}, {L, L ? N * (size_t)p->H * 4 : 0}, {workspace, need}};
    if (!disjoint(in, 6, out, 3)) return RELATION_ERR_INVALID_ARGUMENT;
    int launches = 0;
    st = from_cuda(launch_paged_fwd(pp, bf16, a, &launches, static_cast<cudaStream_t>(stream)));
    if (st == RELATION_OK) api_set_launches(launches);
    return st;
}

}  // extern "C"
