// Paged Relation Cache: kernel-side problem and internal launch functions.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "kernels.h"
#include "paged_schedule.cuh"

namespace relation {

// Kernel-side view of one relation_paged_t.
struct PagedProblem {
    int R, N, H, G;
    int group;  // H / G: Relation heads of one cache head
    FastDiv by_group, by_G;
    int d;      // head width
    int row;    // elements from one cached row to the next
    int pages, page, page_shift, page_mask;
    int width;  // block-table entries of a request
    float tau_S, lambda, inv_sqrt_d;
    int layout;
};

// Element offset of a cached row: token `off` of a page, cache head g.
__host__ __device__ __forceinline__ size_t page_row_offset(const PagedProblem& pp, int64_t page, int off, int g) {
    const int64_t r = pp.layout == 0 ? (page * pp.G + g) * pp.page + off : (page * pp.page + off) * pp.G + g;
    return (size_t)r * (size_t)pp.row;
}

// Requests the forward's schedule holds in shared memory.
constexpr int kPagedMaxRequests = 8192;

cudaError_t launch_paged_plan(const PagedProblem& pp, const int* cached, const int* fresh, const int* free_pages,
                              int64_t free_count, int* table, int* starts, int64_t* slots, int* positions, int* used,
                              unsigned int* status, cudaStream_t s);

cudaError_t launch_paged_store(const PagedProblem& pp, bool bf16, const void* X1, const void* X2, const void* I,
                               const float* theta, int pairing, const RopeTable& tab, const int* positions,
                               const int64_t* slots, void* P1, void* P2_pages, void* I_pages, unsigned int* status,
                               int num_sms, cudaStream_t s);

struct PagedFwdArgs {
    const void *P1, *P2_pages, *I_pages;
    const int *table, *starts, *cached;
    int max_fresh;
    void* Y;
    float* L;
    void* workspace;
    unsigned int* status;
    int num_sms;
};
// Workspace bytes and launches of one forward.
size_t paged_fwd_workspace(const PagedProblem& pp, bool bf16, int max_fresh, int num_sms);
cudaError_t launch_paged_fwd(const PagedProblem& pp, bool bf16, const PagedFwdArgs& a, int* launches, cudaStream_t s);

}  // namespace relation
