// Which kernels a paged forward runs.
//
// bf16: requests of at most kPagedFewRows = 16 packed rows (new tokens times the heads
// of a group) go to the kernel whose bound is the history's bytes, longer ones to the
// tensor-core kernel whose bound is the scores' special functions; each kernel
// passes over the other's requests, and the second is launched only where the
// host's bound on the new tokens lets a request be that long.  At 16 rows, 16 requests of
// 100 to 16384 tokens, the first takes 24, 36 and 52 us (16 heads over 2 of 64, of 128, 32
// over 8 of 64), the second 46, 59 and 129: the limit is where the first kernel's fragments
// end (two groups of 8 rows), below where the two would cross.  float32 has its own pair of
// kernels on the CUDA cores, with the same limit: 85 us against 75 (16 over 2 of 64) and 594
// against 1002 (32 over 8 of 128).
#include "paged_fwd.cuh"

namespace relation {

size_t paged_fwd_workspace(const PagedProblem& pp, bool bf16, bool q8, int max_fresh, int num_sms) {
    if (!bf16) return paged_f32_workspace(pp, max_fresh, num_sms);
    const size_t few = paged_few_workspace(pp, q8, max_fresh, num_sms);  // the two passes overlap: a part each
    return (int64_t)max_fresh * pp.group <= kPagedFewRows ? few : few + paged_tc_workspace(pp, num_sms);
}

cudaError_t launch_paged_fwd(const PagedProblem& pp, bool bf16, const PagedFwdArgs& a, int* launches, cudaStream_t s) {
    if (!bf16) return launch_paged_f32(pp, a, a.workspace, launches, s);
    *launches = 2;
    if ((int64_t)a.max_fresh * pp.group <= kPagedFewRows) return launch_paged_few(pp, a, a.workspace, nullptr, s);
    paged::MergeSide few;  // both passes are merged in one launch
    const cudaError_t e = launch_paged_few(pp, a, a.workspace, &few, s);
    *launches = 3;
    if (e != cudaSuccess) return e;
    return launch_paged_tc(pp, a, static_cast<char*>(a.workspace) + paged_few_workspace(pp, a.scales != nullptr, a.max_fresh, a.num_sms), few,
                           s);
}

}  // namespace relation
