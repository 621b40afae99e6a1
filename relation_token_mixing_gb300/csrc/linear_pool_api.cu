// Host side of Linear Relation over a pool of states (include/relation.h):
// argument checks and dispatch.
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "api_internal.h"
#include "api_spans.h"
#include "linear_pool.h"

namespace relation {
namespace {

relation_status_t check_pool(const relation_linear_packed_t* p) {
    if (p == nullptr) return RELATION_ERR_INVALID_ARGUMENT;
    if (p->R < 1 || p->R > (1 << 20) || p->N < 0 || p->N > (int64_t)INT32_MAX || p->H < 1 || p->H > 1024 ||
        p->states < 1 || p->states > (int64_t)INT32_MAX)
        return RELATION_ERR_INVALID_ARGUMENT;
    if (p->dtype != RELATION_F32 && p->dtype != RELATION_BF16) return RELATION_ERR_INVALID_ARGUMENT;
    if (!(p->tau_S > 0.f) || !isfinite(p->tau_S) || p->d_h < 1) return RELATION_ERR_INVALID_ARGUMENT;
    if (p->dtype != RELATION_BF16 || (p->d_h != 48 && p->d_h != 60 && p->d_h != 64)) return RELATION_ERR_UNSUPPORTED;
    const double d = (double)p->d_h, H = (double)p->H;
    if ((double)p->N * H * d > 1e12 || (double)p->states * H * d * d > 1e12) return RELATION_ERR_INVALID_ARGUMENT;
    return RELATION_OK;
}

// The bound of a request's new tokens that the call works with.
int pool_bound(const relation_linear_packed_t* p, int max_fresh) {
    return max_fresh == 0 || (int64_t)max_fresh > p->N ? (int)p->N : max_fresh;
}

// starts == nullptr: one token a request.
relation_status_t run_pool(const relation_linear_packed_t* p, const void* P1, const void* P2, const void* I,
                           const float* G, const float* A_log, const float* dt_bias, const int32_t* starts,
                           bool packed, int max_fresh, float* states, const int32_t* slots_in, const int32_t* slots_out,
                           void* Y, void* workspace, size_t workspace_bytes, void* stream) {
    relation_status_t st = check_pool(p);
    if (st != RELATION_OK) return st;
    if (max_fresh < 0 || (!packed && p->N < p->R)) return RELATION_ERR_INVALID_ARGUMENT;
    if ((A_log == nullptr) != (dt_bias == nullptr)) return RELATION_ERR_INVALID_ARGUMENT;
    if (states == nullptr || slots_in == nullptr || slots_out == nullptr || (packed && starts == nullptr))
        return RELATION_ERR_INVALID_ARGUMENT;
    const void* rows[] = {P1, P2, I, G, Y};
    for (const void* x : rows)
        if (p->N > 0 && x == nullptr) return RELATION_ERR_INVALID_ARGUMENT;
    for (const void* x : rows)
        if (!aligned(x, 16)) return RELATION_ERR_MISALIGNED;
    if (!aligned(states, 16) || !aligned(workspace, 16)) return RELATION_ERR_MISALIGNED;
    for (const void* x : {(const void*)A_log, (const void*)dt_bias, (const void*)starts, (const void*)slots_in,
                          (const void*)slots_out})
        if (!aligned(x, 4)) return RELATION_ERR_MISALIGNED;
    unsigned int* status;
    int sms;
    if ((st = api_device(&status, &sms)) != RELATION_OK) return st;
    const int bound = packed ? pool_bound(p, max_fresh) : 1;
    const size_t need = packed ? linear_pool_workspace((int)p->R, (int)p->N, (int)p->H, bound, sms) : 0;
    if (need > 0 && workspace == nullptr) return RELATION_ERR_INVALID_ARGUMENT;
    if (workspace_bytes < need) return RELATION_ERR_WORKSPACE_TOO_SMALL;
    const size_t R = (size_t)p->R, n = (size_t)p->N * (size_t)p->H * (size_t)p->d_h,
                 per_head = A_log ? (size_t)p->H * (size_t)p->d_h * 4 : 0;
    const ByteSpan in[] = {{P1, n * 2}, {P2, n * 2}, {I, n * 2}, {G, n * 4}, {A_log, per_head}, {dt_bias, per_head},
                           {starts, starts ? (R + 1) * 4 : 0}, {slots_in, R * 4}, {slots_out, R * 4}};
    const ByteSpan out[] = {{Y, n * 2},
                            {states, (size_t)p->states * (size_t)p->H * (size_t)p->d_h * (size_t)p->d_h * 4},
                            {workspace, need}};
    if (!disjoint(in, 9, out, 3)) return RELATION_ERR_INVALID_ARGUMENT;
    LinearPool a{P1, P2, I, G, A_log, dt_bias, packed ? starts : nullptr, states, slots_in, slots_out, Y, status,
                 (int)p->R, (int)p->N, (int)p->H, (int)p->d_h, (int)p->states, bound,
                 (float)(1.0 / ((double)p->tau_S * sqrt((double)p->d_h)))};
    int launches = 0;
    const cudaError_t e = launch_linear_pool(a, workspace, sms, &launches, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return RELATION_ERR_CUDA;
    api_set_launches(launches);
    return RELATION_OK;
}

}  // namespace
}  // namespace relation

using namespace relation;

extern "C" {

relation_status_t relation_linear_step(const relation_linear_packed_t* p, const void* P1, const void* P2, const void* I,
                                       const float* G, const float* A_log, const float* dt_bias, float* states,
                                       const int32_t* slots_in, const int32_t* slots_out, void* Y, void* stream) {
    return run_pool(p, P1, P2, I, G, A_log, dt_bias, nullptr, false, 1, states, slots_in, slots_out, Y, nullptr, 0,
                    stream);
}

size_t relation_linear_packed_workspace_bytes(const relation_linear_packed_t* p, int max_fresh) {
    if (check_pool(p) != RELATION_OK || max_fresh < 0) return 0;
    unsigned int* status;
    int sms;
    if (api_device(&status, &sms) != RELATION_OK) return 0;
    return linear_pool_workspace((int)p->R, (int)p->N, (int)p->H, pool_bound(p, max_fresh), sms);
}

relation_status_t relation_linear_packed_fwd(const relation_linear_packed_t* p, const void* P1, const void* P2,
                                             const void* I, const float* G, const float* A_log, const float* dt_bias,
                                             const int32_t* starts, int max_fresh, float* states,
                                             const int32_t* slots_in, const int32_t* slots_out, void* Y,
                                             void* workspace, size_t workspace_bytes, void* stream) {
    return run_pool(p, P1, P2, I, G, A_log, dt_bias, starts, true, max_fresh, states, slots_in, slots_out, Y, workspace,
                    workspace_bytes, stream);
}

}  // extern "C"
