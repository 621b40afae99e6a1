// Linear Relation over a pool of states: kernel-side arguments and launches.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace relation {

// Kernel-side view of one relation_linear_packed_t with its tensors.
struct LinearPool {
    const void *P1, *P2, *I;  // [N, H, d] bf16
    const float *G, *A_log, *dt_bias;
    const int* starts;  // [R + 1], or nullptr: request r is token r
    float* states;      // [slots, H, d, d]
    const int *slots_in, *slots_out;
    void* Y;
    unsigned int* status;
    int R, N, H, d, slots;
    int max_fresh;
    float zscale;  // 1 / (tau_S sqrt d)
};

// Workspace bytes and launches of a packed call (max_fresh: of the pool's arguments).
size_t linear_pool_workspace(int R, int N, int H, int max_fresh, int num_sms);
cudaError_t launch_linear_pool(const LinearPool& p, void* workspace, int num_sms, int* launches, cudaStream_t s);

}  // namespace relation
