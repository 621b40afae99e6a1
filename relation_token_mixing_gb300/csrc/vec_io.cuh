// Loads and stores of VC consecutive elements as fp32: 16-, 8- or 4-byte accesses
// for bf16 VC = 8, 4, 2; 16- and 8-byte ones for fp32.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace relation {

template <int BYTES>
struct VecWords;
template <>
struct VecWords<16> { using type = uint4; };
template <>
struct VecWords<8> { using type = uint2; };
template <>
struct VecWords<4> { using type = uint32_t; };

template <typename T, int VC>
struct Vec {
    using Words = typename VecWords<VC * sizeof(T)>::type;
    Words w;
    __device__ __forceinline__ void load(const T* p) { w = __ldg(reinterpret_cast<const Words*>(p)); }
    __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<Words*>(p) = w; }
    __device__ __forceinline__ void unpack(float (&v)[VC]) const {
        if constexpr (sizeof(T) == 4) {
            const float* f = reinterpret_cast<const float*>(&w);
#pragma unroll
            for (int k = 0; k < VC; ++k) v[k] = f[k];
        } else {
            const __nv_bfloat162* b = reinterpret_cast<const __nv_bfloat162*>(&w);
#pragma unroll
            for (int k = 0; k < VC / 2; ++k) {
                const float2 f = __bfloat1622float2(b[k]);
                v[2 * k] = f.x, v[2 * k + 1] = f.y;
            }
        }
    }
    __device__ __forceinline__ void pack(const float (&v)[VC]) {
        if constexpr (sizeof(T) == 4) {
            float* f = reinterpret_cast<float*>(&w);
#pragma unroll
            for (int k = 0; k < VC; ++k) f[k] = v[k];
        } else {
            __nv_bfloat162* b = reinterpret_cast<__nv_bfloat162*>(&w);
#pragma unroll
            for (int k = 0; k < VC / 2; ++k) b[k] = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
        }
    }
};

}  // namespace relation
