// Warp-level tensor-core fragments, swizzled 64-column tiles and the retention
// gate, shared by the Linear Relation kernels.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "ptx_sm100.cuh"

namespace relation {
namespace lin {

constexpr int kDp = 64;         // head width the kernels work in (narrower heads are zero-padded)

// ---------------------------------------------------------------- PTX helpers
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
// (lo, hi) -> packed bf16 pair, lo in the low half.
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Packed fp32 pairs.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    unsigned long long d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(d)
        : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)),
          "l"(*reinterpret_cast<unsigned long long*>(&c)));
    return *reinterpret_cast<float2*>(&d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    unsigned long long d;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(d)
        : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)));
    return *reinterpret_cast<float2*>(&d);
}

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void st_zero16(uint32_t dst) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(dst), "r"(0u) : "memory");
}

// Byte offset of (row r, column c) in a 16 x 64 bf16 tile: 128-byte rows whose
// 16-byte chunks are permuted by the row (conflict-free ldmatrix).
__device__ __forceinline__ uint32_t swz(int r, int c) {
    return (uint32_t)(r * 128 + ((((c >> 3) ^ r) & 7) << 4) + ((c & 7) << 1));
}

// ldmatrix lane addresses (PTX fragment layouts of m16n8k16).
// A operand 16 x 16 from a row-major [m][k] swizzled tile at column k0.
__device__ __forceinline__ uint32_t addr_a(const uint8_t* tile, int k0, int lane) {
    const int m = lane >> 3, r = (lane & 7) + 8 * (m & 1), c = k0 + 8 * (m >> 1);
    return ptx::smem_u32(tile) + swz(r, c);
}
// B fragments of two 8-wide column blocks n0, n0+8 from a [k][n] tile (.trans).
__device__ __forceinline__ uint32_t addr_bt(const uint8_t* tile, int n0, int lane) {
    const int m = lane >> 3, r = (lane & 7) + 8 * (m & 1), c = n0 + 8 * (m >> 1);
    return ptx::smem_u32(tile) + swz(r, c);
}
// A operand from a [k][m] tile (.trans): a0..a3 = (m0-7,k0-7), (m8-15,k0-7),
// (m0-7,k8-15), (m8-15,k8-15).
__device__ __forceinline__ uint32_t addr_at(const uint8_t* tile, int m0, int lane) {
    const int m = lane >> 3, r = (lane & 7) + 8 * (m >> 1), c = m0 + 8 * (m & 1);
    return ptx::smem_u32(tile) + swz(r, c);
}

// softplus(x) = max(x, 0) + log(1 + e^-|x|), which overflows for no x; the
// logarithm's argument is rounded to fp32, an absolute error below 1e-7 in g,
// i.e. in the retention alpha = exp(g) a relative error below 1e-7 x alpha.
__device__ __forceinline__ float softplus_f(float x) { return fmaxf(x, 0.f) + __logf(1.f + __expf(-fabsf(x))); }

}  // namespace lin
}  // namespace relation
