// packed.cuh -- hardware exponential and reciprocal, and the packed FP32 instructions of sm_100a.
#pragma once

#include <stdint.h>

namespace kron {

__device__ __forceinline__ float ex2(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float rcp(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// Two fp32 values in one 64-bit register pair, for the packed FP32 instructions: one issue slot
// for two additions, multiplications or multiply-adds, each rounded as the scalar one.
typedef uint64_t f2;
__device__ __forceinline__ f2 pack2(float lo, float hi) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(f2 v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f2 ex2_2(f2 v) {
    float lo, hi;
    unpack2(v, lo, hi);
    return pack2(ex2(lo), ex2(hi));
}
__device__ __forceinline__ f2 rcp_2(f2 v) {
    float lo, hi;
    unpack2(v, lo, hi);
    return pack2(rcp(lo), rcp(hi));
}
__device__ __forceinline__ f2 dup2(float v) { return pack2(v, v); }

}  // namespace kron
