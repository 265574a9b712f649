#pragma once
// Two fp32 values in one 64-bit register pair, for the f32x2 instructions.  Where a value takes part
// in several operations, keeping the pair itself (not its two halves) spares the copies that put the
// halves side by side for each operation.
#include <cuda_runtime.h>

#include "scan_kernel.cuh"   // ex2_approx, rcp_approx, kLog2e

namespace ssm {

using pair_t = unsigned long long;

__device__ __forceinline__ pair_t pk(float lo, float hi) {
    pair_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ pair_t pk(float v) { return pk(v, v); }
__device__ __forceinline__ float2 halves(pair_t a) {
    float2 d;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(a));
    return d;
}
__device__ __forceinline__ pair_t pfma(pair_t a, pair_t b, pair_t c) {
    pair_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ pair_t pmul(pair_t a, pair_t b) {
    pair_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ pair_t padd(pair_t a, pair_t b) {
    pair_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ pair_t pex2(pair_t a) {
    const float2 v = halves(a);
    return pk(ex2_approx(v.x), ex2_approx(v.y));
}
__device__ __forceinline__ pair_t prcp(pair_t a) {
    const float2 v = halves(a);
    return pk(rcp_approx(v.x), rcp_approx(v.y));
}
// z / (1 + e^-z)
__device__ __forceinline__ pair_t psilu(pair_t z) {
    return pmul(z, prcp(padd(pex2(pmul(z, pk(-kLog2e))), pk(1.f))));
}

}  // namespace ssm
