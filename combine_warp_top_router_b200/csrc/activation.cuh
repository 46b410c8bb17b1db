// activation.cuh -- the experts' activation (internal).
#pragma once

#include "common.cuh"

namespace md {

// 1 / (1 + exp(-g)).  exp(-g) = 2^t with t = -g log2(e); t's rounding error, which
// would be |g| 2^-24 of the result, is put back to first order, so the result is good
// to a few float32 ulps for |g| < 44 and to 2^-17 of itself below -44 (where the
// exponential overflows, it is 0).  11 instructions; with expf and a division the
// kernels that call it were bound by issuing them.
__device__ __forceinline__ float sigmoid(float g)
{
    constexpr float kLog2e = 1.44269504f, kLn2 = 0.693147181f;
    const float t = -g * kLog2e;
    const float lost = fabsf(t) < 64.0f ? fmaf(-g, kLog2e, -t) * kLn2 : 0.0f;
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
    e = lost == 0.0f ? e : fmaf(e, lost, e);  // not where e may be infinite
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return r;
}

}  // namespace md
