// activation.cuh -- the experts' activation (internal).
#pragma once

#include "common.cuh"

namespace md {

// 1 / (1 + exp(-g)), good to a few float32 ulps for every g (to float32's last
// step where it is subnormal).  exp(-g) = 2^t with t = -g log2(e); t's rounding error, which
// would be |g| 2^-24 of the result, is put back to first order.  Below g = -44 the
// result is exp(g) itself, to float32's precision, taken as 2^(64 - t) 2^-64 so that
// nothing overflows on the way.  About 15 instructions; with expf and a division
// the kernels that call it were bound by issuing them.
__device__ __forceinline__ float sigmoid(float g)
{
    constexpr float kLog2e = 1.44269504f, kLn2 = 0.693147181f;
    const float t = -g * kLog2e;
    const bool low = t > 64.0f;
    float lost = fabsf(t) < 256.0f ? fmaf(-g, kLog2e, -t) * kLn2 : 0.0f;  // beyond, the power is 0
    lost = low ? -lost : lost;
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(low ? 64.0f - t : t));
    e = fmaf(e, lost, e);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return low ? e * 5.42101086e-20f : r;  // 2^-64
}

}  // namespace md
