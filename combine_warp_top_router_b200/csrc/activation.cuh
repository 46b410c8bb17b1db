// activation.cuh -- the experts' activation (internal).
#pragma once

#include "common.cuh"

namespace md {

// 1 / (1 + exp(-g)), relative error below 10 * 2^-24 for every g (to float32's last step
// where it is subnormal).  exp(-g) = 2^t exp(-g - t ln 2) with t = -g log2(e) rounded; the
// second factor, which holds t's rounding and that of log2(e), is taken to first
// order, and the float32 ln 2 in it is off by 1.9e-9 |t|, 4 * 2^-24 at g = -87.  The rest: ex2
// (2^-22), the factor's rounding and, above g = -44, 1 + 2^t and its reciprocal.
// Below, the result is exp(g) itself, to float32's precision, taken as
// 2^(64 - t) 2^-64 so that nothing overflows on the way.  About 14 instructions; with
// expf and a division the kernels that call it were bound by issuing them.
__device__ __forceinline__ float sigmoid(float g)
{
    constexpr float kLog2e = 1.44269504f, kLn2 = 0.693147181f;
    const float t = -g * kLog2e;
    const bool low = t > 64.0f;
    float lost = fabsf(t) < 256.0f ? fmaf(-t, kLn2, -g) : 0.0f;  // beyond, the power is 0
    lost = low ? -lost : lost;
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(low ? 64.0f - t : t));
    e = fmaf(e, lost, e);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return low ? e * 5.42101086e-20f : r;  // 2^-64
}

}  // namespace md
