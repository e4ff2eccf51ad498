// quotient.hpp -- x / d for many x and one d, as the division gives it, at a third of its
// instructions.
#pragma once

#include <hip/hip_runtime.h>

namespace mpdt {

// Divisors that quotient() takes: nothing that matters leaves the range of FP32 on the way.
__device__ __forceinline__ bool divides(float d) { return d >= 0x1p-60f && d <= 0x1p60f; }

// x / d rounded to nearest, from the reciprocal r = 1 / d (itself correctly rounded).  x * r
// may be off by two units in the last place; one step with the product's error leaves it
// within one, and from there another step rounds correctly (Markstein's theorem: P.
// Markstein, "Computation of elementary functions on the IBM RISC System/6000 processor",
// 1990).  Holds for finite quotients; those below 2^-66 may come out with fewer bits.  The
// remainder is taken as p * d - x and its part subtracted: for x = -0 that leaves p at -0
// (-0 * d + 0 = +0, -0 - 0 * r = -0), where x - p * d added would make it +0.
__device__ __forceinline__ float quotient(float x, float d, float r) {
    float p = x * r;
    p = __builtin_fmaf(-__builtin_fmaf(p, d, -x), r, p);
    return __builtin_fmaf(-__builtin_fmaf(p, d, -x), r, p);
}

}  // namespace mpdt
