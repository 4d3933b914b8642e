// special.cuh -- the special-function unit's 2^x and 1/x, and the softplus and SiLU
// that are built from them.
#pragma once

#include <cuda_runtime.h>

namespace ssd {

__device__ __forceinline__ float ex2f(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcpf(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {  // a NaN where one is
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// softplus(v) = max(v, 0) + log(1 + e), e = exp(-|v|) in (0, 1], to a few units in the last
// place for every v: log(1 + e) = 2 atanh(s) with s = e / (2 + e) <= 1/3, whose series in
// s^2 <= 1/9 is cut after s^12 / 13 (the rest is below 2e-8), and which keeps its relative
// accuracy for small e; exp(t) = 2^x (1 + t - x ln 2) with x = fl(t log2 e), so that the
// rounding of x does not count.
// In two halves, so that a caller can put other work behind 1 / (2 + e): e, then the rest from v, e and r = 1 / (2 + e).
__device__ __forceinline__ float softplus_exp(float v) {
    const float t = max_nan(-fabsf(v), -200.f);  // e is 0 there
    const float x = t * kLog2e;
    const float e = ex2f(x);
    return fmaf(e, fmaf(x, -kLn2, t), e);
}
__device__ __forceinline__ float softplus_end(float v, float e, float r) {
    const float s = e * r, q = s * s;
    float p = fmaf(q, 2.f / 13.f, 2.f / 11.f);
    p = fmaf(p, q, 2.f / 9.f);
    p = fmaf(p, q, 2.f / 7.f);
    p = fmaf(p, q, 2.f / 5.f);
    p = fmaf(p, q, 2.f / 3.f);
    p = fmaf(p * q, s, s + s);
    return fmaxf(v, 0.f) + p;
}

// silu(z) = z / (1 + exp(-z)).
__device__ __forceinline__ float silu_sfu(float z) { return z * rcpf(1.f + ex2f(-kLog2e * z)); }

}  // namespace ssd
