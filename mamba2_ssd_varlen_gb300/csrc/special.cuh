// special.cuh -- the special-function unit's 2^x and 1/x, and the softplus and SiLU
// that are built from them.
#pragma once

#include <cuda_runtime.h>

namespace ssd {

// Packed fp32 pairs (one 64-bit register pair): two products or sums an issue slot.
using f2 = unsigned long long;
__device__ __forceinline__ f2 pk(float lo, float hi) {
    f2 d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ float2 upk(f2 d) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(d));
    return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

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

// Added to the argument of a decay's 2^x.  The unit's 2^x is low on average: by 5e-9 relative for x in (-2e-3, 0), by
// 1e-8 to 3e-8 down to -0.2 (measured, 2^18 arguments a bin; its documented bound is 2^-22), and a state is a product of as
// many decays as it remembers tokens, so a slow state would end up low by that many times as much.  1.4e-8 raises 2^x by
// 9.7e-9, a quarter of a unit in the last place of a decay near 1: between the two, so that neither the slowest states
// (mostly the initial one) nor the ordinary ones gather much.  Relative error of the final states against 64 bits over
// fixed and drawn prompts: 2e-7 to 1.4e-6 (13 ragged fp32 prompts: 1.2e-6 without it, 7e-7 with it), where exponentials
// rounded correctly give 1e-7 to 2e-7; it costs no time, while a polynomial in place of the unit would cost the fp32 pipe
// ten operations a state and token, more than twice what the recurrence itself takes there.
constexpr float kDecayShift = 1.4e-8f;

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

// The same for a packed pair.
__device__ __forceinline__ f2 softplus_exp(f2 v) {
    const float2 w = upk(v);
    const f2 t = pk(max_nan(-fabsf(w.x), -200.f), max_nan(-fabsf(w.y), -200.f));
    const f2 x = mul2(t, pk(kLog2e, kLog2e));
    const float2 y = upk(x);
    const f2 e = pk(ex2f(y.x), ex2f(y.y));
    return fma2(e, fma2(x, pk(-kLn2, -kLn2), t), e);
}
__device__ __forceinline__ f2 softplus_end(f2 v, f2 e, f2 r) {
    const f2 s = mul2(e, r), q = mul2(s, s);
    f2 p = fma2(q, pk(2.f / 13.f, 2.f / 13.f), pk(2.f / 11.f, 2.f / 11.f));
    p = fma2(p, q, pk(2.f / 9.f, 2.f / 9.f));
    p = fma2(p, q, pk(2.f / 7.f, 2.f / 7.f));
    p = fma2(p, q, pk(2.f / 5.f, 2.f / 5.f));
    p = fma2(p, q, pk(2.f / 3.f, 2.f / 3.f));
    p = fma2(mul2(p, q), s, add2(s, s));
    const float2 w = upk(v);
    return add2(pk(fmaxf(w.x, 0.f), fmaxf(w.y, 0.f)), p);
}

// silu(z) = z / (1 + exp(-z)).
__device__ __forceinline__ float silu_sfu(float z) { return z * rcpf(1.f + ex2f(-kLog2e * z)); }

}  // namespace ssd
