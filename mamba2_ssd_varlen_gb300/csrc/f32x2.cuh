// f32x2.cuh -- packed fp32 pairs (one 64-bit register pair): two fused multiply-adds
// an issue slot, at the rate of two single ones.  And the special-function unit's 2^x
// and 1/x, with what is built from them.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace ssd {

using f2 = uint64_t;

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
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
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
__device__ __forceinline__ f2 dup2(float v) { return pk(v, v); }

__device__ __forceinline__ float ex2f(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ f2 ex2_2(f2 x) {
    const float2 v = upk(x);
    return pk(ex2f(v.x), ex2f(v.y));
}
__device__ __forceinline__ float rcpf(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ f2 rcp_2(f2 x) {
    const float2 v = upk(x);
    return pk(rcpf(v.x), rcpf(v.y));
}

__device__ __forceinline__ float max_nan(float a, float b) {  // a NaN where one is
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLog2eLo = (float)(1.4426950408889634 - (double)kLog2e);
constexpr float kLn2 = 0.6931471805599453f;

// softplus(v) = max(v, 0) + log(1 + e), e = exp(-|v|) in (0, 1], to a few units in the last
// place for every v: log(1 + e) = 2 atanh(s) with s = e / (2 + e) <= 1/3, whose series in
// s^2 <= 1/9 is cut after s^12 / 13 (the rest is below 2e-8), and which keeps its relative
// accuracy for small e; exp(-|v|) = 2^x (1 + r ln 2) with r what x = fl(-|v| log2 e) lost.
__device__ __forceinline__ f2 softplus2(f2 v) {
    const float2 w = upk(v);
    const f2 t = pk(max_nan(-fabsf(w.x), -200.f), max_nan(-fabsf(w.y), -200.f));  // e is 0 there
    const f2 x = mul2(t, dup2(kLog2e));
    f2 r = fma2(t, dup2(kLog2e), mul2(x, dup2(-1.f)));
    r = fma2(t, dup2(kLog2eLo), r);
    f2 e = ex2_2(x);
    e = fma2(e, mul2(r, dup2(kLn2)), e);
    const f2 s = mul2(e, rcp_2(add2(e, dup2(2.f))));
    const f2 q = mul2(s, s);
    f2 p = fma2(q, dup2(1.f / 13.f), dup2(1.f / 11.f));
    p = fma2(p, q, dup2(1.f / 9.f));
    p = fma2(p, q, dup2(1.f / 7.f));
    p = fma2(p, q, dup2(1.f / 5.f));
    p = fma2(p, q, dup2(1.f / 3.f));
    const f2 s2 = add2(s, s);
    p = fma2(mul2(p, q), s2, s2);
    return add2(pk(fmaxf(w.x, 0.f), fmaxf(w.y, 0.f)), p);
}

// silu(z) = z / (1 + exp(-z)).
__device__ __forceinline__ f2 silu2(f2 z) {
    return mul2(z, rcp_2(add2(ex2_2(mul2(z, dup2(-kLog2e))), dup2(1.f))));
}

}  // namespace ssd
