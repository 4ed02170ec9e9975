// gated_math.cuh -- the activations of a gated feed-forward block, in FP32.
//
// Both are g times a logistic function: SiLU g / (1 + e^-g), and the tanh form of
// GELU, g (1 + tanh z) / 2 = g / (1 + e^-2z) with z = sqrt(2/pi) (g + 0.044715 g^3).
// e^x is ex2.approx of t, x log2 e rounded, times 1 + (x - t ln 2): what the rounding left
// of x, up to 2^-24 |x|, goes in to first order, and 2^-22 is left beside the
// approximation's 2^-22; the reciprocal is off by 2^-23, and below -87.3 the function is 0.
// The products take no longer than they spread (with expf 1-2 %).  The gradient, whose
// results are BF16 or codes (2^-8 or 2^-4 of themselves), leaves the first order out and
// is off by 2^-24 |x| more (with expf 226 -> 255 us).
#pragma once
#include <cstdint>

#include "tmem_util.cuh"

namespace mxg {

constexpr int kActSilu = 0, kActGeluTanh = 1;  // mxgemm_act_t
constexpr float kGeluTwo = 1.59576912160573071176f, kGeluCube = 0.044715f;  // 2 sqrt(2 / pi)

// 1 / (1 + e^-x)
__device__ __forceinline__ float logistic(float x) {
  const float y = fminf(fmaxf(-x, -88.f), 88.f), t = y * 1.44269504088896340736f;
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
  e = fmaf(e, fmaf(t, -0.69314718055994530942f, y), e);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return r;
}
// What multiplies g in the activation.
__device__ __forceinline__ float act_weight(float g, int act) {
  return logistic(act == kActSilu ? g : kGeluTwo * g * fmaf(kGeluCube * g, g, 1.f));
}
__device__ __forceinline__ float gated(float g, float u, int act) { return g * act_weight(g, act) * u; }

// dgate, dup and the hidden value of two values' dH, in paired FP32 operations.
struct GatedGrad2 {
  float2 dg, du, h;
};
__device__ __forceinline__ float2 logistic2(float2 e2) {  // 1 / (1 + 2^e2)
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e2.x));
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e2.y));
  e2 = add2(e2, make_float2(1.f, 1.f));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(e2.x));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(e2.y));
  return e2;
}
template <int ACT>
__device__ __forceinline__ GatedGrad2 gated_grad(float2 g, float2 u, float2 dh) {
  auto both = [](float x) { return make_float2(x, x); };
  constexpr float kLog2 = 1.44269504088896340736f;
  float2 p, w;  // the logistic function's value, and the activation's derivative
  if constexpr (ACT == kActSilu) {
    p = logistic2(mul2(g, both(-kLog2)));
    const float2 a = mul2(g, p);
    w = fma2(a, fma2(p, both(-1.f), both(1.f)), p);
  } else {
    const float2 gg = mul2(g, g);
    p = logistic2(mul2(mul2(g, both(-kLog2 * kGeluTwo)), fma2(gg, both(kGeluCube), both(1.f))));
    // (past |g| = 100 a (1 - p) is 0, which is not to meet an infinite slope)
    const float2 slope = fma2(make_float2(fminf(gg.x, 1e4f), fminf(gg.y, 1e4f)), both(3.f * kGeluCube * kGeluTwo), both(kGeluTwo));
    w = fma2(mul2(mul2(g, p), fma2(p, both(-1.f), both(1.f))), slope, p);
  }
  const float2 a = mul2(g, p);
  return GatedGrad2{mul2(mul2(dh, u), w), mul2(dh, a), mul2(a, u)};
}

}  // namespace mxg
