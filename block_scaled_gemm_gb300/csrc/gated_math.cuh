// gated_math.cuh -- the activations of a gated feed-forward block, in FP32.
//
// Both are g times a logistic function: SiLU g / (1 + e^-g), and the tanh form of
// GELU, g (1 + tanh z) / 2 = g / (1 + e^-2z) with z = sqrt(2/pi) (g + 0.044715 g^3).
// e^x is ex2.approx of x log2 e, whose argument's rounding makes it off by 2^-24 |x|
// of itself beside the approximation's 2^-22; the reciprocal is off by 2^-23.
#pragma once
#include <cstdint>

namespace mxg {

constexpr int kActSilu = 0, kActGeluTanh = 1;  // mxgemm_act_t
constexpr float kGeluTwo = 1.59576912160573071176f, kGeluCube = 0.044715f;  // 2 sqrt(2 / pi)

// 1 / (1 + e^-x)
__device__ __forceinline__ float logistic(float x) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.44269504088896340736f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return r;
}
// What multiplies g in the activation.
__device__ __forceinline__ float act_weight(float g, int act) {
  return logistic(act == kActSilu ? g : kGeluTwo * g * fmaf(kGeluCube * g, g, 1.f));
}
__device__ __forceinline__ float gated(float g, float u, int act) { return g * act_weight(g, act) * u; }

// dgate, dup and the hidden value of one value's dH.
struct GatedGrad {
  float dg, du, h;
};
__device__ __forceinline__ GatedGrad gated_grad(float g, float u, float dh, int act) {
  const float p = act_weight(g, act), a = g * p;
  // (past |g| = 100 a (1 - p) is 0, which is not to meet an infinite slope)
  const float slope = act == kActSilu ? 1.f : kGeluTwo * fmaf(3.f * kGeluCube, fminf(g * g, 1e4f), 1.f);
  return GatedGrad{dh * u * fmaf(a * (1.f - p), slope, p), dh * a, a * u};
}

}  // namespace mxg
