// act_pairs.cuh - the activations and their derivatives on pairs of values, to about 1e-6 of the value: for results
// that keep more than the bf16 epilogues' hardware tanh (error 2^-11 of 1) carries - codes, whose rounding it would
// move one time in a hundred, fp32 sums of gradients, and the small values on GeLU's negative side. FAST (bf16
// inputs): the hardware's exponential and reciprocal, two operations of the special-function unit a value; else
// the accurate forms.
#pragma once

#include "gn_common.cuh"

namespace gn {

__device__ __forceinline__ float ex2_ftz(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_ftz(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.4426950408889634f;

// sigmoid(2 u) of the tanh-GeLU's argument: (1 + tanh u) / 2 = 1 / (1 + exp(-2 u))
__device__ __forceinline__ float2 gelu_u2(float2 z, float2 z2) {  // -2 u log2(e)
  return mul2(z, fma2(z2, dup2(-2.0f * kLog2e * kGeluK * kGeluC), dup2(-2.0f * kLog2e * kGeluK)));
}

template <int EPI, bool FAST>
__device__ __forceinline__ float2 act_pair(float2 z) {
  if constexpr (!FAST || EPI == EPI_NONE) {
    return make_float2(epi_fwd<EPI, false>(z.x), epi_fwd<EPI, false>(z.y));
  } else {
    const float2 t = EPI == EPI_SILU ? mul2(z, dup2(-kLog2e)) : gelu_u2(z, mul2(z, z));
    const float2 d = add2(make_float2(ex2_ftz(t.x), ex2_ftz(t.y)), dup2(1.0f));
    return mul2(z, make_float2(rcp_ftz(d.x), rcp_ftz(d.y)));
  }
}
template <int EPI, bool FAST>
__device__ __forceinline__ float2 act_grad_pair(float2 z) {
  if constexpr (!FAST || EPI == EPI_NONE) {
    return make_float2(epi_grad<EPI, false>(z.x), epi_grad<EPI, false>(z.y));
  } else if constexpr (EPI == EPI_SILU) {  // s (1 + z (1 - s))
    const float2 t = mul2(z, dup2(-kLog2e));
    const float2 d = add2(make_float2(ex2_ftz(t.x), ex2_ftz(t.y)), dup2(1.0f));
    const float2 s = make_float2(rcp_ftz(d.x), rcp_ftz(d.y));
    return mul2(s, fma2(z, fma2(s, dup2(-1.0f), dup2(1.0f)), dup2(1.0f)));
  } else {  // p = sigmoid(2 u): p (1 + z (1 - p) (2 u)'); 1 - p = a / (1 + a) without cancellation, a = exp(-|2 u|)
    const float2 z2 = mul2(z, z), t = gelu_u2(z, z2);
    const float2 a = make_float2(ex2_ftz(-fabsf(t.x)), ex2_ftz(-fabsf(t.y)));
    const float2 d = add2(a, dup2(1.0f));
    const float2 r = make_float2(rcp_ftz(d.x), rcp_ftz(d.y)), ra = mul2(r, a);
    const float2 p = make_float2(t.x <= 0.0f ? r.x : ra.x, t.y <= 0.0f ? r.y : ra.y);
    const float2 n = make_float2(t.x <= 0.0f ? ra.x : r.x, t.y <= 0.0f ? ra.y : r.y);
    return mul2(p, fma2(mul2(z, n), fma2(z2, dup2(6.0f * kGeluK * kGeluC), dup2(2.0f * kGeluK)), dup2(1.0f)));
  }
}

}  // namespace gn
