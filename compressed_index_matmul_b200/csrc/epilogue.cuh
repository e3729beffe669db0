// The fused epilogue of a forward (vq_linear_forward_epilogue, vq_experts_forward):
//   y = RN(act(f + bias) * mul + residual),
// f the fp32 product (with the sparse correction's term), every step in fp32 and one
// rounding, at the store.  It runs where the forward kernels round into y, so a fused
// call reads bias, mul and residual once and neither writes nor re-reads the product.
//
// SiLU and the tanh form of GELU are one formula, v * sigmoid(v (c0 + c1 v^2)):
// 1 + tanh(u) = 2 sigmoid(2u), so GELU's tanh form has c0 = 2 sqrt(2/pi), c1 =
// 0.044715 c0, and SiLU c0 = 1, c1 = 0.  This keeps its relative accuracy for
// negative v, where 1 + tanh(u) cancels.  The erf form is v/2 * erfc(-v / sqrt 2) for the
// same reason.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace vq {

__device__ __forceinline__ float apply_act(int act, float v) {
  switch (act) {
    case VQ_ACT_RELU: return v < 0.f ? 0.f : v;  // NaN stays NaN
    case VQ_ACT_SILU:
    case VQ_ACT_GELU_TANH: {
      // (no v * v for SiLU: 0 * inf would make large v a NaN)
      const float u = act == VQ_ACT_SILU ? v : v * fmaf(0.07135481627613502f, v * v, 1.5957691216057308f);
      return v * __fdividef(1.f, 1.f + expf(-u));  // e^-u = inf: the quotient is 0
    }
    case VQ_ACT_GELU: return 0.5f * v * erfcf(v * -0.70710678118654752f);
    default: return v;
  }
}

// Output (m, n) with at = m N + n: the sparse correction's term, then the epilogue.
// mul and residual are read with plain loads: either may be y itself (each element is
// read and then written by one thread).
template <typename T>
__device__ __forceinline__ float finish(const LayerArgs& a, int64_t at, int n, float f) {
  if (a.addend) f += a.addend[at];  // the sparse correction's x . C^T term
  if (a.epi) {
    const float u = a.mul ? Elt<T>::to_f32(a.mul[at]) : 1.f;
    const float r = a.res ? Elt<T>::to_f32(a.res[at]) : 0.f;
    if (a.bias) f += Elt<T>::to_f32(a.bias[n]);
    f = apply_act(a.act_fn, f);
    if (a.mul) f *= u;
    if (a.res) f += r;
  }
  return f;
}

// The same for 16 consecutive tokens tok .. tok + 15 (those below M) of output n: all
// loads are issued before the first use.
template <typename T>
__device__ __forceinline__ void finish16(const LayerArgs& a, int tok, int n, float (&f)[16]) {
  if (a.addend) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (tok + i < a.M) f[i] += a.addend[(int64_t)(tok + i) * a.N + n];
  }
  if (a.epi) {
    uint16_t u[16], r[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int64_t at = (int64_t)(tok + i) * a.N + n;
      const bool in = tok + i < a.M;
      u[i] = (a.mul && in) ? a.mul[at] : (uint16_t)0;
      r[i] = (a.res && in) ? a.res[at] : (uint16_t)0;
    }
    const float b = a.bias ? Elt<T>::to_f32(a.bias[n]) : 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (a.bias) f[i] += b;
      f[i] = apply_act(a.act_fn, f[i]);
      if (a.mul) f[i] *= Elt<T>::to_f32(u[i]);
      if (a.res) f[i] += Elt<T>::to_f32(r[i]);
    }
  }
}

}  // namespace vq
