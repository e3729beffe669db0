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
// same reason.  The exponential and the quotient are the fast ones (__expf, __fdividef): off by
// a few units of 2^-24 relative, plus |u| of them for the exponential's argument, where
// the store rounds to 2^-11 or 2^-8.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace vq {

// v * sigmoid(u): e^-u = inf gives 0, and no more than one operation each of ex2 and rcp.
__device__ __forceinline__ float times_sigmoid(float v, float u) { return __fdividef(v, 1.f + __expf(-u)); }

template <int kAct>
__device__ __forceinline__ float act_of(float v) {
  if (kAct == VQ_ACT_RELU) return v < 0.f ? 0.f : v;  // NaN stays NaN
  if (kAct == VQ_ACT_SILU) return times_sigmoid(v, v);
  if (kAct == VQ_ACT_GELU_TANH) return times_sigmoid(v, v * fmaf(0.07135481627613502f, v * v, 1.5957691216057308f));
  if (kAct == VQ_ACT_GELU) return 0.5f * v * erfcf(v * -0.70710678118654752f);
  return v;
}

__device__ __forceinline__ float apply_act(int act, float v) {
  switch (act) {
    case VQ_ACT_RELU: return act_of<VQ_ACT_RELU>(v);
    case VQ_ACT_SILU: return act_of<VQ_ACT_SILU>(v);
    case VQ_ACT_GELU_TANH: return act_of<VQ_ACT_GELU_TANH>(v);
    case VQ_ACT_GELU: return act_of<VQ_ACT_GELU>(v);
    default: return v;
  }
}

// The same for an array: one choice for all of it.
template <int kAct, int kN>
__device__ __forceinline__ void act_all(float (&f)[kN]) {
#pragma unroll
  for (int i = 0; i < kN; ++i) f[i] = act_of<kAct>(f[i]);
}
template <int kN>
__device__ __forceinline__ void apply_act_all(int act, float (&f)[kN]) {
  switch (act) {
    case VQ_ACT_RELU: act_all<VQ_ACT_RELU>(f); break;
    case VQ_ACT_SILU: act_all<VQ_ACT_SILU>(f); break;
    case VQ_ACT_GELU_TANH: act_all<VQ_ACT_GELU_TANH>(f); break;
    case VQ_ACT_GELU: act_all<VQ_ACT_GELU>(f); break;
    default: break;
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
    if (a.bias) {
      const float b = Elt<T>::to_f32(a.bias[n]);
#pragma unroll
      for (int i = 0; i < 16; ++i) f[i] += b;
    }
    apply_act_all(a.act_fn, f);
    if (a.mul) {
#pragma unroll
      for (int i = 0; i < 16; ++i) f[i] *= Elt<T>::to_f32(u[i]);
    }
    if (a.res) {
#pragma unroll
      for (int i = 0; i < 16; ++i) f[i] += Elt<T>::to_f32(r[i]);
    }
  }
}

}  // namespace vq
