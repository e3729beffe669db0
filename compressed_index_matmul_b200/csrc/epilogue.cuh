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
// the store rounds to 2^-11 or 2^-8; a quotient by more than 2^126 is 0, so an activation below
// |v| 2^-126 is.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace vq {

// The code is kept small, and what a call has no tensor for is jumped over: every forward kernel
// holds it at each of its stores, unrolled over the values of a thread, and a short forward
// waits for instructions that the SM has not run yet (1003 x 960 at M = 77 in 8 splits of K with bias
// and GELU: 24.4 us with every activation and load unrolled and predicated, 22.2 so, 18.0 without an
// epilogue; in the one split now taken 14.2 and 9.5;
// 8192 x 8192 at M = 1024 with bias, GELU and residual: 151 against 134 us, 120 without).  Hence one
// formula for two activations, and a call for the erf form.
struct ActParams {
  float c0, c1;  // the exponent is v (c0 + c1 v^2)
};
__device__ __forceinline__ ActParams act_params(int act) {
  return act == VQ_ACT_GELU_TANH ? ActParams{1.5957691216057308f, 0.07135481627613502f} : ActParams{1.f, 0.f};
}
// v * sigmoid(v (c0 + c1 v^2)); e^-u = inf gives 0.  The square is kept finite: 0 * inf would make a
// large v a NaN under SiLU.
__device__ __forceinline__ float act_sigmoid(const ActParams& p, float v) {
  const float u = v * fmaf(p.c1, fminf(v * v, 1e30f), p.c0);
  return __fdividef(v, 1.f + __expf(-u));
}
static __device__ __noinline__ float act_gelu(float v) { return 0.5f * v * erfcf(v * -0.70710678118654752f); }

// An array of values: one choice for all of it.
template <int kN>
__device__ __forceinline__ void apply_act_all(int act, float (&f)[kN]) {
  if (act == VQ_ACT_NONE) return;
  if (act == VQ_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < kN; ++i) f[i] = act_gelu(f[i]);
  } else if (act == VQ_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < kN; ++i) f[i] = f[i] < 0.f ? 0.f : f[i];  // NaN stays NaN
  } else {
    const ActParams p = act_params(act);
#pragma unroll
    for (int i = 0; i < kN; ++i) f[i] = act_sigmoid(p, f[i]);
  }
}

__device__ __forceinline__ float apply_act(int act, float v) {
  float f[1] = {v};
  apply_act_all(act, f);
  return f[0];
}

// Output (m, n) with at = m N + n: the sparse correction's term, then (kFused) the epilogue.
// mul and residual are read with plain loads: either may be y itself (each element is
// read and then written by one thread).  The small kernels are compiled with and without it too:
// jumped over in one instantiation it cost a short plain forward up to 0.6 us (6640 x 192 M = 4 2.6 us,
// 3.2 so).
template <typename T, bool kFused>
__device__ __forceinline__ float finish(const LayerArgs& a, int64_t at, int n, float f) {
  if (a.addend) f += a.addend[at];  // the sparse correction's x . C^T term
  if (kFused) {
    const float u = a.mul ? Elt<T>::to_f32(a.mul[at]) : 1.f;
    const float r = a.res ? Elt<T>::to_f32(a.res[at]) : 0.f;
    if (a.bias) f += Elt<T>::to_f32(a.bias[n]);
    f = apply_act(a.act_fn, f);
    if (a.mul) f *= u;
    if (a.res) f += r;
  }
  return f;
}

// The same for 16 consecutive tokens tok .. tok + 15 (those below M) of output n, in two steps,
// so that a kernel can issue the loads well before it has the sums.
struct EpilogueIn {
  uint16_t mul[16], res[16];
};
__device__ __forceinline__ void load_tokens16(const uint16_t* p, int64_t at, int N, int have, uint16_t (&v)[16]) {
  p += at;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    v[i] = i < have ? *p : (uint16_t)0;
    p += N;
  }
}
__device__ __forceinline__ void load_epilogue16(const LayerArgs& a, int tok, int n, bool valid, EpilogueIn& in) {
  const int have = valid ? a.M - tok : 0;
  const int64_t at = (int64_t)tok * a.N + n;
  if (a.mul) load_tokens16(a.mul, at, a.N, have, in.mul);
  if (a.res) load_tokens16(a.res, at, a.N, have, in.res);
}

// bias: of output n, 0 without one.
template <typename T, bool kFused>
__device__ __forceinline__ void finish16(const LayerArgs& a, int tok, int n, float bias, const EpilogueIn& in,
                                         float (&f)[16]) {
  if (a.addend) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (tok + i < a.M) f[i] += a.addend[(int64_t)(tok + i) * a.N + n];
  }
  if (kFused) {
    if (a.bias) {
#pragma unroll
      for (int i = 0; i < 16; ++i) f[i] += bias;
    }
    apply_act_all(a.act_fn, f);
    if (a.mul) {
#pragma unroll
      for (int i = 0; i < 16; ++i) f[i] *= Elt<T>::to_f32(in.mul[i]);
    }
    if (a.res) {
#pragma unroll
      for (int i = 0; i < 16; ++i) f[i] += Elt<T>::to_f32(in.res[i]);
    }
  }
}

}  // namespace vq
