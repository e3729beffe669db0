// Shared by the kernels of vq_experts_forward (experts_gemv.cu, experts_tc.cu): the
// arguments, the division of the work into tiles and the decode of one group.
#pragma once

#include "common.cuh"
#include "epilogue.cuh"
#include "internal.h"
#include "ladder.cuh"
#include "tc_ptx.cuh"

namespace vq {

constexpr int kMaxExperts = 1024;

// Device pointers of all experts (expert 0's; the strides follow from the shape).
struct ExpertsArgs {
  const uint16_t* x;       // [x_rows][K]
  uint16_t* y;             // [T][Nout]
  const int32_t* rows;     // [T] or NULL
  const int32_t* offsets;  // [E + 1]
  const uint16_t* bias;    // [E][N] or NULL
  uint32_t* err;           // the handle's error word
  LayerArgs w;             // planes, codebooks and scales of expert 0; N, K, fmt, scale_group, n16, n8, mult
  int E, T, x_rows;
  int Nout;                // N, or N / 2 with glu
  int act, glu, shared;    // shared: one set of codebooks
};

// Expert e's layer: every plane follows the one of the expert before.
__device__ __forceinline__ LayerArgs expert_layer(const ExpertsArgs& a, int e) {
  LayerArgs l = a.w;
  const int64_t NG = (int64_t)l.N * (l.K / 8), at = NG * e;
  l.lo += at;
  l.hi4 += at / 2;
  l.s2 += at / 2;
  l.idx16 += at * l.n16;
  l.idx8 += at;
  l.scales += l.scale_group == 64 ? at / 8 : (int64_t)l.N * e;
  if (!a.shared) {
    const int64_t big = (l.fmt == kFmtVq16 || l.fmt == kFmtVq16Rvq) ? 65536 * 8 : 4096 * 8;
    l.cb1 += big * e;
    l.cb2 += (int64_t)16 * 8 * e;
#pragma unroll
    for (int t = 0; t < 3; ++t) l.cbr[t] += (int64_t)65536 * 8 * e;
    l.cb8 += (int64_t)256 * 8 * e;
  }
  return l;
}

// The tiles of the call, found by every block from the offsets: expert e has the rows
// off[e] .. off[e+1] - 1 and the tiles start[e] .. start[e+1] - 1, RT row tiles of W times
// ceil(rows / tok) tiles of `tok` rows, the tiles of one row tile adjacent.
struct ExpertTiles {
  int off[kMaxExperts + 1];
  int start[kMaxExperts + 1];
};

// Offsets are clamped into [0, T] and to at least the one before (a running maximum), so
// the row counts are never negative and add up to at most T.  All `threads` threads of the
// block; `part` holds 2 ints per warp.
__device__ __forceinline__ void find_tiles(const ExpertsArgs& a, int tok, int RT, ExpertTiles& t, int* part,
                                           int threads) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, nw = threads / 32;
  const int per = (a.E + 1 + threads - 1) / threads;  // consecutive entries of a thread
  const int lo = min(tid * per, a.E + 1), hi = min(lo + per, a.E + 1);
  int m = 0;
  for (int e = lo; e < hi; ++e) m = max(m, min(max(a.offsets[e], 0), a.T));
  int run = m;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, run, o);
    if (lane >= o) run = max(run, u);
  }
  if (lane == 31) part[warp] = run;
  __syncthreads();
  int before = __shfl_up_sync(0xffffffffu, run, 1);
  if (lane == 0) before = 0;
  for (int w = 0; w < warp; ++w) before = max(before, part[w]);
  for (int e = lo; e < hi; ++e) {
    before = max(before, min(max(a.offsets[e], 0), a.T));
    t.off[e] = before;
  }
  __syncthreads();
  int n = 0;
  for (int e = lo; e < min(hi, a.E); ++e) n += RT * ((t.off[e + 1] - t.off[e] + tok - 1) / tok);
  int sum = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += u;
  }
  if (lane == 31) part[nw + warp] = sum;
  __syncthreads();
  int at = sum - n;
  for (int w = 0; w < warp; ++w) at += part[nw + w];
  for (int e = lo; e < hi; ++e) {
    t.start[e] = at;
    if (e < a.E) at += RT * ((t.off[e + 1] - t.off[e] + tok - 1) / tok);
  }
  __syncthreads();
}

// The expert that tile u belongs to (start[e] <= u < start[e+1]).
__device__ __forceinline__ int expert_of(const ExpertTiles& t, int E, int u) {
  int lo = 0, hi = E;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.start[mid] <= u) lo = mid; else hi = mid;
  }
  return lo;
}

// One group of a one- or two-stage format, with the rounding of the materialised weights
// (vq_debug_dequant): w_j = RN_T(fl32(s * fl32(c1_j + c2_j))).  The MMAs take both operands in x's
// 16-bit type, so W is rounded to it, as on the single layer's paths; against fp32 weights the error
// of a gated bf16 product grows from 1.6e-3 to 2.9e-3 (relative norm, the result's rounding in both),
// of a plain bf16 one to 2.3e-3, of fp16 ones from 2.1e-4 to 2.3e-4 .. 2.8e-4.  Forming s c1 + s c2 with
// two mixed-precision multiply-adds a weight was no faster, and the sum in packed fp16 gained 2 %
// for one rounding more: the decode waits for the shared-memory pipe (9 wavefronts a gather of 32
// codewords, 4 for the shuffles), not for its arithmetic.
template <typename T, bool kTwo>
__device__ __forceinline__ void decode_scaled(const uint4& c1, const uint32_t (&c2)[4], unsigned short s,
                                              uint32_t* out) {
  const uint32_t w1[4] = {c1.x, c1.y, c1.z, c1.w};
  const uint32_t sb = __float_as_uint(__half2float(__ushort_as_half(s)));
  const uint64_t sv = (uint64_t)sb | ((uint64_t)sb << 32);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float lo, hi;
    if (kTwo) {
      const float2 b = f16x2_to_f32x2(c2[q]);
      asm("{ .reg .f16 l, h; mov.b32 {l, h}, %2; add.rn.f32.f16 %0, l, %3; add.rn.f32.f16 %1, h, %4; }"
          : "=f"(lo), "=f"(hi)
          : "r"(w1[q]), "f"(b.x), "f"(b.y));
    } else {
      const float2 a = f16x2_to_f32x2(w1[q]);
      lo = a.x;
      hi = a.y;
    }
    uint64_t m;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(m)
        : "l"((uint64_t)__float_as_uint(lo) | ((uint64_t)__float_as_uint(hi) << 32)), "l"(sv));
    out[q] = Elt<T>::pack(__uint_as_float((uint32_t)m), __uint_as_float((uint32_t)(m >> 32)));
  }
}

// One output of a gated matrix; gate and up have their bias.
__device__ __forceinline__ float gated(int act, float gate, float up) { return apply_act(act, gate) * up; }

}  // namespace vq
