// Routing (vq_router_forward) and its inverse (vq_experts_combine).
//
// Routing.  For token t with logits l: the k largest (equal logits: the lower expert
// number first), their softmax weights, and the (token, choice) pairs in the order of
// their experts (a stable counting sort).  Bytes: the logits once, 16 per pair.
//   - One warp per token; lane i holds the logits of experts i, i + 32, ... as unsigned
//     keys whose order is that of the numbers (0: masked).  A choice is two warp-wide
//     integer reductions (the largest key, then the lowest expert that has it), so ties
//     are decided exactly and no sort of the row is needed.
//   - The sort needs every pair's rank among the pairs of its expert.  A block owns
//     consecutive tokens; a warp counts its pairs per expert as it walks its tokens (a
//     token's experts are distinct, so its lanes never meet), and an exclusive scan of
//     the warps' counts, in token order, makes those counts ranks.  Blocks
//     are combined by a second kernel: every block's counts go to a [blocks][E] table,
//     and each block of the second kernel sums the counts of the blocks before its own
//     and of all blocks.  No atomic decides an order: the result is the same every time.
//   - Up to 2 kRouteTile tokens one block does all of it in one launch.
// A prompt is bound by the choices' instructions, a chain of reductions each: 8192 tokens of 128
// experts, k = 8, take 15 us, nearly all of it in the first kernel, which uses half of its issue
// slots and moves 4.2 MB.
//
// Combine.  out[t] = sum_j w[t][j] y[slot[t][j]] + residual[t]: every y row is read once
// and every output row written once, 16 bytes a thread, the k loads of a thread in
// flight together: bound by HBM (see combine_kernel).
#include <new>

#include "api_util.h"
#include "common.cuh"

namespace vq {

constexpr int kRouteWarps = 16;
constexpr int kRouteThreads = 32 * kRouteWarps;
constexpr int kRouteMaxE = 512;
constexpr int kRouteMaxK = 32;
constexpr int kRoutePer = 4;      // tokens of a warp that are chosen and ranked together
constexpr int kRouteTile = kRoutePer * kRouteWarps;
constexpr int kRouteBlocks = 128; // blocks of the two-kernel form, at most
constexpr int kRouteMaxT = 1 << 30; // token numbers, rounded up to whole tiles, stay 32-bit

struct RouteArgs {
  const void* logits;
  int32_t* ids;
  float* weights;
  int32_t* offsets;
  int32_t* rows;
  int32_t* slots;
  int32_t* counts;  // [blocks][E] (the two-kernel form)
  int T, E, k, renorm;
  int tokens_per_block;
};

// Unsigned key in the order of the numbers; NaN and -inf (masked) get 0, which no
// other number has (-FLT_MAX has 0x00800000).
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v);
  const uint32_t key = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  return (v != v || b == 0xFF800000u) ? 0u : key;
}
__device__ __forceinline__ float key_value(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? (key & 0x7FFFFFFFu) : ~key);
}

template <typename L> __device__ __forceinline__ float load_logit(const void* p, int64_t i) {
  return Elt<L>::to_f32(static_cast<const uint16_t*>(p)[i]);
}
template <> __device__ __forceinline__ float load_logit<float>(const void* p, int64_t i) {
  return static_cast<const float*>(p)[i];
}

// The keys of token t: lane i holds those of experts i, i + 32, ... (E <= 32 EPL).
template <typename L, int EPL>
__device__ __forceinline__ void load_keys(const RouteArgs& a, int t, int lane, uint32_t (&key)[EPL]) {
  float v[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i)
    v[i] = lane + 32 * i < a.E ? load_logit<L>(a.logits, (int64_t)t * a.E + lane + 32 * i) : __uint_as_float(0xFF800000u);
#pragma unroll
  for (int i = 0; i < EPL; ++i) key[i] = order_key(v[i] + 0.f);  // -0 and +0 are equal logits: one key
}

// The choices of P tokens by one warp, from their keys: lane j < k ends with choice j of token
// q (expert or -1) and its weight.  The tokens' chains of reductions are independent, so a warp
// that has several of them waits for one latency instead of P.
template <int EPL, int P>
__device__ __forceinline__ void choose(const RouteArgs& a, uint32_t (&key)[P][EPL], int lane, int (&id)[P],
                                       float (&w)[P]) {
  uint32_t best[P], m[P], top[P], mine[P];  // this lane's largest key, the warp's, the token's, the chosen one's
  float all[P];
#pragma unroll
  for (int q = 0; q < P; ++q) {
    best[q] = 0u;
#pragma unroll
    for (int i = 0; i < EPL; ++i) best[q] = max(best[q], key[q][i]);
    m[q] = __reduce_max_sync(0xffffffffu, best[q]);
    id[q] = -1;
    mine[q] = 0u;
    all[q] = 0.f;
  }
#pragma unroll
  for (int q = 0; q < P; ++q) top[q] = m[q];
  if (!a.renorm) {  // the sum over all experts, while every key is still there
#pragma unroll
    for (int q = 0; q < P; ++q) {
      const float mx = key_value(top[q]);
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (key[q][i]) all[q] += key[q][i] == top[q] ? 1.f : expf(key_value(key[q][i]) - mx);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int q = 0; q < P; ++q) all[q] += __shfl_xor_sync(0xffffffffu, all[q], o);
  }
  for (int j = 0; j < a.k; ++j) {
    int e[P], win[P];
#pragma unroll
    for (int q = 0; q < P; ++q) {
      e[q] = kRouteMaxE;
      if (best[q] == m[q]) {
#pragma unroll
        for (int i = EPL - 1; i >= 0; --i)
          if (key[q][i] == m[q]) e[q] = lane + 32 * i;
      }
    }
#pragma unroll
    for (int q = 0; q < P; ++q) win[q] = __reduce_min_sync(0xffffffffu, e[q]);
#pragma unroll
    for (int q = 0; q < P; ++q) {
      if (lane == j && m[q] != 0u) {  // 0: nothing unmasked is left
        id[q] = win[q];
        mine[q] = m[q];
      }
      if (win[q] == e[q]) {  // this lane's expert was taken (or every key is 0 already)
        best[q] = 0u;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          if (lane + 32 * i == win[q]) key[q][i] = 0u;
          best[q] = max(best[q], key[q][i]);
        }
      }
    }
#pragma unroll
    for (int q = 0; q < P; ++q) m[q] = __reduce_max_sync(0xffffffffu, best[q]);
  }
  float p[P];
#pragma unroll
  for (int q = 0; q < P; ++q) {
    p[q] = 0.f;
    if (id[q] >= 0) p[q] = mine[q] == top[q] ? 1.f : expf(key_value(mine[q]) - key_value(top[q]));
    if (a.renorm) all[q] = p[q];
  }
  if (a.renorm) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int q = 0; q < P; ++q) all[q] += __shfl_xor_sync(0xffffffffu, all[q], o);
  }
#pragma unroll
  for (int q = 0; q < P; ++q) w[q] = id[q] >= 0 ? p[q] / all[q] : 0.f;
}

// Shared memory of a block: running counts of its experts before the current tile, and
// the tile's per-warp counts.
struct RouteSmem {
  int base[kRouteMaxE];               // pairs of expert e in this block's earlier tiles
  int cnt[kRouteWarps][kRouteMaxE];   // then: the pairs of the warps before
  int scan[kRouteThreads / 32];
};

// Choices and ranks of tokens [t0, t1): writes ids and weights, and into slots the rank of
// every pair among the block's pairs of its expert (-1 for a masked place).  On return
// sm.base[e] counts the block's pairs.
template <typename L, int EPL, int P>
__device__ __forceinline__ void choose_and_rank(const RouteArgs& a, int t0, int t1, RouteSmem& sm) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kTile = P * kRouteWarps;  // tokens ranked together: P of a warp
  for (int e = tid; e < a.E; e += kRouteThreads) sm.base[e] = 0;
  for (int tile = t0; tile < t1; tile += kTile) {
    uint32_t key[P][EPL];  // the logits of the warp's tokens are loaded together
#pragma unroll
    for (int q = 0; q < P; ++q) {
      if (tile + P * warp + q < t1) {
        load_keys<L, EPL>(a, tile + P * warp + q, lane, key[q]);
      } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i) key[q][i] = 0u;
      }
    }
    for (int e = lane; e < a.E; e += 32) sm.cnt[warp][e] = 0;
    __syncwarp();
    int id[P], rank[P];
    float w[P];
    choose<EPL, P>(a, key, lane, id, w);
#pragma unroll
    for (int q = 0; q < P; ++q) {
      const int t = tile + P * warp + q;
      rank[q] = 0;
      if (t < t1 && lane < a.k) {
        a.ids[(int64_t)t * a.k + lane] = id[q];
        a.weights[(int64_t)t * a.k + lane] = w[q];
      }
      // a token's experts are distinct, so its pairs do not rank against each other
      if (id[q] >= 0) {
        rank[q] = sm.cnt[warp][id[q]];
        sm.cnt[warp][id[q]] = rank[q] + 1;
      }
      __syncwarp();
    }
    __syncthreads();
    for (int e = tid; e < a.E; e += kRouteThreads) {  // exclusive scan over the warps, on top of base
      int run = sm.base[e];
#pragma unroll
      for (int w = 0; w < kRouteWarps; ++w) {
        const int c = sm.cnt[w][e];
        sm.cnt[w][e] = run;
        run += c;
      }
      sm.base[e] = run;
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < P; ++q) {
      const int t = tile + P * warp + q;
      if (t < t1 && lane < a.k)
        a.slots[(int64_t)t * a.k + lane] = id[q] >= 0 ? sm.cnt[warp][id[q]] + rank[q] : -1;
    }
    __syncthreads();  // cnt is cleared again
  }
}

// Exclusive prefix sums over the experts of total[0 .. E), in place; total's sum goes to
// every thread.  E <= kRouteThreads.
__device__ __forceinline__ int scan_experts(int* total, int E, int* part) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int v = tid < E ? total[tid] : 0, s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += u;
  }
  if (lane == 31) part[warp] = s;
  __syncthreads();
  int before = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < kRouteWarps; ++w) {
    if (w < warp) before += part[w];
    sum += part[w];
  }
  if (tid < E) total[tid] = before + s - v;
  __syncthreads();
  return sum;
}

// Turns the ranks in slots into places and fills rows: first[e] is the place of the
// block's first pair of expert e.
__device__ __forceinline__ void place_pairs(const RouteArgs& a, int t0, int t1, const int* first) {
  const int64_t end = (int64_t)t1 * a.k;
  for (int64_t i = (int64_t)t0 * a.k + threadIdx.x; i < end; i += kRouteThreads) {
    const int e = a.ids[i];
    if (e < 0) continue;
    const int at = first[e] + a.slots[i];
    a.slots[i] = at;
    a.rows[at] = (int)(i / a.k);
  }
}

// P: tokens of a warp at a time.  kOne: this block does everything.
template <typename L, int EPL, int P, bool kOne>
__global__ void __launch_bounds__(kRouteThreads) route_kernel(RouteArgs a) {
  __shared__ RouteSmem sm;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int t0 = blockIdx.x * a.tokens_per_block, t1 = min(a.T, t0 + a.tokens_per_block);
  choose_and_rank<L, EPL, P>(a, t0, t1, sm);
  if (kOne) {
    __syncthreads();
    const int sum = scan_experts(sm.base, a.E, sm.scan);
    for (int e = threadIdx.x; e < a.E; e += kRouteThreads) a.offsets[e] = sm.base[e];
    if (threadIdx.x == 0) a.offsets[a.E] = sum;
    place_pairs(a, t0, t1, sm.base);  // this block's own ids and slots, written before the barriers
  } else {
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += kRouteThreads) a.counts[(int64_t)blockIdx.x * a.E + e] = sm.base[e];
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// The second kernel: blocks and their tokens as in the first.
__global__ void __launch_bounds__(kRouteThreads) route_place_kernel(RouteArgs a) {
  __shared__ int before[kRouteMaxE], total[kRouteMaxE], part[kRouteThreads / 32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, nb = gridDim.x;
  for (int e = tid; e < a.E; e += kRouteThreads) before[e] = total[e] = 0;
  __syncthreads();
  // threads over (part of the blocks, expert): consecutive threads take consecutive experts
  const int parts = max(1, kRouteThreads / a.E);
  const int e = tid % a.E, pt = tid / a.E;
  if (pt < parts) {
    int b = 0, s = 0;
#pragma unroll 8
    for (int i = pt; i < nb; i += parts) {
      const int c = a.counts[(int64_t)i * a.E + e];
      if (i < (int)blockIdx.x) b += c;
      s += c;
    }
    atomicAdd(&before[e], b);  // integers: the order does not matter
    atomicAdd(&total[e], s);
  }
  __syncthreads();
  const int sum = scan_experts(total, a.E, part);
  if (blockIdx.x == 0) {
    for (int i = tid; i < a.E; i += kRouteThreads) a.offsets[i] = total[i];
    if (tid == 0) a.offsets[a.E] = sum;
  }
  for (int i = tid; i < a.E; i += kRouteThreads) before[i] += total[i];
  __syncthreads();
  const int t0 = blockIdx.x * a.tokens_per_block;
  place_pairs(a, t0, min(a.T, t0 + a.tokens_per_block), before);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

static cudaError_t launch_pdl(void (*kern)(RouteArgs), int grid, const RouteArgs& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kRouteThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

// Tokens that one block routes in one launch; more are cut over kRouteBlocks blocks.
static int route_blocks(int T) {
  if (T <= 2 * kRouteTile) return 1;
  const int tiles = (T + kRouteTile - 1) / kRouteTile;
  return tiles < kRouteBlocks ? tiles : kRouteBlocks;
}

template <typename L, int EPL>
static cudaError_t launch_route_t(RouteArgs a, cudaStream_t s) {
  const int blocks = route_blocks(a.T);
  if (blocks == 1) {
    a.tokens_per_block = a.T;
    // up to a token a warp, the other three would only be instructions
    return a.T <= kRouteWarps ? launch_pdl(route_kernel<L, EPL, 1, true>, 1, a, s)
                              : launch_pdl(route_kernel<L, EPL, kRoutePer, true>, 1, a, s);
  }
  const int tiles = (a.T + kRouteTile - 1) / kRouteTile;
  a.tokens_per_block = (tiles + blocks - 1) / blocks * kRouteTile;
  const int grid = (a.T + a.tokens_per_block - 1) / a.tokens_per_block;
  cudaError_t e = launch_pdl(route_kernel<L, EPL, kRoutePer, false>, grid, a, s);
  return e != cudaSuccess ? e : launch_pdl(route_place_kernel, grid, a, s);
}

template <typename L>
static cudaError_t launch_route(const RouteArgs& a, cudaStream_t s) {
  if (a.E <= 64) return launch_route_t<L, 2>(a, s);
  if (a.E <= 128) return launch_route_t<L, 4>(a, s);
  if (a.E <= 256) return launch_route_t<L, 8>(a, s);
  return launch_route_t<L, 16>(a, s);
}

// ---------------------------------------------------------------------------- combine

struct CombineArgs {
  const uint16_t* y;
  const float* weights;
  const int32_t* slots;
  const uint16_t* res;
  uint16_t* out;
  int64_t total;  // T * N / 8
  int y_rows, k, N8;
};

// One thread per 8 outputs of a token.  KB rows are loaded before the first is used.
template <typename T, int KB>
__global__ void __launch_bounds__(256) combine_kernel(CombineArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i < a.total) {
    const int64_t t = i / a.N8;
    const int c = (int)(i - t * a.N8);
    float acc[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[q] = 0.f;
    uint4 r = make_uint4(0, 0, 0, 0);
    if (a.res) r = reinterpret_cast<const uint4*>(a.res)[i];
    for (int j0 = 0; j0 < a.k; j0 += KB) {
      uint4 v[KB];
      float w[KB];
      bool in[KB];
#pragma unroll
      for (int j = 0; j < KB; ++j) {
        const int s = j0 + j < a.k ? a.slots[t * a.k + j0 + j] : -1;
        in[j] = s >= 0 && s < a.y_rows;
        v[j] = in[j] ? reinterpret_cast<const uint4*>(a.y)[(int64_t)s * a.N8 + c] : make_uint4(0, 0, 0, 0);
        w[j] = in[j] ? a.weights[t * a.k + j0 + j] : 0.f;
      }
#pragma unroll
      for (int j = 0; j < KB; ++j) {
        if (!in[j]) continue;
        const uint32_t u[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          acc[2 * q] = fmaf(w[j], Elt<T>::to_f32((uint16_t)u[q]), acc[2 * q]);
          acc[2 * q + 1] = fmaf(w[j], Elt<T>::to_f32((uint16_t)(u[q] >> 16)), acc[2 * q + 1]);
        }
      }
    }
    if (a.res) {
      const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        acc[2 * q] += Elt<T>::to_f32((uint16_t)u[q]);
        acc[2 * q + 1] += Elt<T>::to_f32((uint16_t)(u[q] >> 16));
      }
    }
    reinterpret_cast<uint4*>(a.out)[i] = make_uint4(Elt<T>::pack(acc[0], acc[1]), Elt<T>::pack(acc[2], acc[3]),
                                                    Elt<T>::pack(acc[4], acc[5]), Elt<T>::pack(acc[6], acc[7]));
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <typename T>
static cudaError_t launch_combine(const CombineArgs& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.total + 255) / 256));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return a.k <= 2   ? cudaLaunchKernelEx(&cfg, combine_kernel<T, 2>, a)
         : a.k <= 4 ? cudaLaunchKernelEx(&cfg, combine_kernel<T, 4>, a)
                    : cudaLaunchKernelEx(&cfg, combine_kernel<T, 8>, a);
}

}  // namespace vq

// -------------------------------------------------------------------------------- ABI

using namespace vq;

struct vq_router_s {
  vq_router_desc d;
  int device;
  int32_t* counts;  // [kRouteBlocks][E]
};

VQ_API vq_status vq_router_create(const vq_router_desc* desc, vq_router_t* out) {
  if (out == nullptr) return fail(VQ_ERR_INVALID_ARG, "out is NULL");
  *out = nullptr;
  if (desc == nullptr) return fail(VQ_ERR_INVALID_ARG, "desc is NULL");
  if (desc->E < 1 || desc->k < 1 || desc->k > desc->E)
    return fail(VQ_ERR_INVALID_ARG, "E=%d, k=%d: need 1 <= k <= E", desc->E, desc->k);
  if (desc->E > kRouteMaxE || desc->k > kRouteMaxK)
    return fail(VQ_ERR_UNSUPPORTED, "E=%d, k=%d: at most %d experts and %d choices", desc->E, desc->k, kRouteMaxE,
                kRouteMaxK);
  if (desc->renorm != 0 && desc->renorm != 1) return fail(VQ_ERR_INVALID_ARG, "renorm=%d must be 0 or 1", desc->renorm);
  if (desc->max_T < 1 || desc->max_T > kRouteMaxT || (int64_t)desc->max_T * desc->k > INT32_MAX)
    return fail(VQ_ERR_INVALID_ARG, "max_T=%d: need 1 <= max_T <= 2^30 and max_T * k < 2^31", desc->max_T);
  DeviceInfo dev{};
  vq_status st = query_device(&dev);
  if (st) return st;
  if ((st = refuse_alloc())) return st;
  vq_router_s* h = new (std::nothrow) vq_router_s{};
  if (!h) return fail(VQ_ERR_NOMEM, "host allocation of the handle failed");
  h->d = *desc;
  h->device = dev.device;
  if (route_blocks(desc->max_T) > 1) {
    const size_t bytes = sizeof(int32_t) * kRouteBlocks * (size_t)desc->E;
    cudaError_t e = cudaMalloc(&h->counts, bytes);
    if (e != cudaSuccess) {
      delete h;
      cudaGetLastError();
      return fail(VQ_ERR_NOMEM, "cudaMalloc of %zu bytes of counts failed: %s", bytes, cudaGetErrorString(e));
    }
  }
  *out = h;
  return VQ_OK;
}

VQ_API vq_status vq_router_destroy(vq_router_t h) {
  if (h == nullptr) return VQ_OK;
  cudaError_t e = cudaSuccess;
  if (h->counts) e = free_on_device(h->device, h->counts);
  delete h;
  return e == cudaSuccess ? VQ_OK : cuda_fail(e, "vq_router_destroy");
}

VQ_API vq_status vq_router_forward(vq_router_t h, const void* logits, int32_t dtype, int32_t* ids, float* weights,
                                   int32_t* offsets, int32_t* rows, int32_t* slots, int32_t T, void* stream) {
  if (h == nullptr) return fail(VQ_ERR_INVALID_ARG, "handle is NULL");
  const vq_router_desc& d = h->d;
  if (T < 0 || T > d.max_T) return fail(VQ_ERR_INVALID_ARG, "T=%d outside [0, max_T=%d]", T, d.max_T);
  if (dtype != VQ_F16 && dtype != VQ_BF16 && dtype != VQ_F32)
    return fail(VQ_ERR_INVALID_ARG, "dtype=%d is not VQ_F16, VQ_BF16 or VQ_F32", dtype);
  vq_status st;
  if ((st = check_ptr(offsets, "offsets"))) return st;
  if (T > 0 && ((st = check_ptr(logits, "logits")) || (st = check_ptr(ids, "ids")) || (st = check_ptr(weights, "weights")) ||
                (st = check_ptr(rows, "rows")) || (st = check_ptr(slots, "slots"))))
    return st;
  if (T > 0) {
    const size_t pairs = (size_t)T * d.k * 4;
    const struct {
      const void* p;
      size_t bytes;
      const char* name;
    } bufs[6] = {{logits, (size_t)T * d.E * (dtype == VQ_F32 ? 4 : 2), "logits"}, {ids, pairs, "ids"},
                 {weights, pairs, "weights"}, {offsets, sizeof(int32_t) * (d.E + 1), "offsets"}, {rows, pairs, "rows"},
                 {slots, pairs, "slots"}};
    for (int i = 0; i < 6; ++i)
      for (int j = 0; j < i; ++j)
        if (overlaps(bufs[i].p, bufs[i].bytes, bufs[j].p, bufs[j].bytes))
          return fail(VQ_ERR_INVALID_ARG, "%s overlaps %s", bufs[i].name, bufs[j].name);
  }
  if ((st = check_current_device(h->device))) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (T == 0) {
    e = cudaMemsetAsync(offsets, 0, sizeof(int32_t) * (d.E + 1), s);
    return e == cudaSuccess ? VQ_OK : cuda_fail(e, "vq_router_forward");
  }
  RouteArgs a{};
  a.logits = logits;
  a.ids = ids;
  a.weights = weights;
  a.offsets = offsets;
  a.rows = rows;
  a.slots = slots;
  a.counts = h->counts;
  a.T = T;
  a.E = d.E;
  a.k = d.k;
  a.renorm = d.renorm;
  e = dtype == VQ_F32 ? launch_route<float>(a, s) : dtype == VQ_BF16 ? launch_route<__nv_bfloat16>(a, s) : launch_route<__half>(a, s);
  return e == cudaSuccess ? VQ_OK : cuda_fail(e, "vq_router_forward launch");
}

VQ_API vq_status vq_experts_combine(const void* y, int32_t y_rows, const float* weights, const int32_t* slots,
                                    const void* residual, void* out, int32_t T, int32_t k, int32_t N, int32_t dtype,
                                    void* stream) {
  if (T < 0 || y_rows < 0) return fail(VQ_ERR_INVALID_ARG, "T=%d and y_rows=%d must not be negative", T, y_rows);
  if (k < 1 || k > kRouteMaxK) return fail(VQ_ERR_INVALID_ARG, "k=%d outside [1, %d]", k, kRouteMaxK);
  if (N < 1) return fail(VQ_ERR_INVALID_ARG, "N=%d must be positive", N);
  if (N % 8 != 0 || N > (1 << 24)) return fail(VQ_ERR_UNSUPPORTED, "N=%d: need a multiple of 8, at most 2^24", N);
  if (dtype != VQ_F16 && dtype != VQ_BF16) return fail(VQ_ERR_INVALID_ARG, "dtype=%d is not VQ_F16 or VQ_BF16", dtype);
  if (T == 0) return VQ_OK;
  vq_status st;
  if ((y_rows > 0 && (st = check_ptr(y, "y"))) || (st = check_ptr(weights, "weights")) || (st = check_ptr(slots, "slots")) ||
      (st = check_ptr(out, "out")))
    return st;
  if (residual && (st = check_ptr(residual, "residual"))) return st;
  const size_t ob = (size_t)T * N * 2;
  if (y_rows > 0 && overlaps(y, (size_t)y_rows * N * 2, out, ob)) return fail(VQ_ERR_INVALID_ARG, "out overlaps y");
  if (residual && residual != out && overlaps(residual, ob, out, ob))
    return fail(VQ_ERR_INVALID_ARG, "out partially overlaps residual");
  if (overlaps(weights, (size_t)T * k * 4, out, ob) || overlaps(slots, (size_t)T * k * 4, out, ob))
    return fail(VQ_ERR_INVALID_ARG, "out overlaps weights or slots");
  CombineArgs a{};
  a.y = static_cast<const uint16_t*>(y);
  a.weights = weights;
  a.slots = slots;
  a.res = static_cast<const uint16_t*>(residual);
  a.out = static_cast<uint16_t*>(out);
  a.N8 = N / 8;
  a.total = (int64_t)T * a.N8;
  if ((a.total + 255) / 256 > INT32_MAX) return fail(VQ_ERR_UNSUPPORTED, "T=%d x N=%d is too large for one launch", T, N);
  a.y_rows = y_rows;
  a.k = k;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = dtype == VQ_BF16 ? launch_combine<__nv_bfloat16>(a, s) : launch_combine<__half>(a, s);
  return e == cudaSuccess ? VQ_OK : cuda_fail(e, "vq_experts_combine launch");
}
