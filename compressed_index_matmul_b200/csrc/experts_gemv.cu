// Products grouped by expert for few rows per expert (vq_experts_forward): y[r] =
// act(x[rows[r]] . W_e^T + b), decoded in registers and multiplied with warp MMAs.
//
// With a handful of rows per expert the decode of W is the work (2 N K / 8 codeword
// gathers per expert, whatever the row count), so the kernel is built around it:
//   tile    16 rows of W (glu: 8 gate rows and the 8 up rows that go with them) x up to 16
//           rows of x, over all of K; the tiles of all experts are numbered in expert order
//           (find_tiles) and cut into one contiguous, equal range per block
//   block   16 decode warps and a producer warp, one block per SM.  The decode warps form
//           groups of wk warps; a group takes a tile at a time and its warps take the
//           128-input slices of K in turn.  A warp walks (tile, slice) as one sequence and
//           loads the index bytes of its next slice before it decodes the current one, across
//           tiles and experts too, so the index loads are never waited for at a tile's end
//   lane    (g, c) = (lane / 4, lane % 4): rows g and g + 8 of the tile, groups 4 i + c of
//           the slice (i = 0 .. 3).  The decoded group is a fragment of mma m16n8k16's A
//           operand as it stands: MMA 2 i + h takes elements 4 h .. 4 h + 3, the same
//           permutation of k on both operands, so x comes as 16-byte loads, 64 contiguous bytes
//           per row
// The 12-bit codebooks (64 KiB an expert) live in shared memory in two slots: the producer
// copies the next expert's while the current one is used; a decode warp arrives on a slot's
// barrier when it leaves an expert.  The 16-bit codebooks are gathered through L2.
// The warps of a group meet once per tile, at a named barrier, and add their sums in warp order
// (two buffers, so one barrier suffices); the other groups go on meanwhile.  The result of a
// row does not depend on the other rows.
#include "experts.cuh"

namespace vq {

constexpr int kXgWarps = 16;                       // decode warps
constexpr int kXgThreads = 32 * (kXgWarps + 1);    // + the producer
constexpr int kXgTok = 16;                         // x rows of a tile
constexpr int kXgRedStride = 20;                   // floats per token of a warp's sums (16 rows; conflict-free)
constexpr int kXgRedWarp = kXgTok * kXgRedStride;  // floats of a warp's sums
constexpr int kXgSlot12 = 65536 + 256;             // a codebook slot: cb1, cb2
constexpr int kXgSlot8 = 4096;                     // the ladder's 8-bit codebook

struct XgSmem {
  int tiles, red, bars, bytes;
};
__host__ __device__ constexpr XgSmem xg_smem(int fmt) {
  XgSmem s{};
  const int slot = fmt == kFmtVq16 ? 0 : fmt == kFmtVq16Rvq ? kXgSlot8 : kXgSlot12;
  s.red = 2 * slot;
  s.tiles = s.red + 2 * kXgWarps * kXgRedWarp * 4;
  s.bars = (s.tiles + (int)sizeof(ExpertTiles) + 15) / 16 * 16;
  s.bytes = s.bars + 256;
  return s;
}

// Index bytes of one row's slice (w = 16 groups, or 8 in a 64-wide last one) and its scales.
template <int FMT> struct XgIdx {
  uint32_t lo[4], hi[2], s2[2], sc;
};
template <> struct XgIdx<kFmtVq16> {
  uint32_t lo[8], sc;
};
template <> struct XgIdx<kFmtVq16Rvq> {
  uint32_t lo[8], sc;
};

template <int FMT>
__device__ __forceinline__ void load_row(const LayerArgs& l, int s, int n, bool valid, XgIdx<FMT>& q) {
  constexpr bool k16 = (FMT == kFmtVq16 || FMT == kFmtVq16Rvq);
  q = XgIdx<FMT>{};
  if (!valid) return;
  const int w = slice_width(s, l.K / 8);
  const int64_t e = (int64_t)16 * s * l.N + (int64_t)n * w;
  if constexpr (k16) {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(l.idx16 + e));
    q.lo[0] = a.x; q.lo[1] = a.y; q.lo[2] = a.z; q.lo[3] = a.w;
    if (w == 16) {
      const uint4 b = __ldg(reinterpret_cast<const uint4*>(l.idx16 + e) + 1);
      q.lo[4] = b.x; q.lo[5] = b.y; q.lo[6] = b.z; q.lo[7] = b.w;
    }
  } else if (w == 16) {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(l.lo + e));
    const uint2 h = __ldg(reinterpret_cast<const uint2*>(l.hi4 + e / 2));
    q.lo[0] = a.x; q.lo[1] = a.y; q.lo[2] = a.z; q.lo[3] = a.w;
    q.hi[0] = h.x; q.hi[1] = h.y;
    if (FMT == kFmtRvq12_4) {
      const uint2 r = __ldg(reinterpret_cast<const uint2*>(l.s2 + e / 2));
      q.s2[0] = r.x; q.s2[1] = r.y;
    }
  } else {
    const uint2 a = __ldg(reinterpret_cast<const uint2*>(l.lo + e));
    q.lo[0] = a.x; q.lo[1] = a.y;
    q.hi[0] = __ldg(reinterpret_cast<const uint32_t*>(l.hi4 + e / 2));
    if (FMT == kFmtRvq12_4) q.s2[0] = __ldg(reinterpret_cast<const uint32_t*>(l.s2 + e / 2));
  }
  if (l.scale_group == 64) {  // one scale per 8 groups: 2 (or 1) per row and slice
    if (w == 16) q.sc = __ldg(reinterpret_cast<const uint32_t*>(l.scales + e / 8));
    else q.sc = __ldg(l.scales + e / 8);
  } else {
    q.sc = __ldg(l.scales + n) * 0x10001u;
  }
}

// A warp's place in its sequence of (tile, slice).
struct XgWalk {
  int u, s;  // tile and slice; u >= end: done
  int e;     // the tile's expert
  int rt, tk;
};

template <int FMT, typename T>
__global__ void __launch_bounds__(kXgThreads, 1) experts_gemv_kernel(const __grid_constant__ ExpertsArgs a, int wk) {
  extern __shared__ __align__(128) unsigned char smem[];
  constexpr bool k16 = (FMT == kFmtVq16 || FMT == kFmtVq16Rvq);
  constexpr bool kTwo = (FMT == kFmtRvq12_4);
  constexpr bool kLadder = (FMT == kFmtVq16Rvq);
  constexpr bool kBook = (FMT != kFmtVq16);  // a codebook in shared memory
  constexpr int kSlot = k16 ? kXgSlot8 : kXgSlot12;
  constexpr XgSmem lay = xg_smem(FMT);
  float* red = reinterpret_cast<float*>(smem + lay.red);
  ExpertTiles& tiles = *reinterpret_cast<ExpertTiles*>(smem + lay.tiles);
  const uint32_t bars = smem_u32(smem + lay.bars);
  auto full = [&](int i) { return bars + 8u * i; };
  auto empty = [&](int i) { return bars + 16u + 8u * i; };
  volatile int* abortf = reinterpret_cast<volatile int*>(smem + lay.bars + 32);
  int* part = reinterpret_cast<int*>(smem + lay.bars + 64);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int N = a.w.N, K = a.w.K;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(full(i), 1);
      ptx::mbar_init(empty(i), kXgWarps);
    }
    *abortf = 0;
    ptx::fence_barrier_init();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int per_tile = a.glu ? 8 : 16;  // outputs of a tile
  find_tiles(a, kXgTok, (a.Nout + per_tile - 1) / per_tile, tiles, part, kXgThreads);
  const int total = tiles.start[a.E];
  const int ubeg = (int)((int64_t)total * blockIdx.x / gridDim.x), uend = (int)((int64_t)total * (blockIdx.x + 1) / gridDim.x);
  if (ubeg >= uend) return;

  if (warp == kXgWarps) {
    // ------------------------------------------------------------ producer
    if (kBook && lane == 0) {
      const int e0 = expert_of(tiles, a.E, ubeg);
      int i = 0;
      for (int e = e0; e < a.E && tiles.start[e] < uend; ++e) {
        if (tiles.start[e] == tiles.start[e + 1]) continue;  // no rows
        if (a.shared && i > 0) break;
        if (i >= 2 && (*abortf || !ptx::mbar_wait(empty(i & 1), ((i >> 1) - 1) & 1, a.err))) {
          *abortf = 1;
          break;
        }
        const uint32_t dst = smem_u32(smem) + kSlot * (i & 1), bar = full(i & 1);
        const int64_t at = a.shared ? 0 : e;
        if (k16) {
          if (a.w.n8 == 0) break;
          ptx::mbar_arrive_expect_tx(bar, kXgSlot8);
          ptx::bulk_load(dst, a.w.cb8 + at * 256 * 8, kXgSlot8, bar);
        } else {
          ptx::mbar_arrive_expect_tx(bar, 65536u + (kTwo ? 256u : 0u));
          ptx::bulk_load(dst, a.w.cb1 + at * 4096 * 8, 65536u, bar);
          if (kTwo) ptx::bulk_load(dst + 65536u, a.w.cb2 + at * 16 * 8, 256u, bar);
        }
        ++i;
      }
      // Do not leave while a copy into this block's shared memory may be in flight.
      for (int j = i > 2 ? i - 2 : 0; j < i; ++j) ptx::mbar_wait(full(j & 1), (j >> 1) & 1, a.err);
    }
    return;
  }

  // -------------------------------------------------------------- decode
  const int g = lane >> 2, c = lane & 3;
  const int grp = warp / wk, kp = warp % wk, ngrp = kXgWarps / wk;
  const int nsl = (K + 127) / 128;
  const bool books = kBook && (!k16 || a.w.n8);
  const uint32_t csel = 0x4440u | (uint32_t)c;  // byte c, zero-extended
  const uint32_t c4 = 4u * c;

  auto set_tile = [&](XgWalk& w) {
    while (w.e + 1 < a.E && w.u >= tiles.start[w.e + 1]) ++w.e;
    const int tt = (tiles.off[w.e + 1] - tiles.off[w.e] + kXgTok - 1) / kXgTok;
    const int local = w.u - tiles.start[w.e];
    w.rt = local / tt;
    w.tk = local - w.rt * tt;
  };
  auto tile_rows = [&](const XgWalk& w, int (&n)[2], bool (&ok)[2]) {
    if (a.glu) {
      n[0] = 8 * w.rt + g;
      n[1] = a.Nout + n[0];
      ok[0] = ok[1] = n[0] < a.Nout;
    } else {
      n[0] = 16 * w.rt + g;
      n[1] = n[0] + 8;
      ok[0] = n[0] < N;
      ok[1] = n[1] < N;
    }
  };
  auto load_slice = [&](const XgWalk& w, XgIdx<FMT> (&q)[2]) {
    int n[2];
    bool ok[2];
    tile_rows(w, n, ok);
    const LayerArgs l = expert_layer(a, w.e);
    load_row<FMT>(l, w.s, n[0], ok[0], q[0]);
    load_row<FMT>(l, w.s, n[1], ok[1], q[1]);
  };

  XgWalk cur{};
  cur.u = ubeg + grp;
  cur.s = kp;
  cur.e = expert_of(tiles, a.E, ubeg);
  int book_e = cur.e, book_i = 0;  // the expert whose slot this warp uses, and its place in the producer's sequence
  bool book_ready = false;
  XgIdx<FMT> iq[2], nq[2];
  if (cur.u < uend) {
    set_tile(cur);
    if (cur.s < nsl) load_slice(cur, iq);
  }
  int tok_e = -1, tok_tk = -1;
  const uint16_t* xp[2] = {a.x, a.x};
  bool xin[2] = {false, false};
  int nt = 1;
  uint32_t cb2r[4] = {0, 0, 0, 0};
  const uint4* cbs = reinterpret_cast<const uint4*>(smem);
  int buf = 0;

  // Past the bound (never on a healthy device) the sums are wrong and the error word is set.
  auto wait_book = [&]() {
    if (!*abortf && !ptx::mbar_wait(full(book_i & 1), (book_i >> 1) & 1, a.err)) *abortf = 1;
    book_ready = true;
  };
  // Go on from expert book_e; one with rows has a place in the producer's sequence, and its
  // copy must have landed before its slot is given back (an arrival made earlier would count
  // for the slot's expert before).
  auto leave_expert = [&]() {
    if (tiles.start[book_e + 1] > tiles.start[book_e]) {
      if (!book_ready) wait_book();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(empty(book_i & 1));
      ++book_i;
      book_ready = false;
    }
    ++book_e;
  };

  while (cur.u < uend) {
    const int u = cur.u;
    if (books) {
      while (!a.shared && book_e < cur.e) leave_expert();
      if (!book_ready) {
        wait_book();
        cbs = reinterpret_cast<const uint4*>(smem + kSlot * (book_i & 1));
        if (kTwo) {
          const uint4 v = cbs[4096 + (lane & 15)];
          cb2r[0] = v.x; cb2r[1] = v.y; cb2r[2] = v.z; cb2r[3] = v.w;
        }
      }
    }
    if (tok_e != cur.e || tok_tk != cur.tk) {
      tok_e = cur.e;
      tok_tk = cur.tk;
      const int first = tiles.off[cur.e] + kXgTok * cur.tk, last = tiles.off[cur.e + 1];
      nt = last - first > 8 ? 2 : 1;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int r = first + 8 * t + g;
        const int xr = r < last ? (a.rows ? a.rows[r] : r) : -1;
        xin[t] = xr >= 0 && xr < a.x_rows;
        xp[t] = a.x + (int64_t)(xin[t] ? xr : 0) * K + 8 * c;
      }
    }
    float acc[2][4];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[t][i] = 0.f;
    const LayerArgs l = expert_layer(a, cur.e);
    int rown[2];
    bool rok[2];
    tile_rows(cur, rown, rok);

    XgWalk nxt = cur;
    for (int s = kp; s < nsl; s += wk) {
      nxt.s = s + wk;
      if (nxt.s >= nsl) {
        nxt.s = kp;
        nxt.u = u + ngrp;
        if (nxt.u < uend) set_tile(nxt);
      }
      if (nxt.u < uend) load_slice(nxt, nq);
      const int w = slice_width(s, K / 8);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (4 * i >= w) break;
        uint4 xq[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          xq[t] = make_uint4(0, 0, 0, 0);
          if (t < nt && xin[t]) xq[t] = *reinterpret_cast<const uint4*>(xp[t] + 128 * s + 32 * i);
        }
        uint32_t wq[2][4];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const unsigned short sc = (unsigned short)(i < 2 ? iq[r].sc : iq[r].sc >> 16);
          uint32_t i1;
          uint32_t c2[4] = {0, 0, 0, 0};
          if constexpr (k16) {
            i1 = ((c & 2 ? iq[r].lo[2 * i + 1] : iq[r].lo[2 * i]) >> (16 * (c & 1))) & 0xFFFFu;
          } else {
            uint32_t b;
            asm("prmt.b32 %0, %1, 0, %2;" : "=r"(b) : "r"(iq[r].lo[i]), "r"(csel));
            i1 = b | (((iq[r].hi[i >> 1] >> (16 * (i & 1) + c4)) & 15u) << 8);
            if (kTwo) {
              const int i2 = (int)((iq[r].s2[i >> 1] >> (16 * (i & 1) + c4)) & 15u);
#pragma unroll
              for (int v = 0; v < 4; ++v) c2[v] = __shfl_sync(0xffffffffu, cb2r[v], i2);
            }
          }
          const uint4 c1 = k16 ? __ldg(reinterpret_cast<const uint4*>(l.cb1) + i1) : cbs[i1];
          if constexpr (kLadder) {
            float v[8];
            const uint32_t w1[4] = {c1.x, c1.y, c1.z, c1.w};
#pragma unroll
            for (int p = 0; p < 4; ++p) {
              const float2 f = f16x2_to_f32x2(w1[p]);
              v[2 * p] = f.x;
              v[2 * p + 1] = f.y;
            }
            const int64_t ent = (int64_t)16 * s * N + (int64_t)rown[r] * w + 4 * i + c, NG = (int64_t)N * (K / 8);
#pragma unroll
            for (int t = 2; t <= 4; ++t) {
              if (!rok[r]) continue;
              if (t <= l.n16)
                fma_codeword(l.mult[t - 2], __ldg(reinterpret_cast<const uint4*>(l.cbr[t - 2]) + __ldg(l.idx16 + (t - 1) * NG + ent)), v);
              else if (t == l.n16 + 1 && l.n8)
                fma_codeword(l.mult[t - 2], cbs[__ldg(l.idx8 + ent)], v);
            }
            pack_scaled<T>(v, __half2float(__ushort_as_half(sc)), wq[r]);
          } else {
            decode_scaled<T, kTwo>(c1, c2, sc, wq[r]);
          }
        }
        const uint32_t af0[4] = {wq[0][0], wq[1][0], wq[0][1], wq[1][1]};
        const uint32_t af1[4] = {wq[0][2], wq[1][2], wq[0][3], wq[1][3]};
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (t < nt) {
            Mma16816<T>::run(acc[t], af0, xq[t].x, xq[t].y);
            Mma16816<T>::run(acc[t], af1, xq[t].z, xq[t].w);
          }
        }
      }
      iq[0] = nq[0];
      iq[1] = nq[1];
    }

    // The group's sums: [token][row of the tile], this warp's share of K.
    float* mine = red + (buf * kXgWarps + warp) * kXgRedWarp;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      if (t < nt) {
        float* p = mine + (8 * t + 2 * c) * kXgRedStride + g;
        p[0] = acc[t][0];
        p[kXgRedStride] = acc[t][1];
        p[8] = acc[t][2];
        p[kXgRedStride + 8] = acc[t][3];
      }
    }
    asm volatile("bar.sync %0, %1;" ::"r"(1 + grp), "r"(32 * wk) : "memory");
    {
      const float* src = red + (buf * kXgWarps + grp * wk) * kXgRedWarp;
      const int first = tiles.off[cur.e] + kXgTok * cur.tk, have = min(tiles.off[cur.e + 1] - first, kXgTok);
      const uint16_t* bias = a.bias ? a.bias + (int64_t)cur.e * N : nullptr;
      for (int o = 32 * kp + lane; o < per_tile * have; o += 32 * wk) {
        const int tok = a.glu ? o >> 3 : o >> 4, rr = o & (per_tile - 1);
        const int n = per_tile * cur.rt + rr;
        if (n >= a.Nout) continue;
        float f = 0.f, up = 0.f;
        for (int j = 0; j < wk; ++j) {
          f += src[j * kXgRedWarp + tok * kXgRedStride + rr];
          if (a.glu) up += src[j * kXgRedWarp + tok * kXgRedStride + rr + 8];
        }
        if (bias) {
          f += Elt<T>::to_f32(bias[n]);
          if (a.glu) up += Elt<T>::to_f32(bias[a.Nout + n]);
        }
        f = apply_act(a.act, f);
        if (a.glu) f *= up;
        a.y[(int64_t)(first + tok) * a.Nout + n] = Elt<T>::from_f32(f);
      }
    }
    buf ^= 1;
    cur = nxt;
    if (kp >= nsl) {  // this warp has no slice: it only follows the tiles
      cur.u = u + ngrp;
      if (cur.u < uend) set_tile(cur);
    }
  }
  // The experts of the block's range that other groups still work on.
  if (books && !a.shared)
    while (book_e < a.E && tiles.start[book_e] < uend) leave_expert();
}

// Warps per tile: as many as give every warp of the device a share of the tiles of eight experts
// (a token's, say; or of all, where there are fewer), at most one per slice of K.  It goes by the
// layer and E alone, so that a row's sum is taken in the same order whatever the call's other rows.  At 8 rows for 8 experts, us: 2048 x 2048
// 20.7 with 2 warps, 21.5 with 4, 24.1 with 1 (no sums to exchange, but 14 % of the warps idle).
static int xg_wk(int E, int N, int K, int num_sms) {
  const int nsl = (K + 127) / 128, tiles = (E < 8 ? E : 8) * ((N + 15) / 16);
  int wk = 16;
  while (wk > 1 && (wk > nsl || (int64_t)wk * tiles > (int64_t)kXgWarps * num_sms)) wk /= 2;
  return wk;
}

template <int FMT, typename T>
static cudaError_t launch_xg_t(const ExpertsArgs& a, int num_sms, cudaStream_t s) {
  auto kern = experts_gemv_kernel<FMT, T>;
  constexpr XgSmem lay = xg_smem(FMT);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, lay.bytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(num_sms);
  cfg.blockDim = dim3(kXgThreads);
  cfg.dynamicSmemBytes = lay.bytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a, xg_wk(a.E, a.w.N, a.w.K, num_sms));
}

template <typename T>
static cudaError_t launch_xg(const ExpertsArgs& a, int num_sms, cudaStream_t s) {
  switch (a.w.fmt) {
    case kFmtRvq12: return launch_xg_t<kFmtRvq12, T>(a, num_sms, s);
    case kFmtRvq12_4: return launch_xg_t<kFmtRvq12_4, T>(a, num_sms, s);
    case kFmtVq16Rvq: return launch_xg_t<kFmtVq16Rvq, T>(a, num_sms, s);
    default: return launch_xg_t<kFmtVq16, T>(a, num_sms, s);
  }
}

cudaError_t launch_experts_gemv(const ExpertsArgs& a, int num_sms, cudaStream_t s) {
  return a.w.act == VQ_BF16 ? launch_xg<__nv_bfloat16>(a, num_sms, s) : launch_xg<__half>(a, num_sms, s);
}

}  // namespace vq
