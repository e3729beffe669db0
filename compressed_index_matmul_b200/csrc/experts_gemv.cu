// Products grouped by expert for few rows per expert (vq_experts_forward): y[r] =
// act(x[rows[r]] . W_e^T + b), decoded in registers and multiplied with warp MMAs.
//
// With a handful of rows per expert the decode of W is the work (2 N K / 8 codeword
// gathers per expert, whatever the row count), so the kernel is built around it:
//   tile    16 rows of W (glu: 8 gate rows and the 8 up rows that go with them) x up to 16
//           rows of x, over all of K; the tiles of all experts are numbered in expert order
//           (find_tiles) and cut into one contiguous, equal range per block
//   block   16 warps with 128 registers each, one block per SM (a 17th warp, for the copies, would
//           leave 96: 88 us for 64 experts x 4 rows of 2048 x 1024, against 70; 67 now).  The warps form
//           groups of wk; a group takes a tile at a time and its warps take the 128-input
//           slices of K in turn.  A warp walks (tile, slice) as one sequence and
//           loads the index bytes of its next slice before it decodes the current one, across
//           tiles and experts too, so the index loads are never waited for at a tile's end
//   lane    (g, c) = (lane / 4, lane % 4): rows g and g + 8 of the tile, groups 4 i + c of
//           the slice (i = 0 .. 3).  The decoded group is a fragment of mma m16n8k16's A
//           operand as it stands: MMA 2 i + h takes elements 4 h .. 4 h + 3, the same
//           permutation of k on both operands, so x comes as 16-byte loads, 64 contiguous bytes
//           per row
// The 12-bit codebooks (64 KiB an expert) live in shared memory in two slots, the next expert's
// copied while the current one is used: the last warp to leave an expert starts the copy into
// its slot.  The 16-bit codebooks are gathered through L2.
// The warps of a group meet once per tile, at a named barrier, and add their sums in warp order
// (two buffers, so one barrier suffices); the other groups go on meanwhile.  The result of a
// row does not depend on the other rows.
// Bound: the shared-memory pipe.  A gather of 32 codewords of 16 bytes takes about 10 wavefronts
// (random banks), the stage-2 codewords 4 shuffles, x and the indices the rest: 20 cycles of an SM for 256
// weights, 3.7 T weights a second on 148 SMs at 1.965 GHz.  Measured, the launch, the offsets and the
// codebooks included: 2.1 for 88 M weights (42 experts x 1 to 4 rows of 2048 x 1024, 41 us), 1.7 for
// 34 M (8 experts x 1 row of 2048 x 2048, 19.6 us), where the shared-memory pipe is 41 % busy: the
// chains of load, gather and MMA of 16 warps do not fill it.
#include <type_traits>

#include "experts.cuh"

namespace vq {

constexpr int kXgWarps = 16;                       // decode warps
constexpr int kXgThreads = 32 * kXgWarps;          // four warps per SM sub-partition: 128 registers each
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

// Entry `q` (32 bits: an expert has fewer than 2^31) of the planes of layer l, row n.
template <int FMT>
__device__ __forceinline__ void load_row(const LayerArgs& l, uint32_t q, int n, bool full, XgIdx<FMT>& r) {
  constexpr bool k16 = (FMT == kFmtVq16 || FMT == kFmtVq16Rvq);
  if constexpr (k16) {
    const uint4* src = reinterpret_cast<const uint4*>(l.idx16 + q);
    const uint4 a = __ldg(src);
    r.lo[0] = a.x; r.lo[1] = a.y; r.lo[2] = a.z; r.lo[3] = a.w;
    if (full) {
      const uint4 b = __ldg(src + 1);
      r.lo[4] = b.x; r.lo[5] = b.y; r.lo[6] = b.z; r.lo[7] = b.w;
    }
  } else if (full) {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(l.lo + q));
    const uint2 h = __ldg(reinterpret_cast<const uint2*>(l.hi4 + q / 2));
    r.lo[0] = a.x; r.lo[1] = a.y; r.lo[2] = a.z; r.lo[3] = a.w;
    r.hi[0] = h.x; r.hi[1] = h.y;
    if (FMT == kFmtRvq12_4) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(l.s2 + q / 2));
      r.s2[0] = v.x; r.s2[1] = v.y;
    }
  } else {
    const uint2 a = __ldg(reinterpret_cast<const uint2*>(l.lo + q));
    r.lo[0] = a.x; r.lo[1] = a.y;
    r.hi[0] = __ldg(reinterpret_cast<const uint32_t*>(l.hi4 + q / 2));
    if (FMT == kFmtRvq12_4) r.s2[0] = __ldg(reinterpret_cast<const uint32_t*>(l.s2 + q / 2));
  }
  if (l.scale_group == 64)  // one scale per 8 groups: 2 (or 1) per row and slice
    r.sc = full ? __ldg(reinterpret_cast<const uint32_t*>(l.scales + q / 8)) : (uint32_t)__ldg(l.scales + q / 8);
  else
    r.sc = __ldg(l.scales + n) * 0x10001u;
}

template <int FMT, typename T>
__global__ void __launch_bounds__(kXgThreads, 1) experts_gemv_kernel(const __grid_constant__ ExpertsArgs a, int wk) {
  extern __shared__ __align__(128) unsigned char smem[];
  constexpr bool k16 = (FMT == kFmtVq16 || FMT == kFmtVq16Rvq);
  constexpr bool kTwo = (FMT == kFmtRvq12_4);
  constexpr bool kLadder = (FMT == kFmtVq16Rvq);
  constexpr int kSlot = k16 ? kXgSlot8 : kXgSlot12;
  constexpr XgSmem lay = xg_smem(FMT);
  float* red = reinterpret_cast<float*>(smem + lay.red);
  ExpertTiles& tiles = *reinterpret_cast<ExpertTiles*>(smem + lay.tiles);
  const uint32_t bars = smem_u32(smem + lay.bars);
  auto full = [&](int i) { return bars + 8u * (i & 1); };            // the codebook of the sequence's i-th expert landed
  uint32_t* left = reinterpret_cast<uint32_t*>(smem + lay.bars + 16);  // [2] warps that have left a slot's expert
  volatile int* abortf = reinterpret_cast<volatile int*>(smem + lay.bars + 32);
  int* part = reinterpret_cast<int*>(smem + lay.bars + 64);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int N = a.w.N, K = a.w.K;
  if (tid == 0) {
    ptx::mbar_init(full(0), 1);
    ptx::mbar_init(full(1), 1);
    left[0] = left[1] = 0;
    *abortf = 0;
    ptx::fence_barrier_init();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int per_tile = a.glu ? 8 : 16;  // outputs of a tile
  find_tiles(a, kXgTok, (a.Nout + per_tile - 1) / per_tile, tiles, part, kXgThreads);
  const int total = tiles.start[a.E];
  const int ubeg = (int)((int64_t)total * blockIdx.x / gridDim.x), uend = (int)((int64_t)total * (blockIdx.x + 1) / gridDim.x);
  if (ubeg >= uend) return;

  // The experts of the block's range that have rows are its sequence; the i-th one's codebook
  // goes to slot i % 2.
  const bool books = FMT != kFmtVq16 && (!k16 || a.w.n8);
  auto next_busy = [&](int e) {  // the first expert from e on with tiles in the range, or E
    while (e < a.E && tiles.start[e] == tiles.start[e + 1]) ++e;
    return e < a.E && tiles.start[e] < uend ? e : a.E;
  };
  auto load_book = [&](int e, int i) {
    const uint32_t dst = smem_u32(smem) + kSlot * (i & 1);
    const int64_t at = a.shared ? 0 : e;
    if (k16) {
      ptx::mbar_arrive_expect_tx(full(i), kXgSlot8);
      ptx::bulk_load(dst, a.w.cb8 + at * 256 * 8, kXgSlot8, full(i));
    } else {
      ptx::mbar_arrive_expect_tx(full(i), 65536u + (kTwo ? 256u : 0u));
      ptx::bulk_load(dst, a.w.cb1 + at * 4096 * 8, 65536u, full(i));
      if (kTwo) ptx::bulk_load(dst + 65536u, a.w.cb2 + at * 16 * 8, 256u, full(i));
    }
  };
  const int e_first = expert_of(tiles, a.E, ubeg);
  if (books && tid == 0) {
    load_book(e_first, 0);
    const int e = a.shared ? a.E : next_busy(e_first + 1);
    if (e < a.E) load_book(e, 1);
  }

  const int g = lane >> 2, c = lane & 3;
  const int grp = warp / wk, kp = warp % wk, ngrp = kXgWarps / wk;
  const int nsl = (K + 127) / 128;
  const bool tail = (K & 127) != 0;             // the last slice has 8 groups
  const uint32_t csel = 0x4440u | (uint32_t)c;  // byte c, zero-extended
  const uint32_t c4 = 4u * c;

  // The warp's place in the sequence of its codebooks.
  int book_e = e_first, book_i = 0;
  bool book_ready = !books;
  // Past the bound (never on a healthy device) the sums are wrong and the error word is set.
  auto wait_book = [&]() {
    if (!*abortf && !ptx::mbar_wait(full(book_i), (book_i >> 1) & 1, a.err)) *abortf = 1;
    book_ready = true;
  };
  // Go on to the next expert of the sequence.  The last warp to leave one refills its slot.  A
  // slot must be full before a warp leaves it, or it would count for the slot's expert before.
  auto leave_expert = [&]() {
    if (!book_ready) wait_book();
    __syncwarp();
    uint32_t n = 0;
    if (lane == 0)
      asm volatile("atom.acq_rel.cta.shared::cta.add.u32 %0, [%1], 1;" : "=r"(n) : "r"(smem_u32(left + (book_i & 1))) : "memory");
    if (lane == 0 && n == kXgWarps - 1) {
      left[book_i & 1] = 0;  // before the copy, whose landing lets the next leave
      int e = next_busy(book_e + 1);
      if (e < a.E) e = next_busy(e + 1);
      if (e < a.E) {
        ptx::fence_proxy_async_smem();
        load_book(e, book_i + 2);
      }
    }
    book_e = next_busy(book_e + 1);
    ++book_i;
    book_ready = false;
  };

  // The load stream runs one slice ahead of the decode: tile lu of expert le, slice ls.
  int lu = ubeg + grp, le = e_first, ls = kp, lrt = 0, ltk = 0;  // kp < nsl: a group has at most nsl warps
  uint32_t lq = 0;         // entry of (slice ls, row 0)
  int rA = 0, rB = 0;      // the lane's two rows of W; past the last one they repeat it (not stored)
  LayerArgs lw = expert_layer(a, le);
  const uint32_t slice_step = 16u * (uint32_t)N;
  auto load_tile = [&]() {
    int e = le;
    while (e + 1 < a.E && lu >= tiles.start[e + 1]) ++e;
    if (e != le) {
      le = e;
      lw = expert_layer(a, e);
    }
    const int tt = (tiles.off[e + 1] - tiles.off[e] + kXgTok - 1) / kXgTok, local = lu - tiles.start[e];
    lrt = tt == 1 ? local : local / tt;
    ltk = tt == 1 ? 0 : local - lrt * tt;
    if (a.glu) {
      rA = min(8 * lrt + g, a.Nout - 1);
      rB = a.Nout + rA;
    } else {
      rA = min(16 * lrt + g, N - 1);
      rB = min(16 * lrt + g + 8, N - 1);
    }
    ls = kp;
    lq = slice_step * (uint32_t)kp;
  };
  auto load_slice = [&](XgIdx<FMT> (&q)[2]) {
    const bool whole = !tail || ls + 1 < nsl;
    const uint32_t w = whole ? 16u : 8u;
    load_row<FMT>(lw, lq + w * rA, rA, whole, q[0]);
    load_row<FMT>(lw, lq + w * rB, rB, whole, q[1]);
  };
  // The next slice of the stream; false at its end.
  auto advance = [&]() {
    ls += wk;
    lq += slice_step * (uint32_t)wk;
    if (ls >= nsl) {
      lu += ngrp;
      if (lu >= uend) return false;
      load_tile();
    }
    return true;
  };

  XgIdx<FMT> iq[2], nq[2];
  bool more = lu < uend;
  if (more) {
    load_tile();
    load_slice(iq);
  }
  int tok_e = -1, tok_tk = -1, nt = 1;
  const uint16_t* xp[2] = {a.x, a.x};
  uint32_t bad = 0;  // bit t: row t of the x tile is out of range and counts as zeros
  uint32_t cb2r[4] = {0, 0, 0, 0};
  const uint4* cbs = reinterpret_cast<const uint4*>(smem);
  int buf = 0;

  while (more) {
    const int e = le, rt = lrt, tk = ltk;  // the tile that is decoded now
    const int rowA = rA, rowB = rB;
    const LayerArgs l = lw;
    if (books) {
      while (!a.shared && book_e != e) leave_expert();
      if (!book_ready) {
        wait_book();
        cbs = reinterpret_cast<const uint4*>(smem + kSlot * (book_i & 1));
        if (kTwo) {
          const uint4 v = cbs[4096 + (lane & 15)];
          cb2r[0] = v.x; cb2r[1] = v.y; cb2r[2] = v.z; cb2r[3] = v.w;
        }
      }
    }
    if (tok_e != e || tok_tk != tk) {
      tok_e = e;
      tok_tk = tk;
      const int first = tiles.off[e] + kXgTok * tk, last = tiles.off[e + 1];
      nt = last - first > 8 ? 2 : 1;
      bad = 0;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        // places past the last row repeat it; a row out of range reads row 0 and is zeroed at the end
        const int r = min(first + 8 * t + g, last - 1);
        const int xr = a.rows ? a.rows[r] : r;
        const bool in = xr >= 0 && xr < a.x_rows;
        xp[t] = a.x + (int64_t)(in ? xr : 0) * K + 8 * c;
        const uint32_t m = __ballot_sync(0xffffffffu, !in);  // bit 4 g: row g
#pragma unroll
        for (int i = 0; i < 8; ++i) bad |= ((m >> (4 * i)) & 1u) << (8 * t + i);
      }
    }
    float acc[2][4];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[t][i] = 0.f;

    // One slice into acc; NT: x row tiles of 8.
    auto slice = [&](auto ntc, int s) {
      constexpr int NT = decltype(ntc)::value;
      const bool whole = !tail || s + 1 < nsl;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i == 2 && !whole) break;
        uint4 xq[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) xq[t] = *reinterpret_cast<const uint4*>(xp[t] + 128 * s + 32 * i);
        uint32_t wq[2][4];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const unsigned short sc = (unsigned short)(i < 2 ? iq[r].sc : iq[r].sc >> 16);
          uint32_t i1;
          [[maybe_unused]] uint32_t c2[4] = {0, 0, 0, 0};
          if constexpr (k16) {
            i1 = ((c & 2 ? iq[r].lo[2 * i + 1] : iq[r].lo[2 * i]) >> (16 * (c & 1))) & 0xFFFFu;
          } else {
            uint32_t b;
            asm("prmt.b32 %0, %1, 0, %2;" : "=r"(b) : "r"(iq[r].lo[i]), "r"(csel));
            i1 = b | (((iq[r].hi[i >> 1] >> (16 * (i & 1) + c4)) & 15u) << 8);
            if (kTwo) {
              const int i2 = (int)(iq[r].s2[i >> 1] >> (16 * (i & 1) + c4));  // the shuffle takes it modulo 16
#pragma unroll
              for (int v = 0; v < 4; ++v) c2[v] = __shfl_sync(0xffffffffu, cb2r[v], i2, 16);
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
            const int64_t NG = (int64_t)N * (K / 8);
            const int64_t ent = (int64_t)slice_step * s + (int64_t)(r ? rowB : rowA) * (whole ? 16 : 8) + 4 * i + c;
#pragma unroll
            for (int t = 2; t <= 4; ++t) {
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
        for (int t = 0; t < NT; ++t) {
          Mma16816<T>::run(acc[t], af0, xq[t].x, xq[t].y);
          Mma16816<T>::run(acc[t], af1, xq[t].z, xq[t].w);
        }
      }
    };
    for (int s = kp; s < nsl; s += wk) {
      more = advance();
      if (more) load_slice(nq);
      if (nt == 1)
        slice(std::integral_constant<int, 1>{}, s);
      else
        slice(std::integral_constant<int, 2>{}, s);
      iq[0] = nq[0];
      iq[1] = nq[1];
    }

    if (bad) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if ((bad >> (8 * t + 2 * c + (i & 1))) & 1u) acc[t][i] = 0.f;
    }
    const int first = tiles.off[e] + kXgTok * tk, have = min(tiles.off[e + 1] - first, kXgTok);
    const uint16_t* bias = a.bias ? a.bias + (int64_t)e * N : nullptr;
    uint16_t* y = a.y + (int64_t)first * a.Nout;
    if (wk == 1) {
      // The whole sum is in this warp: lane (g, c) has rows g and g + 8 (glu: a gate and its up
      // row) of tokens 2 c and 2 c + 1.
      const int n0 = per_tile * rt + g;
      const float b0 = bias ? Elt<T>::to_f32(bias[rowA]) : 0.f, b1 = bias ? Elt<T>::to_f32(bias[rowB]) : 0.f;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (t >= nt) break;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int tok = 8 * t + 2 * c + h;
          if (tok >= have) continue;
          const float f0 = acc[t][h] + b0, f1 = acc[t][2 + h] + b1;
          uint16_t* yt = y + (int64_t)tok * a.Nout + n0;
          if (a.glu) {
            if (n0 < a.Nout) yt[0] = Elt<T>::from_f32(gated(a.act, f0, f1));
          } else {
            if (n0 < N) yt[0] = Elt<T>::from_f32(apply_act(a.act, f0));
            if (n0 + 8 < N) yt[8] = Elt<T>::from_f32(apply_act(a.act, f1));
          }
        }
      }
      continue;
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
    const float* src = red + (buf * kXgWarps + grp * wk) * kXgRedWarp;
    for (int o = 32 * kp + lane; o < per_tile * have; o += 32 * wk) {
      const int tok = a.glu ? o >> 3 : o >> 4, rr = o & (per_tile - 1);
      const int n = per_tile * rt + rr;
      if (n >= a.Nout) continue;
      float f = 0.f, up = 0.f;
      for (int j = 0; j < wk; ++j) f += src[j * kXgRedWarp + tok * kXgRedStride + rr];
      if (bias) f += Elt<T>::to_f32(bias[n]);
      f = apply_act(a.act, f);
      if (a.glu) {
        for (int j = 0; j < wk; ++j) up += src[j * kXgRedWarp + tok * kXgRedStride + rr + 8];
        if (bias) up += Elt<T>::to_f32(bias[a.Nout + n]);
        f *= up;
      }
      y[(int64_t)tok * a.Nout + n] = Elt<T>::from_f32(f);
    }
    buf ^= 1;
  }
  // The experts of the block's range that other groups still work on.
  if (books && !a.shared)
    while (book_e < a.E) leave_expert();
}

// Warps per tile: as many as give every warp of the device a share of the tiles of eight experts
// (a token's, say; or of all, where there are fewer), at most one per slice of K.  It goes by the
// layer and E alone, so that a row's sum is taken in the same order whatever the call's other rows.
// At 8 rows for 8 experts of 2048 x 2048, us: 20.7 with 2 warps, 21.5 with 4, 24.1 with 1 (no sums to
// exchange, but 14 % of the warps idle).
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
