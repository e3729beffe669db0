// Products grouped by expert for many rows per expert (vq_experts_forward): y[r] =
// act(x[rows[r]] . W_e^T + b) on the tensor cores, W decoded into tensor memory.
//
// A persistent pair of blocks (a cluster of two, one per SM) walks tiles of 256 rows of W (glu:
// 128 gate rows and the 128 up rows that go with them) x up to Tmax rows of x, over all of K.
// Each block decodes half of the tile's rows of W and holds half of its x rows in shared memory;
// tcgen05.mma.cta_group::2 multiplies both, so an SM reads half of the x that a tile of its
// own would need (with tiles per block the x loads, 32 KiB per 64 inputs and SM, ran at the
// L2's 7 TB/s and set the pace).  The tiles of all experts are numbered in expert order
// (find_tiles) and cut into one contiguous range of equal cost per pair, so a pair changes its
// expert, and with it the codebook in shared memory, once or twice.
//   warp 0     lane 0: x, per 128-input slice, a TMA load per 64 inputs of the block's half of the
//              tile's x rows (a box of 32, 64 or 128 rows, 128-byte swizzle: one large load
//              instead of several small ones) into a ring of four stages.  Both blocks' loads
//              complete on the first block's barrier, where the MMAs are issued
//   warp 1     allocates TMEM; in the first block an elected lane issues tcgen05.mma (M = 256, N =
//              the tile's rows rounded up to 16, K = 16), A from both blocks' TMEM, B from both
//              blocks' shared memory, and commits each stage to both
//   warp 2     the expert's 12-bit codebook (one bulk copy when it changes) and, per
//              128-input slice, the index bytes of the block's rows (one contiguous run per
//              plane; glu: two; a lane each) into a ring of four slots
//   warps 4..  decode: four per TMEM lane quarter; thread = one row of W (its lane).
//              Slice `js` of the pair's whole sequence goes to warp js % 4 of every quarter, into A
//              stage js % 4 (64 TMEM columns, 128 inputs).  After a tile's last slice the same
//              threads read the accumulator, apply bias and activation and store y: consecutive
//              lanes are consecutive columns, and rows past the expert's last are not written.
// All rings run on across tiles: while the decode warps store one tile, x and the indices
// of the next are already on their way.  With Tmax <= 128 the accumulator has two buffers, so
// the MMAs of the next tile need not wait for the stores either.
// Rows that come through `rows` are first copied into row order (gather_rows_kernel): T K
// elements written and read once more, 15 us of a 16384 x 2048 gather.  Gathering them in the x
// loads instead (TMA tile::gather4) took 40 ns per four rows, 2.6 us a k block of 256 rows,
// several times what its decode takes.
// Every mbarrier wait is bounded; a timeout sets the handle's error word, and the block winds
// down (waits for its own copies and MMAs, frees TMEM).
#include <cuda.h>

#include <type_traits>

#include "experts.cuh"

namespace vq {

constexpr int kXtRows = 128;
constexpr int kXtParts = 4;                            // decode warps per TMEM lane quarter, and A stages
constexpr int kXtDecode = 4 * kXtParts;                // decode warps
constexpr int kXtThreads = 32 * (4 + kXtDecode);
constexpr int kXtStages = 4;                           // x stages of a slice (128 inputs)
constexpr int kXtMaxT = 256;
constexpr int kXtSlots = kXtParts;                     // index slices in flight
constexpr uint32_t kXtACols = 64;                      // TMEM columns of one A stage (128 k of 16-bit pairs)
constexpr uint32_t kXtIdxHi = 16 * kXtRows, kXtIdxS2 = 24 * kXtRows, kXtIdxSc = 32 * kXtRows, kXtIdxSlot = 36 * kXtRows;  // bytes
constexpr uint32_t kXtOffTiles = 65536;                // after the codebook
constexpr uint32_t kXtOffBars = kXtOffTiles + (sizeof(ExpertTiles) + 15) / 16 * 16;
constexpr uint32_t kXtOffIdx = kXtOffBars + 768;
constexpr uint32_t kXtOffX = (kXtOffIdx + kXtSlots * kXtIdxSlot + 1023) / 1024 * 1024;
// Tmax is 128 or 256 (twice the heights of the larger boxes).
constexpr uint32_t xt_smem(int Tmax) { return kXtOffX + kXtStages * (Tmax / 2) * 256u + 1024u; }
static_assert(xt_smem(kXtMaxT) <= 232448, "shared memory of the widest tile");
// A pair takes all 512 TMEM columns of both SMs, and two pairs that each hold one SM's and wait for
// the other's would never go on, nor a pair and a tc_gemm_kernel block: no two of them fit an SM's
// 228 KiB (tc_gemm_kernel takes 92 KiB and more).
static_assert(xt_smem(kXtMaxT / 2) >= 147456, "no other block that allocates TMEM may share the SM");

constexpr int kXtBoxes = 3;        // x rows of one TMA load: 32, 64 or 128
constexpr int kXtTileCost = 600;   // cost of a tile's decode, in x rows (13.6 us + 23 ns a row at K = 2048)

struct XtMaps {
  CUtensorMap x[kXtBoxes];
};

// xs[r] = x[rows[r]], zeros where the row is out of range.  One block per row.
__global__ void __launch_bounds__(128) gather_rows_kernel(const uint4* __restrict__ x, const int32_t* __restrict__ rows,
                                                          uint4* __restrict__ xs, int K8, int x_rows) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t r = blockIdx.x;
  const int xr = rows[r];
  const bool in = xr >= 0 && xr < x_rows;
  for (int i = threadIdx.x; i < K8; i += 128) xs[r * K8 + i] = in ? x[(int64_t)xr * K8 + i] : make_uint4(0, 0, 0, 0);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Arrive on a barrier of block `rank` of the pair.  What the arrivals tell of is in TMEM (decoded
// weights stored, sums read), ordered by the tcgen05 fences on both sides, so the cheap default scope
// serves (a release at cluster scope held each decode warp up for more than 1000 cycles).
__device__ __forceinline__ void arrive_at(uint32_t bar, uint32_t rank) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(ptx::map_shared_rank(bar, rank)) : "memory");
}
// A 2-D tensor load into this block's shared memory that completes on `bar`, a barrier of either block
// of the pair (an address from map_shared_rank): the thread that waits there sees the bytes
// of both blocks landed, with nothing in between to pass their arrival on.
__device__ __forceinline__ void pair_tma_load_2d(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
      "%3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}
// The pair's TMEM and MMA (cta_group::2; both blocks allocate and free).
__device__ __forceinline__ void pair_tmem_alloc(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void pair_umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrive once on `bar` of both blocks when every MMA this thread issued before has completed.
__device__ __forceinline__ void pair_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
               "h"((unsigned short)3)
               : "memory");
}

// One tile: its expert, its place, its x rows.
struct XtTile {
  int e, rt, first, n, T;  // first row of y, rows (<= Tmax), n rounded up to 16
};

template <int FMT, typename T, bool kStaged>
__global__ void __launch_bounds__(kXtThreads, 1)
    experts_tc_kernel(const __grid_constant__ XtMaps maps, const __grid_constant__ ExpertsArgs a, int Tmax,
                      int nacc) {
  extern __shared__ unsigned char smem_raw[];
  constexpr bool k16 = (FMT == kFmtVq16 || FMT == kFmtVq16Rvq);
  constexpr bool kLadder = (FMT == kFmtVq16Rvq);
  constexpr bool kBook = !k16;
  constexpr bool kTwo = (FMT == kFmtRvq12_4);
  static_assert(!(kLadder && kStaged), "the residual ladder reads its indices directly");
  constexpr int kSt = kXtStages;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;  // the swizzle of the x tiles goes by address bits
  unsigned char* sm = smem_raw + (base - raw);
  const uint4* cb1s = reinterpret_cast<const uint4*>(sm);
  ExpertTiles& tiles = *reinterpret_cast<ExpertTiles*>(sm + kXtOffTiles);
  const uint32_t bar0 = base + kXtOffBars;
  auto full_b = [&](int s) { return bar0 + 8u * s; };
  auto acc_full = [&](int b) { return bar0 + 8u * (2 * kSt + b); };
  auto acc_empty = [&](int b) { return bar0 + 8u * (2 * kSt + 2 + b); };
  const uint32_t cb_full = bar0 + 8u * (2 * kSt + 4), cb_empty = cb_full + 8u, bar1 = cb_full + 16u;
  auto full_a = [&](int s) { return bar1 + 8u * s; };
  auto empty_a = [&](int s) { return bar1 + 8u * (kXtParts + s); };
  auto idx_full = [&](int s) { return bar1 + 8u * (2 * kXtParts + s); };
  auto idx_empty = [&](int s) { return bar1 + 8u * (3 * kXtParts + s); };
  static_assert(8 * (2 * kSt + 6 + 4 * kXtParts) <= 384, "barriers overlap the flags");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + kXtOffBars + 384);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + kXtOffBars + 388);
  int* part_sums = reinterpret_cast<int*>(sm + kXtOffBars + 392);  // 2 per warp
  static_assert(392 + 8 * kXtThreads / 32 <= 768, "scan area");
  const uint32_t b_bytes = (uint32_t)(Tmax / 2) * 128u;  // 64 inputs of the block's half of the tile's rows
  auto b_tile = [&](int s, int h) { return base + kXtOffX + b_bytes * (2 * s + h); };

  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int N = a.w.N, K = a.w.K, G = K / 8;
  const int nsl = (K + 127) / 128;
  const int out_tile = a.glu ? kXtRows / 2 : kXtRows;  // columns of y of the block's half of a tile
  const uint32_t rank = __shfl_sync(0xffffffffu, cluster_rank(), 0);
  const int RT = (a.Nout + 2 * out_tile - 1) / (2 * out_tile);  // row tiles of the pair
  const uint32_t acols = (uint32_t)Tmax;
  const uint32_t acol0 = acols * nacc;  // then the A stages
  const uint32_t tcols = 512u;  // acol0 + kXtParts * kXtACols is above 256

  if (tid == 0) {
    for (int s = 0; s < kSt; ++s)
      ptx::mbar_init(full_b(s), 1);  // the first block's expect_tx arrival (+ both blocks' bytes; first block only)
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(acc_full(b), 1);
      ptx::mbar_init(acc_empty(b), 2 * kXtDecode);  // both blocks' decode warps (first block only)
    }
    ptx::mbar_init(cb_full, 1);
    ptx::mbar_init(cb_empty, kXtDecode);
    for (int s = 0; s < kXtParts; ++s) {
      ptx::mbar_init(full_a(s), 8);     // one decode warp per TMEM lane quarter, both blocks (first block only)
      ptx::mbar_init(empty_a(s), 1);    // one tcgen05.commit
      ptx::mbar_init(idx_full(s), 1);
      ptx::mbar_init(idx_empty(s), 4);  // the warps that decode the slice
    }
    *abort_flag = 0;
    ptx::fence_barrier_init();
  }
  if (warp == 1) {
    pair_tmem_alloc(smem_u32(tmem_slot), tcols);
  }
  ptx::tc_fence_before();
  __syncwarp();
  ptx::cluster_sync();  // the barriers of both blocks are initialised
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  find_tiles(a, Tmax, RT, tiles, part_sums, kXtThreads);
  // Rows of each of expert e's tiles: even, a multiple of 16.
  auto tile_rows = [&](int e) {
    const int n = tiles.off[e + 1] - tiles.off[e], tt = (n + Tmax - 1) / Tmax;
    return tt == 0 ? 0 : ((n + tt - 1) / tt + 15) & ~15;
  };
  // The block's tiles.  Expert e's tiles cost kXtTileCost + their rows each; the tile at which a share
  // of the whole cost is reached ends one block's range and starts the next one's.
  float* cost = reinterpret_cast<float*>(sm + kXtOffX);  // [E + 1], in the x area before its first use
  if (warp == 0) {
    float run = 0.f;
    for (int e0 = 0; e0 < a.E; e0 += 32) {
      const int e = e0 + lane;
      const float c = e < a.E ? (float)(tiles.start[e + 1] - tiles.start[e]) * (float)(kXtTileCost + tile_rows(e)) : 0.f;
      float sum = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += v;
      }
      if (e < a.E) cost[e] = run + sum - c;
      run += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (lane == 0) cost[a.E] = run;
    __syncwarp();
    if (lane < 2) {
      const int b = (int)(blockIdx.x / 2) + lane, pairs = (int)(gridDim.x / 2);
      int u = b == 0 ? 0 : tiles.start[a.E];
      if (b > 0 && b < pairs) {
        const float c = run * ((float)b / (float)pairs);
        int lo = 0, hi = a.E;
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (cost[mid] <= c) lo = mid; else hi = mid;
        }
        const int k = (int)((c - cost[lo]) / (float)(kXtTileCost + tile_rows(lo)));
        u = tiles.start[lo] + max(0, min(k, tiles.start[lo + 1] - tiles.start[lo]));
      }
      part_sums[lane] = u;
    }
    ptx::fence_proxy_async_smem();  // TMA writes the x area next
  }
  __syncthreads();
  const int ubeg = part_sums[0], uend = part_sums[1];

  // Tile u; `e` walks along (it starts at the range's first expert).
  int e_walk = ubeg < uend ? expert_of(tiles, a.E, ubeg) : 0;
  auto tile_of = [&](int u) {
    while (e_walk + 1 < a.E && u >= tiles.start[e_walk + 1]) ++e_walk;
    XtTile t;
    t.e = e_walk;
    const int beg = tiles.off[e_walk], n = tiles.off[e_walk + 1] - beg, tt = (n + Tmax - 1) / Tmax;
    const int local = u - tiles.start[e_walk];
    const int rp = local / tt, tk = local - rp * tt;
    t.rt = 2 * rp + (int)rank;
    const int rows = tile_rows(e_walk);
    t.first = beg + tk * rows;
    t.n = min(rows, n - tk * rows);
    t.T = (t.n + 15) & ~15;
    return t;
  };

  if (warp == 0) {
    // ------------------------------------------------------------ x rows
    if (lane == 0) {
      int js = 0;
      bool ok = true;
      for (int u = ubeg; ok && u < uend; ++u) {
        const XtTile t = tile_of(u);
        const int half = t.T / 2, first = t.first + (int)rank * half;
        const int box = half <= 32 ? 32 : half <= 64 ? 64 : 128;  // rows past the half are loaded and not used
        const CUtensorMap* map = &maps.x[box >> 6];
        for (int j = 0; j < nsl; ++j, ++js) {
          const int s = js % kSt, before = js - kSt;  // the slice that the stage held
          if (before >= 0 && !ptx::mbar_wait(empty_a(before % kXtParts), (before / kXtParts) & 1, a.err)) {
            *abort_flag = 1;
            ok = false;
            break;
          }
          // The second block's bytes may land before the first block expects them: the phase cannot
          // end without its arrival, and the next one's loads wait for the MMAs of this one.
          const int blocks = slice_width(j, G) / 8;
          if (rank == 0) ptx::mbar_arrive_expect_tx(full_b(s), (uint32_t)(2 * blocks * box) * 128u);
          const uint32_t bar = ptx::map_shared_rank(full_b(s), 0);
          for (int h = 0; h < blocks; ++h) pair_tma_load_2d(b_tile(s, h), map, 128 * j + 64 * h, first, bar);
        }
      }
      // Do not leave while a copy into this block's shared memory may be in flight: the MMAs of the
      // last slices come after both blocks' copies (and if they never come, the copies have had the
      // waits' second).
      for (int i = js > kSt ? js - kSt : 0; i < js; ++i)
        ptx::mbar_wait(empty_a(i % kXtParts), (i / kXtParts) & 1, a.err);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (the first block's)
    // The whole warp walks the tiles and waits, and one elected lane issues: with warp-uniform
    // control flow the descriptors are in uniform registers, as tcgen05.mma takes them.  Issued
    // from a loop of one lane, an MMA took 80 to 120 cycles and set the kernel's pace.
    constexpr uint32_t kAbFmt = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
    const uint32_t utmem = __shfl_sync(0xffffffffu, tmem, 0);
    bool ok = true;
    int js = 0, ui = 0;
    for (int u = ubeg; rank == 0 && ok && u < uend; ++u, ++ui) {
      const XtTile t = tile_of(u);
      const uint32_t idesc = __shfl_sync(0xffffffffu, ptx::idesc_f16(kAbFmt, 2 * kXtRows, (uint32_t)t.T), 0);
      const int b = ui % nacc;
      const uint32_t acc = utmem + acols * b;
      for (int j = 0; j < nsl; ++j, ++js) {
        const int st = js % kXtParts, s = js % kSt;
        // One poll for all that the slice waits for, a barrier a lane: the decode's gathers keep the
        // shared-memory pipe's queue long, and every poll goes through it (250 to 500 cycles).
        uint32_t bar = full_a(st), par = (uint32_t)(js / kXtParts) & 1u;
        bool wait = lane == 0;
        if (lane == 1) {
          bar = full_b(s);
          par = (uint32_t)(js / kSt) & 1u;
          wait = true;
        }
        if (lane == 2 && j == 0 && ui >= nacc) {  // the decode warps have read the accumulator's last tile
          bar = acc_empty(b);
          par = (uint32_t)((ui / nacc) - 1) & 1u;
          wait = true;
        }
        if (!ptx::mbar_wait_lanes(bar, par, wait, abort_flag, a.err)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        const uint32_t at = utmem + acol0 + kXtACols * st;
        const uint64_t b0 = ptx::smem_desc_sw128(b_tile(s, 0)), b1 = ptx::smem_desc_sw128(b_tile(s, 1));
        const bool two = slice_width(j, G) == 16;
        if (ptx::elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)  // A: +8 TMEM columns; B: +32 bytes along K inside the swizzle atom
            pair_umma_ts(acc, at + 8u * kk, b0 + 2u * kk, idesc, (j | kk) != 0);
          if (two) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) pair_umma_ts(acc, at + 32u + 8u * kk, b1 + 2u * kk, idesc, 1u);
          }
          pair_commit(empty_a(st));  // frees the slice's A and x stages
          if (j + 1 == nsl) pair_commit(acc_full(b));
        }
        __syncwarp();
      }
    }
    if (!ok) *abort_flag = 1;
    // The last commit covers every MMA before it: wait for it, so that neither block, which this warp
    // joins at the barrier below, releases TMEM or shared memory under one (on a whole run the decode
    // warps have waited already).
    if (js) ptx::mbar_wait(empty_a((js - 1) % kXtParts), ((js - 1) / kXtParts) & 1, a.err);
  } else if (warp == 2) {
    // ------------------------------------------------------------ codebooks and index slices
    // Lane 4 h + p copies plane p (lo or idx16, hi4, s2, scales) of run h of the tile's rows (glu: the
    // gate rows and the up rows, 64 rows apart in the slot; else one run).  One lane issuing all
    // the copies of a slice was slower than the decode.
    if (kBook || kStaged || kLadder) {
      const bool block_scales = a.w.scale_group == 64;
      const int run = lane >> 2, plane = lane & 3;
      const bool mine = kStaged && run < (a.glu ? 2 : 1) &&
                        (plane == 0 || (plane == 1 && !k16) || (plane == 2 && kTwo) || (plane == 3 && block_scales));
      // bytes of a row and slice of 16 groups
      const int row16 = plane == 0 ? (k16 ? 32 : 16) : plane == 3 ? 4 : 8;
      const uint32_t off = plane == 0 ? 0u : plane == 1 ? kXtIdxHi : plane == 2 ? kXtIdxS2 : kXtIdxSc;
      const uint32_t all16 = (k16 ? 32u : 24u + (kTwo ? 8u : 0u)) + (block_scales ? 4u : 0u);  // of all planes
      bool ok = true;
      int js = 0, books = 0, last_e = -1;
      for (int u = ubeg; ok && u < uend; ++u) {
        const XtTile t = tile_of(u);
        const LayerArgs l = expert_layer(a, t.e);
        if ((kBook || (kLadder && a.w.n8)) && (books == 0 || (!a.shared && t.e != last_e))) {
          if (books > 0 && !ptx::mbar_wait(cb_empty, (books - 1) & 1, a.err)) {
            ok = false;
            break;
          }
          if (lane == 0) {
            const uint32_t bytes = kBook ? 65536u : 4096u;
            ptx::mbar_arrive_expect_tx(cb_full, bytes);
            ptx::bulk_load(base, kBook ? l.cb1 : l.cb8, bytes, cb_full);
          }
          __syncwarp();
          ++books;
        }
        last_e = t.e;
        if (!kStaged) continue;
        const int r0 = out_tile * t.rt, nr = max(0, min(out_tile, a.Nout - r0)), runs = a.glu ? 2 : 1;
        const unsigned char* src = plane == 0   ? (k16 ? reinterpret_cast<const unsigned char*>(l.idx16) : l.lo)
                                   : plane == 1 ? l.hi4
                                   : plane == 2 ? l.s2
                                                : reinterpret_cast<const unsigned char*>(l.scales);
        const int64_t row = r0 + (int64_t)run * a.Nout;
        for (int j = 0; j < nsl; ++j, ++js) {
          const int sl = js % kXtSlots;
          if (js >= kXtSlots && !ptx::mbar_wait(idx_empty(sl), ((js / kXtSlots) - 1) & 1, a.err)) {
            ok = false;
            break;
          }
          const int w = slice_width(j, G);
          const uint32_t bar = idx_full(sl);
          if (lane == 0) ptx::mbar_arrive_expect_tx(bar, (uint32_t)(runs * nr) * all16 * (uint32_t)w / 16u);
          __syncwarp();
          if (mine && nr > 0) {
            const int bytes = row16 * w / 16;  // of a row
            ptx::bulk_load(base + kXtOffIdx + kXtIdxSlot * sl + off + (uint32_t)(64 * run * bytes),
                           src + (int64_t)row16 * j * N + row * bytes, (uint32_t)(nr * bytes), bar);
          }
        }
      }
      if (!ok) *abort_flag = 1;
      for (int i = js > kXtSlots ? js - kXtSlots : 0; i < js; ++i)
        ptx::mbar_wait(idx_full(i % kXtSlots), (i / kXtSlots) & 1, a.err);
      if (books) ptx::mbar_wait(cb_full, (books - 1) & 1, a.err);
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ decode
    const int q = warp & 3, part = (warp - 4) >> 2;
    const bool block_scales = a.w.scale_group == 64;
    // Row of the tile in the index slot, and of the output: with glu lanes 0..15 of a quarter hold
    // gate rows and lanes 16..31 the up rows of the same columns.
    const int col = a.glu ? 16 * q + (lane & 15) : 32 * q + lane;  // column of y within the tile
    const bool is_up = a.glu && lane >= 16;
    const int srow = is_up ? 64 + col : col;
    const uint32_t tlane = tmem + ((uint32_t)(32 * q) << 16);
    bool ok = true;
    int js0 = 0, ui = 0, books = 0, last_e = -1;
    uint32_t cb2r[4] = {0, 0, 0, 0};
    XtTile prev{};         // the tile before, whose sums this warp has not stored yet
    bool pending = false;

    // Bias, activation and stores of tile `t`, the block's ui-th.  A warp does it after its first
    // block of the next tile, so that the tensor cores finish the tile's last blocks meanwhile and
    // find the next tile's first ones decoded.
    auto finish_tile = [&](const XtTile& t, int ui) {
      const int n = out_tile * t.rt + col;
      const bool valid = n < a.Nout;
      const int r = is_up ? a.Nout + n : n;
      const int b = ui % nacc;
      if (!ptx::mbar_wait(acc_full(b), (ui / nacc) & 1, a.err)) return false;
      ptx::tc_fence_after();
      const float bv = (a.bias && valid) ? Elt<T>::to_f32(a.bias[(int64_t)t.e * N + r]) : 0.f;
      for (int c0 = 16 * part; c0 < t.n; c0 += 16 * kXtParts) {
        uint32_t v[16];
        ptx::tmem_ld16(tlane + acols * b + c0, v);
        ptx::tmem_wait_ld();
        const int left = t.n - c0;
        float f[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] = __uint_as_float(v[i]) + bv;
        uint16_t* y = a.y + (int64_t)(t.first + c0) * a.Nout + n;
        if (!a.glu) {
          apply_act_all(a.act, f);
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (valid && i < left) y[(int64_t)i * a.Nout] = Elt<T>::from_f32(f[i]);
        } else {
          // gate lanes finish the even token of each pair, up lanes the odd one
          float gate[8], up[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float other = __shfl_xor_sync(0xffffffffu, is_up ? f[2 * i] : f[2 * i + 1], 16);
            gate[i] = is_up ? other : f[2 * i];
            up[i] = is_up ? f[2 * i + 1] : other;
          }
          apply_act_all(a.act, gate);
          if (is_up) y += a.Nout;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (valid && 2 * i + (is_up ? 1 : 0) < left) y[(int64_t)(2 * i) * a.Nout] = Elt<T>::from_f32(gate[i] * up[i]);
        }
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_at(acc_empty(b), 0);
      return true;
    };
    for (int u = ubeg; ok && u < uend; ++u, ++ui) {
      const XtTile t = tile_of(u);
      const LayerArgs l = expert_layer(a, t.e);
      const int n = out_tile * t.rt + col;  // column of y
      const bool valid = n < a.Nout;
      const int r = is_up ? a.Nout + n : n;  // row of W
      if (books == 0 || (!a.shared && t.e != last_e)) {
        if (kTwo) {
          const uint4 v = reinterpret_cast<const uint4*>(l.cb2)[lane & 15];
          cb2r[0] = v.x; cb2r[1] = v.y; cb2r[2] = v.z; cb2r[3] = v.w;
        }
        if (kBook || (kLadder && a.w.n8)) {
          if (books > 0) {  // done with the codebook before
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(cb_empty);
          }
          if (!ptx::mbar_wait(cb_full, books & 1, a.err)) ok = false;
        }
        ++books;
      }
      last_e = t.e;
      const unsigned short row_scale = (!block_scales && valid) ? l.scales[r] : (unsigned short)0;
      // this warp's slices of the tile: those with (js0 + j) % P == part, all into its own A stage
      const uint32_t ta = tlane + acol0 + kXtACols * (uint32_t)part;
      for (int j = (part + kXtParts - js0 % kXtParts) % kXtParts; ok && j < nsl; j += kXtParts) {
        const int w = slice_width(j, G), round = (js0 + j) / kXtParts;
        if (kStaged && !ptx::mbar_wait(idx_full(part), round & 1, a.err)) {
          ok = false;
          break;
        }
        uint32_t lo[k16 ? 8 : 4], hi[2] = {0, 0}, s2[2] = {0, 0}, sc2 = row_scale * 0x10001u;
#pragma unroll
        for (int i = 0; i < (k16 ? 8 : 4); ++i) lo[i] = 0;
        if (valid) {
          if (kStaged) {
            const unsigned char* slot = sm + kXtOffIdx + kXtIdxSlot * part;
            if (w == 16) {
              const uint4 v = *reinterpret_cast<const uint4*>(slot + srow * (k16 ? 32 : 16));
              lo[0] = v.x; lo[1] = v.y; lo[2] = v.z; lo[3] = v.w;
              if constexpr (k16) {
                const uint4 v2 = *reinterpret_cast<const uint4*>(slot + srow * 32 + 16);
                lo[4] = v2.x; lo[5] = v2.y; lo[6] = v2.z; lo[7] = v2.w;
              } else {
                const uint2 h = *reinterpret_cast<const uint2*>(slot + kXtIdxHi + srow * 8);
                hi[0] = h.x; hi[1] = h.y;
                if (kTwo) {
                  const uint2 q2 = *reinterpret_cast<const uint2*>(slot + kXtIdxS2 + srow * 8);
                  s2[0] = q2.x; s2[1] = q2.y;
                }
              }
              if (block_scales) sc2 = *reinterpret_cast<const uint32_t*>(slot + kXtIdxSc + srow * 4);
            } else {  // a 64-wide last slice
              if constexpr (k16) {
                const uint4 v = *reinterpret_cast<const uint4*>(slot + srow * 16);
                lo[0] = v.x; lo[1] = v.y; lo[2] = v.z; lo[3] = v.w;
              } else {
                const uint2 v = *reinterpret_cast<const uint2*>(slot + srow * 8);
                lo[0] = v.x; lo[1] = v.y;
                hi[0] = *reinterpret_cast<const uint32_t*>(slot + kXtIdxHi + srow * 4);
                if (kTwo) s2[0] = *reinterpret_cast<const uint32_t*>(slot + kXtIdxS2 + srow * 4);
              }
              if (block_scales) sc2 = *reinterpret_cast<const uint16_t*>(slot + kXtIdxSc + srow * 2);
            }
          } else if constexpr (k16) {
            const int64_t e = (int64_t)16 * j * N + (int64_t)r * w;
            const uint4 v = *reinterpret_cast<const uint4*>(l.idx16 + e);
            lo[0] = v.x; lo[1] = v.y; lo[2] = v.z; lo[3] = v.w;
            if (w == 16) {
              const uint4 v2 = *reinterpret_cast<const uint4*>(l.idx16 + e + 8);
              lo[4] = v2.x; lo[5] = v2.y; lo[6] = v2.z; lo[7] = v2.w;
            }
            if (block_scales)
              sc2 = w == 16 ? *reinterpret_cast<const uint32_t*>(l.scales + e / 8) : (uint32_t)l.scales[e / 8];
          }
        }
        if (kStaged) {
          // The slot is free once every lane's bytes are in its registers.  Which lane says so depends
          // on the bytes, so the arrival comes after them whatever order the loads complete in: with
          // lane 0 arriving after a __syncwarp, the scales of 16-bit layers were at times those of four
          // slices later (why that order did not hold was not established).
          uint32_t seen = sc2;
#pragma unroll
          for (int i = 0; i < (k16 ? 8 : 4); ++i) seen ^= lo[i];
          if (!k16) seen ^= hi[0] ^ hi[1] ^ s2[0] ^ s2[1];
          if (lane == (int)(__reduce_or_sync(0xffffffffu, seen) & 31u)) ptx::mbar_arrive(idx_empty(part));
        }
        bool waited = round == 0;  // the MMAs of this stage's slice before are done
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // blocks of 64 inputs
          if (h == 1 && w == 8) break;
          // All eight gathers of a block are issued before the first is used.
          uint4 c1[8];
#pragma unroll
          for (int g = 0; g < 8; ++g) {
            uint32_t i1;
            if constexpr (k16)
              i1 = (lo[4 * h + (g >> 1)] >> (16 * (g & 1))) & 0xFFFFu;
            else
              i1 = ((lo[2 * h + (g >> 2)] >> (8 * (g & 3))) & 0xFFu) | (((hi[h] >> (4 * g)) & 15u) << 8);
            c1[g] = kBook ? cb1s[i1] : __ldg(reinterpret_cast<const uint4*>(l.cb1) + i1);
          }
          LadderIdx res{};
          if constexpr (kLadder)
            if (valid) load_ladder_block(l, (int64_t)16 * j * N + (int64_t)r * w + 8 * h, res);
          const unsigned short sc = (unsigned short)(h ? sc2 >> 16 : sc2);
          const float scf = kLadder ? __half2float(__ushort_as_half(sc)) : 0.f;
          if (!waited) {
            waited = true;
            if (!ptx::mbar_wait(empty_a(part), (round - 1) & 1, a.err)) ok = false;
            ptx::tc_fence_after();
          }
#pragma unroll
          for (int c = 0; c < 2; ++c) {  // 4 groups (16 TMEM columns) at a time
            uint32_t out[16];
#pragma unroll
            for (int g4 = 0; g4 < 4; ++g4) {
              const int g = 4 * c + g4;
              if constexpr (kLadder) {
                float v[8];
                ladder_sum(l, res, g, c1[g], cb1s, v);
                pack_scaled<T>(v, scf, out + 4 * g4);
              } else {
                uint32_t c2[4] = {0, 0, 0, 0};
                if (kTwo) {
                  const int i2 = (int)(s2[h] >> (4 * g));  // the shuffle takes it modulo 16
#pragma unroll
                  for (int w4 = 0; w4 < 4; ++w4) c2[w4] = __shfl_sync(0xffffffffu, cb2r[w4], i2, 16);
                }
                decode_scaled<T, kTwo>(c1[g], c2, sc, out + 4 * g4);
              }
            }
            ptx::tmem_st16(ta + 32u * h + 16u * c, out);
          }
        }
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        if (!ok) break;
        __syncwarp();
        if (lane == 0) arrive_at(full_a(part), 0);
        if (pending) {
          ok = finish_tile(prev, ui - 1);
          pending = false;
        }
      }
      js0 += nsl;
      if (ok && pending) ok = finish_tile(prev, ui - 1);  // no block of this tile was this warp's
      prev = t;
      pending = ok;
    }
    if (ok && pending) ok = finish_tile(prev, ui - 1);
    if (!ok) *abort_flag = 1;
  }

  // Every thread of both blocks gets here (all waits above are bounded).
  ptx::tc_fence_before();
  __syncwarp();
  ptx::cluster_sync();
  if (warp == 1) {
    ptx::tc_fence_after();
    pair_tmem_dealloc(tmem, tcols);
  }
}

// ------------------------------------------------------------------ host side

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<EncodeTiledFn>(ptr);
    return static_cast<EncodeTiledFn>(nullptr);
  }();
  return fn;
}

template <int FMT, typename T, bool kStaged>
static cudaError_t launch_xt_t(ExpertsArgs a, void* xs, int Tmax, int num_sms, cudaStream_t s) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return cudaErrorNotSupported;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (a.rows) {  // x in row order
    cfg.gridDim = dim3(a.T);
    cfg.blockDim = dim3(128);
    cudaError_t e = cudaLaunchKernelEx(&cfg, gather_rows_kernel, reinterpret_cast<const uint4*>(a.x), a.rows,
                                       static_cast<uint4*>(xs), a.w.K / 8, a.x_rows);
    if (e != cudaSuccess) return e;
    a.x = static_cast<const uint16_t*>(xs);
    a.rows = nullptr;
    a.x_rows = a.T;
  }
  XtMaps maps;
  const CUtensorMapDataType dt =
      a.w.act == VQ_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const cuuint64_t dims[2] = {(cuuint64_t)a.w.K, (cuuint64_t)a.x_rows};
  const cuuint64_t strides[1] = {(cuuint64_t)a.w.K * 2};
  const cuuint32_t estr[2] = {1, 1};
  for (int i = 0; i < kXtBoxes; ++i) {
    const int rows = 32 << i;  // half a tile of at most Tmax rows never takes a larger box than Tmax / 2
    const cuuint32_t box[2] = {64, (cuuint32_t)(rows < Tmax / 2 ? rows : Tmax / 2)};
    if (enc(&maps.x[i], dt, 2, const_cast<uint16_t*>(a.x), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  auto kern = experts_tc_kernel<FMT, T, kStaged>;
  const int smem = (int)xt_smem(Tmax);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int nacc = 2 * Tmax + kXtParts * (int)kXtACols <= 512 ? 2 : 1;
  cfg.gridDim = dim3(num_sms / 2 * 2);
  cfg.blockDim = dim3(kXtThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, maps, a, Tmax, nacc);
}

template <typename T>
static cudaError_t launch_xt(const ExpertsArgs& a, void* xs, int Tmax, int num_sms, cudaStream_t s) {
  switch (a.w.fmt) {
    case kFmtRvq12: return launch_xt_t<kFmtRvq12, T, true>(a, xs, Tmax, num_sms, s);
    case kFmtRvq12_4: return launch_xt_t<kFmtRvq12_4, T, true>(a, xs, Tmax, num_sms, s);
    case kFmtVq16Rvq: return launch_xt_t<kFmtVq16Rvq, T, false>(a, xs, Tmax, num_sms, s);
    default: return launch_xt_t<kFmtVq16, T, true>(a, xs, Tmax, num_sms, s);
  }
}

cudaError_t launch_experts_tc(const ExpertsArgs& a, void* xs, int Tmax, int num_sms, cudaStream_t s) {
  return a.w.act == VQ_BF16 ? launch_xt<__nv_bfloat16>(a, xs, Tmax, num_sms, s) : launch_xt<__half>(a, xs, Tmax, num_sms, s);
}

}  // namespace vq
