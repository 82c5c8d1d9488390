// Latent attention of one query row per sequence over a paged latent cache (bf16 or fp8): every
// cached key of the sequence, or the keys an index row selects (fp8), on tcgen05.  The kernel here
// serves up to 64 heads, latent_pair.cu's 65 to 128; split, join and launch are common.
//
//   o[t, h] = sum_j softmax_j(tau * q[t, h] . kv_j) * kv_j[:512]      kv_j: row j of sequence t
//
// All heads of a row read the same latent rows, so the work is a stream of rows with two small
// products on top.  Formulation as in the sparse kernel: a CTA owns HB columns (heads) and walks
// the rows in 64-row tiles, both products run with the rows on the M side,
//     S^T[r, c]  = Rows[r, :576] . Q[c, :576]            M = 64 rows,   N = HB, K = 576
//     O^T[d, c] += Rows[:, d]^T  . P^T[r, c]             M = 128 dims,  N = HB, K = 64
// and a tile lies once in shared memory, as nine 64-dim blocks in the 128-byte swizzle, K-major
// for the first product and MN-major for the second.  O^T (512 x HB fp32) stays in TMEM.
//
// Split over the length.  The tiles of all sequences form one line; each of the G groups of CTAs
// (a group is one CTA per block of HB heads) takes an equal share of consecutive tiles, whatever
// the lengths are: sequences that lie inside a share are finished there, the others leave
// unnormalised partials (fp32 O, the max in use, both sums) that a second kernel joins.  The
// lengths are device data: every CTA finds its share from a block scan over them.
//
// How rows arrive.  bf16: TMA boxes of half a page's rows.  fp8: eight converter warps load codes into
// registers up to two tiles ahead and store the bf16 tile; power-of-two scales make that exact.  Either
// way a tile is filled and freed in two halves (latent dims 0 .. 255; the rest and the rotary dims), so
// the first product starts on one while the other is on its way (16 heads, fp8: 800 -> 747 us; bf16 and
// 64 heads the same).  Rows past the sequence's end, or on a page outside the cache, are written as
// zeros before the products (an uninitialised page may hold NaN, which a zero weight does not cancel).
//
// What bounds it (64 rows of 8K to 131K keys, 4.8M in all; a copy moves 6.78 TB/s here).  bf16 reads
// 5.6 GB: 797 us at 16 heads, 803 at 32, 875 at 64 (7.0, 6.9 and 6.4 TB/s): HBM.  fp8 reads 3.1 GB: 729 us at
// 16 heads, 800 at 32, 1051 at 64 (4.3, 3.9, 3.0 TB/s): no one unit.  At 64 heads L1 and shared memory are at
// 43 % of their rate, the tensor pipe at 37, DRAM at 32; the operand reads and the converters' writes of its
// tiles (312 KB, at 128 bytes a clock) would take some 630 us.  What is left is the way of a tile from codes
// through registers and shared memory to its two products, with two tiles under way; how much of it each step
// takes has not been measured.  Selected keys (2048 of each row): 39 us at 16 heads, 61 at 64: the gathers'
// latency, the partials and their join.
#include <cuda_bf16.h>

#include <algorithm>

#include "latent_attn.cuh"

namespace dsa {
namespace {

constexpr int kBlkBytes = kRows * 128;
constexpr int kTileBytes = kKB * kBlkBytes;

template <int HB, bool FP8>
struct LCfg {
  static constexpr int Q_BYTES = HB * kDqk * 2;
  static constexpr int DYN_SMEM = 1024 + 2 * kTileBytes + Q_BYTES;
  // softmax warps (fp8: four, which leaves the converters 128 registers)
  static constexpr int SW = HB >= 32 && !FP8 ? 8 : 4;
  static constexpr int SOFT = 32 * SW;
  static constexpr int NP = FP8 ? 8 : 1;               // producer warps
  static constexpr int S_WARP = SW + NP;
  static constexpr int PV_WARP = S_WARP + 1;
  static constexpr int THREADS = 32 * (SW + NP + 2);
  static constexpr int CW = HB / (SW / 4);             // columns per softmax warp
  static constexpr int NR = CW / 8;
  static constexpr uint32_t TMEM_COLS = 6 * HB <= 128 ? 128 : 6 * HB <= 256 ? 256 : 512;
  static constexpr int S_COL = 4 * HB;
  static_assert(HB % 16 == 0 && HB <= 64 && CW % 16 == 0, "columns");
};

struct LShared {
  uint64_t full[2][2], empty[2][2];   // by tile parity and half: latent dims 0 .. 255; 256 .. 511 and the rotary dims
  // [2]: by tile parity.  (One p_full for all tiles would not do: the softmax may be two tiles ahead of
  // the PV warp's look, and a barrier two phases on reads as not yet complete.)
  uint64_t q_full, q_empty, s_full[2], s_empty[2], p_full[2], o_done[2], o_free, mma_done;
  uint32_t tmem_base, abort_flag, soft_abort;
  uint32_t keys[2][4];                // SEL, by tile parity and sixteen rows: those that hold a key
  CtaFaults faults;
  Share share;
  alignas(16) float red[4][64];
  alignas(16) float red2[4][64];
  alignas(16) float m_used[64];
  alignas(16) float l_run[64];
  alignas(16) float l_sum[64];
  alignas(16) float alpha[64];
};
static_assert(LCfg<64, true>::DYN_SMEM + sizeof(LShared) <= 232448, "HB = 64 must fit in shared memory");

template <int HB, bool FP8, bool SEL>
__global__ void __launch_bounds__(LCfg<HB, FP8>::THREADS, 1)
    latent_attn_kernel(const __grid_constant__ CUtensorMap tmap_kv, const __grid_constant__ CUtensorMap tmap_v,
                       const __grid_constant__ CUtensorMap tmap_q,
                       const __grid_constant__ LArgs a) {
  using C = LCfg<HB, FP8>;
  constexpr int NR = C::NR;
  static_assert(FP8 || !SEL, "selected rows of a bf16 cache take the sparse kernel's gather walk");
  extern __shared__ uint8_t smem_raw[];
  __shared__ LShared sh;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sT = smem;                        // two tiles
  uint8_t* sQ = smem + 2 * kTileBytes;       // HB x 576, nine blocks of HB x 128 B
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int grp = blockIdx.x / a.n_hb, hb = blockIdx.x - grp * a.n_hb;

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      // fp8: each warp of the group (second half: and each thread's copies)
      mbar_init(&sh.full[s][0], FP8 ? C::NP / 2 : 1);
      mbar_init(&sh.full[s][1], FP8 ? 33 * (C::NP / 2) : 1);
      mbar_init(&sh.empty[s][0], 1);
      mbar_init(&sh.empty[s][1], 1);
      mbar_init(&sh.s_full[s], 1);
      mbar_init(&sh.s_empty[s], C::SW);
      mbar_init(&sh.p_full[s], C::SW);
      mbar_init(&sh.o_done[s], 1);
    }
    mbar_init(&sh.q_full, 1);
    mbar_init(&sh.q_empty, 1);
    mbar_init(&sh.o_free, C::SW);
    mbar_init(&sh.mma_done, 2);
    sh.abort_flag = 0;
    sh.soft_abort = 0;
    sh.faults.bits = sh.faults.count = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (threadIdx.x == 32) {
    tma_prefetch_desc(&tmap_q);
    if constexpr (!FP8) {
      tma_prefetch_desc(&tmap_kv);
      tma_prefetch_desc(&tmap_v);
    }
  }
  if (warp == C::PV_WARP) {
    tmem_alloc(&sh.tmem_base, C::TMEM_COLS);
    tmem_relinquish();
  }
  grid_trigger();
  grid_wait();
  const long long share = find_share<SEL, C::THREADS>(a, grp, hb == 0, sh.share, sh.faults);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem_base;
  Walk<SEL> walk(a, share > 0 ? sh.share.row0 : 0, share > 0 ? sh.share.tile0 : 0, share);
  Seg sg{};

  if (warp >= C::SW && warp < C::S_WARP) {
    // ---------------------------------------------------------------- Q and the rows
    const int pw = warp - C::SW;
    uint32_t g = 0;
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, wait_bar(bar, parity, &sh.abort_flag, &sh.faults.bits, a.wait_ns));
    };
    if constexpr (!FP8) {
      while (ok && walk.next(sg)) {
        const int32_t* bt = a.pg.block_table + static_cast<size_t>(sg.row) * a.pg.max_pages;
        int ahead = gload(bt + (sg.i0 >> 1));
        for (int n = 0; n < sg.n && ok; ++n, ++g) {
          const int i = sg.i0 + n, page = ahead;
          if (n + 1 < sg.n) ahead = gload(bt + ((i + 1) >> 1));
          const bool bad = page < 0 || page >= a.pg.n_pages;
          if (bad && lane == 0 && hb == 0) report(sh.faults, DEV_ERR_BAD_INDEX);
          if (a.stop_after >= 0 && g >= static_cast<uint32_t>(a.stop_after)) {
            ok = false;   // test hook: stop feeding the pipeline; the waits behind it run out
            break;
          }
          uint8_t* st = sT + (g & 1) * kTileBytes;
          const int row = bad ? 0 : (page << kPageShift) + (i & 1) * kRows;
#pragma unroll 1
          for (int h = 0; h < 2 && ok; ++h) {
            uint64_t* full = &sh.full[g & 1][h];
            if (g >= 2) ok = wait(&sh.empty[g & 1][h], ((g >> 1) - 1) & 1);
            if (ok && lane == 0) {
              mbar_arrive_expect_tx(full, (4 + h) * kBlkBytes);
              tma_load_3d(st + 4 * h * kBlkBytes, &tmap_v, full, 0, row, 4 * h);
              if (h) tma_load_3d(st + 8 * kBlkBytes, &tmap_kv, full, 0, row, 8);
            }
          }
          __syncwarp();
        }
      }
    }
    if constexpr (FP8) {
      // Two groups of four warps take the tiles in turn, so one group's loads are in flight while the
      // other converts; a warp takes sixteen rows of its group's tiles.  (One group with two tiles in
      // flight per warp was slower: a wait for any result also waited for the other tile's loads.)
      // A load instruction takes 256 bytes of two rows, whole 128-byte lines; eight lanes of a store
      // phase cover two rows x every other 16-byte chunk, which the swizzle spreads over all banks.
      // Lane l looks after row l & 15: its offset is found two of the group's tiles ahead, its page
      // one, its codes as soon as the registers are free, across segments.  The rotary dims, which
      // need no conversion, are copied when the slot is free, out of L2.
      const uint32_t turn = pw >> 2;                                      // tiles with g & 1 == turn, in slot `turn`
      const int row_base = 16 * (pw & 3), my_row = row_base + (lane & 15);
      const int c = lane & 3, par = (lane >> 2) & 1, blk4 = lane >> 3;    // codes 16 c .. of block blk4 (+ 4), row parity
      uint4 w[16];
      uint32_t sc = 0;                       // scale word of row lane & 15
      int at = -1;                           // its cache row (-1: zeros)
      Walk<SEL> aw(walk);
      Seg as;
      int ai = 0;
      bool alive = aw.next(as);
      int len0 = alive ? row_len(a.pg, as.row) : 0;
      int j1 = -1, row1 = 0, len1 = 0;       // offset of row lane & 15 known
      int j2 = -1, page2 = -1;               // page known
      bool past2 = false;
      auto advance = [&]() {
        if (alive && ++ai == as.n) {
          ai = 0;
          alive = aw.next(as);
          if (alive) len0 = row_len(a.pg, as.row);
        }
      };
      int j0 = -1, row0 = 0, lenx = 0;       // the offset after that, found while w holds nothing
      auto offset_step = [&]() {
        j1 = j0;         // (asked for a tile ago)
        row1 = row0;
        len1 = lenx;
        j0 = -1;
        if (!alive) return;
        row0 = as.row;
        lenx = len0;
        const int s = (as.i0 + ai) * kRows + my_row;
        j0 = !SEL ? s : s < a.topk ? gload(a.idx + static_cast<size_t>(row0) * a.topk + s) : -1;
        advance();
        advance();
      };
      auto page_step = [&]() {
        j2 = j1;
        past2 = j1 >= len1;
        page2 = -1;
        // (unselected: the page of a row past the end is still the tile's page)
        if (j1 >= 0 && (!SEL || !past2))
          page2 = gload(a.pg.block_table + static_cast<size_t>(row1) * a.pg.max_pages + (j1 >> kPageShift));
      };
      auto fetch_step = [&]() {
        const bool in = static_cast<uint32_t>(page2) < static_cast<uint32_t>(a.pg.n_pages);
        // a key on a page outside the cache, or (selected) past the end; the tile's tail is neither
        if (!in && j2 >= 0 && (SEL || my_row == 0) && lane < 16 && hb == 0) report(sh.faults, DEV_ERR_BAD_INDEX);
        const int row = in ? (page2 << kPageShift) + (j2 & (kPageRows - 1)) : 0;   // a row of the cache in any case
        at = in && !past2 ? row : -1;
        const int off = blk4 * 64 + c * 16;
        if constexpr (SEL) {
          int from[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) from[k] = __shfl_sync(0xffffffffu, row, 2 * k + par);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint8_t* src = a.latent + static_cast<size_t>(from[k]) * kDv + off;
            w[2 * k] = gload_once(src);
            w[2 * k + 1] = gload_once(src + 256);
          }
        } else {
          // the tile's rows follow one another (rows past the end lie in the same page)
          const uint8_t* src = a.latent + static_cast<size_t>(row + (in ? par - (lane & 15) : par)) * kDv + off;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            w[2 * k] = gload_once(src + 2 * k * kDv);
            w[2 * k + 1] = gload_once(src + 2 * k * kDv + 256);
          }
        }
        sc = gload(reinterpret_cast<const uint32_t*>(a.scale) + row);
        asm volatile("prefetch.global.L2 [%0];" ::"l"(a.rope + static_cast<size_t>(row) * 64));
      };
      if (turn) advance();
      offset_step();
      offset_step();
      page_step();
      offset_step();
      fetch_step();
      page_step();
      const uint32_t tile = smem_u32(sT + turn * kTileBytes);
      // the lane's line of row par in block blk4, swizzled for chunk 2 c; row 2 k + par's lies 256 k on, its
      // swizzle differs by 2 k (mod 8)
      const uint32_t lane_line =
          tile + blk4 * kBlkBytes + (row_base + par) * 128 + (static_cast<uint32_t>((2 * c) ^ par) << 4);
      // one tile: registers -> the bf16 tile, then the registers' next fetch
      auto tile_step = [&]() -> bool {
        if (a.stop_after >= 0 && g >= static_cast<uint32_t>(a.stop_after)) return false;   // test hook
        const uint32_t line = opaque(lane_line);
        uint32_t rsc[8];                     // scale words of this lane's rows; all ones: no key
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          rsc[k] = __shfl_sync(0xffffffffu, sc, 2 * k + par);
          if (__shfl_sync(0xffffffffu, at, 2 * k + par) < 0) rsc[k] = 0xFFFFFFFFu;
        }
        // half by half: the first product starts on the first while the second is converted, and the
        // previous tile's second product leaves the first half before it is done with the other
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (g >= 2 && !wait(&sh.empty[turn][h], ((g >> 1) - 1) & 1)) return false;
          if (h == 1) {
            const uint32_t rl = opaque(tile) + 8 * kBlkBytes + row_base * 128;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int q = 4 * k + (lane >> 3);                          // row, 16-byte chunk lane & 7
              const int from = __shfl_sync(0xffffffffu, at, q);
              cp_async_16_zfill(rl + q * 128 + (((lane & 7) ^ (q & 7)) << 4),
                                a.rope + static_cast<size_t>(max(from, 0)) * 64 + (lane & 7) * 8, from >= 0);
            }
            cp_async_mbar_arrive(&sh.full[turn][1]);
            if constexpr (SEL) {
              const uint32_t keys = __ballot_sync(0xffffffffu, at >= 0) & 0xFFFFu;
              if (lane == 0) sh.keys[turn][pw & 3] = keys;
            }
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint32_t d = line ^ (static_cast<uint32_t>((2 * k) & 7) << 4);
            // a row without a key: times zero
            const uint32_t m = rsc[k] == 0xFFFFFFFFu ? 0u : fp8_mult((rsc[k] >> (16 * h + 8 * (blk4 >> 1))) & 0xFFu);
            const uint4 v = w[2 * k + h];
            uint32_t o[8];
            fp8x4_to_bf16(v.x, m, o[0], o[1]);
            fp8x4_to_bf16(v.y, m, o[2], o[3]);
            fp8x4_to_bf16(v.z, m, o[4], o[5]);
            fp8x4_to_bf16(v.w, m, o[6], o[7]);
            sts128(d + 256 * k + 4 * h * kBlkBytes, o[0], o[1], o[2], o[3]);
            sts128((d ^ 16u) + 256 * k + 4 * h * kBlkBytes, o[4], o[5], o[6], o[7]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.full[turn][h]);
        }
        offset_step();
        fetch_step();
        page_step();
        return true;
      };
      for (g = turn; ok && g < static_cast<uint32_t>(share); g += 2) ok = tile_step();
      cp_async_wait<0>();
    }
    // let every copy this CTA started land before its shared memory can be released (a wait that ran out
    // between a tile's halves leaves one more wait here than copies: bounded)
    if constexpr (!FP8) {
      if (lane == 0)
        for (uint32_t j = g > 2 ? g - 2 : 0; j < g; ++j)
          for (int h = 0; h < 2; ++h) mbar_drain(&sh.full[j & 1][h], (j >> 1) & 1, 200000000ull);
    }
  } else if (warp < C::SW) {
    // ---------------------------------------------------------------- softmax + epilogue
    constexpr int kSoft = C::SOFT;
    const int tid = threadIdx.x;
    const int qd = warp & 3;                       // TMEM lane quarter
    const int c_off = (warp >> 2) * C::CW;         // this warp's columns: [c_off, c_off + CW)
    const int r0 = qd * 16 + (lane >> 2);          // S^T rows held: r0 and r0 + 8
    const int cq = 2 * (lane & 3);                 // column pair within each group of 8 columns
    const uint32_t t_lane = static_cast<uint32_t>(qd * 32) << 16;
    const int n_cols = min(HB, a.H - hb * HB);
    // A failed (timed-out) wait is published through sh.soft_abort, written only before a
    // named barrier and read right after it, so all softmax warps leave at the same point.
    uint32_t g = 0;
    bool stop = false;
    while (!stop && walk.next(sg)) {
      if (tid < HB) sh.m_used[tid] = -INFINITY;
      float lp[2 * NR], lu[2 * NR];   // per column: sums of the rounded weights, and of the weights
#pragma unroll
      for (int c = 0; c < 2 * NR; ++c) lp[c] = lu[c] = 0.f;
      named_bar_sync(1, kSoft);
      const int len = row_len(a.pg, sg.row);
      const int32_t* bt = a.pg.block_table + static_cast<size_t>(sg.row) * a.pg.max_pages;
      for (int n = 0; n < sg.n; ++n, ++g) {
        const int i = sg.i0 + n;
        const int sb = g & 1;
        bool rv0, rv1;                 // rows r0 / r0 + 8 hold a key
        if constexpr (!SEL) {
          const int nv = tile_rows(a, len, i, gload(bt + (i >> 1)));
          rv0 = r0 < nv;
          rv1 = r0 + 8 < nv;
        }
        bool ok = wait_bar(&sh.s_full[sb], (g >> 1) & 1, &sh.abort_flag, &sh.faults.bits, a.wait_ns);
        if constexpr (SEL) {
          // (long complete: S took the tile.  Looking the rows up here once more, two loads one after the other,
          // held up the tiles: 64 heads, 128 selections of 2048, 112 us where this takes 99.)
          ok = ok && wait_bar(&sh.full[sb][1], (g >> 1) & 1, &sh.abort_flag, &sh.faults.bits, a.wait_ns);
          const uint32_t keys = sh.keys[sb][qd] >> (lane >> 2);
          rv0 = keys & 1u;
          rv1 = keys & 0x100u;
        }
        ok = __all_sync(0xffffffffu, ok);
        float sc[4 * NR];   // [4k + j]: j = 0,1 row r0 columns 8k+cq, +1;  j = 2,3 row r0 + 8
        bool need = false;
        if (ok) {
          tc_fence_after();
          uint32_t v[4 * NR];
          tmem_ld_16x256b<NR>(tmem + t_lane + C::S_COL + sb * HB + c_off, v);
          tmem_ld_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.s_empty[sb]);
#pragma unroll
          for (int kk = 0; kk < NR; ++kk) {
            const float2 mu = *reinterpret_cast<const float2*>(&sh.m_used[c_off + 8 * kk + cq]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const bool valid = (j & 2) ? rv1 : rv0;
              const float x = valid ? __uint_as_float(v[4 * kk + j]) * a.scale_log2 : -INFINITY;
              sc[4 * kk + j] = x;
              need |= x > ((j & 1) ? mu.y : mu.x) + 8.f;   // only a max that grew by > 2^8 forces a rescale
            }
          }
        }
        // one barrier-reduction per tile decides whether the slow path runs
        if (!ok && lane == 0) sh.soft_abort = 1;
        if (bar_or(1, kSoft, need || !ok)) {
          if (ok) {
#pragma unroll
            for (int kk = 0; kk < NR; ++kk) {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float x = fmaxf(sc[4 * kk + e], sc[4 * kk + 2 + e]);
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                if (lane < 4) sh.red[qd][c_off + 8 * kk + cq + e] = x;
              }
            }
            // O^T may only be rescaled once the previous tile's PV has finished
            if (n > 0) {
              ok = wait_bar(&sh.o_done[(g - 1) & 1], ((g - 1) >> 1) & 1, &sh.abort_flag, &sh.faults.bits, a.wait_ns);
              ok = __all_sync(0xffffffffu, ok);
              if (!ok && lane == 0) sh.soft_abort = 1;
            }
          }
          named_bar_sync(1, kSoft);
          stop = sh.soft_abort != 0;
          if (!stop && tid < HB) {
            const float m = fmaxf(fmaxf(sh.red[0][tid], sh.red[1][tid]), fmaxf(sh.red[2][tid], sh.red[3][tid]));
            float al = 1.f;
            if (m > sh.m_used[tid] + 8.f) {
              al = exp2f(sh.m_used[tid] - m);         // 0 when the old max is -inf
              sh.m_used[tid] = m;
            }
            sh.alpha[tid] = al;
          }
          named_bar_sync(1, kSoft);
          if (stop) break;
          tc_fence_after();
          bool any = false;
#pragma unroll
          for (int kk = 0; kk < NR; ++kk) {
            const float2 al = *reinterpret_cast<const float2*>(&sh.alpha[c_off + 8 * kk + cq]);
            lp[2 * kk] *= al.x;
            lp[2 * kk + 1] *= al.y;
            lu[2 * kk] *= al.x;
            lu[2 * kk + 1] *= al.y;
          }
#pragma unroll
          for (int c0 = 0; c0 < HB; c0 += 16) {
            float ar[16];
            lrow16(ar, &sh.alpha[c0]);
#pragma unroll
            for (int c = 0; c < 16; ++c) any |= ar[c] != 1.f;
          }
          if (any && n > 0) {
#pragma unroll 1
            for (int b = 0; b < 4; ++b) {
#pragma unroll 1
              for (int hw = 0; hw < C::CW / 16; ++hw) {
                const int hh = c_off / 16 + hw;
                uint32_t o[16];
                tmem_ld16(tmem + t_lane + b * HB + hh * 16, o);
                tmem_ld_wait();
                float ar[16];
                lrow16(ar, &sh.alpha[hh * 16]);
#pragma unroll
                for (int h = 0; h < 16; ++h) o[h] = __float_as_uint(__uint_as_float(o[h]) * ar[h]);
                tmem_st16(tmem + t_lane + b * HB + hh * 16, o);
              }
            }
            tmem_st_wait();
          }
        }
        // P = 2^(s - m), rounded to bf16 for the second product (at most 2^-8 of each weight, no
        // bias), into the tile's rope block, which S^T no longer needs.  The output is divided by
        // the sum of the rounded weights, so that they add up to one; the log-sum-exp takes the
        // sum of the unrounded ones.
        const uint32_t p_base = smem_u32(sT + sb * kTileBytes + (kKB - 1) * kBlkBytes);
#pragma unroll
        for (int kk = 0; kk < NR; ++kk) {
          float2 mu = *reinterpret_cast<const float2*>(&sh.m_used[c_off + 8 * kk + cq]);
          mu.x = mu.x == -INFINITY ? 0.f : mu.x;      // only masked entries so far: 2^(-inf - 0) = 0
          mu.y = mu.y == -INFINITY ? 0.f : mu.y;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int r = r0 + 8 * h;
            const float p0 = ex2f(sc[4 * kk + 2 * h] - mu.x);
            const float p1 = ex2f(sc[4 * kk + 2 * h + 1] - mu.y);
            const __nv_bfloat162 pb = __floats2bfloat162_rn(p0, p1);
            const int chunk = c_off / 8 + kk;
            sts32(p_base + r * 128 + ((chunk ^ (r & 7)) << 4) + cq * 2, *reinterpret_cast<const uint32_t*>(&pb));
            lp[2 * kk] += __low2float(pb);
            lp[2 * kk + 1] += __high2float(pb);
            lu[2 * kk] += p0;
            lu[2 * kk + 1] += p1;
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_full[sb]);
      }
      if (stop) break;
      // segment end: column sums over the 64 rows, then the output or a partial
#pragma unroll
      for (int kk = 0; kk < NR; ++kk) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = lp[2 * kk + e], y = lu[2 * kk + e];
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) {
            x += __shfl_xor_sync(0xffffffffu, x, o);
            y += __shfl_xor_sync(0xffffffffu, y, o);
          }
          if (lane < 4) {
            sh.red[qd][c_off + 8 * kk + cq + e] = x;
            sh.red2[qd][c_off + 8 * kk + cq + e] = y;
          }
        }
      }
      bool ok = wait_bar(&sh.o_done[(g - 1) & 1], ((g - 1) >> 1) & 1, &sh.abort_flag, &sh.faults.bits, a.wait_ns);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok && lane == 0) sh.soft_abort = 1;
      named_bar_sync(1, kSoft);
      stop = sh.soft_abort != 0;
      if (tid < HB) {
        const float l = (sh.red[0][tid] + sh.red[1][tid]) + (sh.red[2][tid] + sh.red[3][tid]);
        sh.l_run[tid] = l;
        sh.alpha[tid] = l == 0.f ? 0.f : 1.f / l;   // a NaN sum stays NaN; a sum of zero (no key) gives zeros
        sh.l_sum[tid] = (sh.red2[0][tid] + sh.red2[1][tid]) + (sh.red2[2][tid] + sh.red2[3][tid]);
      }
      named_bar_sync(1, kSoft);
      if (stop) break;
      tc_fence_after();
      const size_t pslot = static_cast<size_t>(grp) * 2 + (sg.i0 > 0 ? 0 : 1);
#pragma unroll 1
      for (int hw = 0; hw < C::CW / 16; ++hw) {
        const int hh = c_off / 16 + hw;
#pragma unroll 1
        for (int b2 = 0; b2 < 4; b2 += 2) {
          uint32_t o[2][16];
#pragma unroll
          for (int b = 0; b < 2; ++b) tmem_ld16(tmem + t_lane + (b2 + b) * HB + hh * 16, o[b]);
          tmem_ld_wait();
          if (sg.whole) {
            uint16_t* orow = a.out + (static_cast<size_t>(sg.row) * a.H + hb * HB) * kDv + qd * 32 + lane + b2 * 128;
            float inv[16];
            lrow16(inv, &sh.alpha[hh * 16]);
#pragma unroll
            for (int h = 0; h < 16; ++h) {
              const int c = hh * 16 + h;
              if (c >= n_cols) continue;
#pragma unroll
              for (int b = 0; b < 2; ++b) {
                const __nv_bfloat16 ob = __float2bfloat16_rn(__uint_as_float(o[b][h]) * inv[h]);
                orow[static_cast<size_t>(c) * kDv + b * 128] = *reinterpret_cast<const uint16_t*>(&ob);
              }
            }
          } else {
            float* prow = a.part_o + (pslot * a.H + hb * HB) * kDv + qd * 32 + lane + b2 * 128;
#pragma unroll
            for (int h = 0; h < 16; ++h) {
              const int c = hh * 16 + h;
              if (c >= n_cols) continue;
#pragma unroll
              for (int b = 0; b < 2; ++b) prow[static_cast<size_t>(c) * kDv + b * 128] = __uint_as_float(o[b][h]);
            }
          }
        }
      }
      if (tid < n_cols) {
        if (sg.whole) {
          if (a.lse) {
            const float l = sh.l_sum[tid];
            a.lse[static_cast<size_t>(sg.row) * a.H + hb * HB + tid] =
                l == 0.f ? -INFINITY : (sh.m_used[tid] + log2f(l)) * 0.69314718055994531f;
          }
        } else {
          const size_t n = static_cast<size_t>(a.n_grp) * 2 * a.H, at = pslot * a.H + hb * HB + tid;
          a.part_m[at] = sh.m_used[tid];
          a.part_m[n + at] = sh.l_run[tid];
          a.part_m[2 * n + at] = sh.l_sum[tid];
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.o_free);
      named_bar_sync(1, kSoft);        // per-column state may be reset now
    }
  } else {
    // ---------------------------------------------------------------- MMA issuers
    constexpr uint32_t id_qk = idesc_bf16_f32(64, HB, 0, 0);
    constexpr uint32_t id_pv = idesc_bf16_f32(128, HB, 1, 1);
    const uint32_t st0 = smem_u32(sT);
    uint32_t g = 0, it = 0;
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, wait_bar(bar, parity, &sh.abort_flag, &sh.faults.bits, a.wait_ns));
    };
    const uint64_t dq0 = sdesc_sw128(smem_u32(sQ), 16, 1024);
    while (ok && walk.next(sg)) {
      if (warp == C::S_WARP) {
        const int len = row_len(a.pg, sg.row);
        const int32_t* bt = a.pg.block_table + static_cast<size_t>(sg.row) * a.pg.max_pages;
        // the segment's HB rows of q, once the previous ones have been read
        if (it > 0 && !(ok = wait(&sh.q_empty, (it - 1) & 1))) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&sh.q_full, C::Q_BYTES);
#pragma unroll 1
          for (int kb = 0; kb < kKB; ++kb)
            tma_load_2d(sQ + kb * (HB * 128), &tmap_q, &sh.q_full, kb * 64, sg.row * a.H + hb * HB);
        }
        __syncwarp();
        ok = wait(&sh.q_full, it & 1);
        if (!ok && lane == 0) mbar_drain(&sh.q_full, it & 1, 200000000ull);   // the copy lands before we leave
        for (int n = 0; n < sg.n && ok; ++n, ++g) {
          const int sb = g & 1;
          int nv = kRows;
          if constexpr (!FP8) nv = tile_rows(a, len, sg.i0 + n, gload(bt + ((sg.i0 + n) >> 1)));
          if (g >= 2 && !(ok = wait(&sh.s_empty[sb], ((g >> 1) - 1) & 1))) break;
          const uint64_t da = sdesc_sw128(st0 + sb * kTileBytes, 16, 1024);
          const uint32_t d_s = tmem + C::S_COL + sb * HB;
#pragma unroll
          for (int h = 0; h < 2 && ok; ++h) {
            if (!(ok = wait(&sh.full[sb][h], (g >> 1) & 1))) break;
            if constexpr (FP8) {
              fence_proxy_async_smem();        // the rotary dims' cp.async copies
            } else if (nv < kRows) {
              // rows without a key become zeros in the blocks of latent dims (a swizzled row is one 128-byte
              // line of its block; their rotary dims only reach masked scores)
#pragma unroll 1
              for (int kb = 4 * h; kb < 4 * h + 4; ++kb) {
                const uint32_t blk = st0 + sb * kTileBytes + kb * kBlkBytes;
#pragma unroll 1
                for (uint32_t o = nv * 128 + lane * 16; o < kBlkBytes; o += 512) sts128(blk + o, 0u, 0u, 0u, 0u);
              }
              fence_proxy_async_smem();
              __syncwarp();
            }
            tc_fence_after();
            // (fp8: rolled, for the instruction cache)
#pragma unroll FP8 ? 1 : 5
            for (int kb = 4 * h; kb < 4 + 5 * h; ++kb)
              umma_bf16_x4_elect<2, 2>(d_s, da + static_cast<uint64_t>((kb * kBlkBytes) >> 4),
                                       dq0 + static_cast<uint64_t>((kb * HB * 128) >> 4), id_qk, kb ? 1u : 0u);
          }
          if (!ok) break;
          umma_commit_elect(&sh.s_full[sb]);
        }
        if (ok) umma_commit_elect(&sh.q_empty);
      } else {
        for (int n = 0; n < sg.n && ok; ++n, ++g) {
          ok = wait(&sh.p_full[g & 1], (g >> 1) & 1);
          if constexpr (FP8) fence_proxy_async_smem();
          if (ok && n == 0 && it > 0) ok = wait(&sh.o_free, (it - 1) & 1);
          if (!ok) break;
          tc_fence_after();
          const uint32_t tb = st0 + (g & 1u) * kTileBytes;
          const uint64_t dv = sdesc_sw128(tb, kBlkBytes, 1024);
          const uint64_t dp = sdesc_sw128(tb + (kKB - 1) * kBlkBytes, kBlkBytes, 1024);
          const uint32_t acc0 = n > 0 ? 1u : 0u;
#pragma unroll FP8 ? 1 : 4
          for (int b = 0; b < 4; ++b) {    // four K steps of 16 rows (2048 B)
            umma_bf16_x4_elect<128, 128>(tmem + b * HB, dv + static_cast<uint64_t>((2 * b * kBlkBytes) >> 4), dp, id_pv,
                                         acc0);
            if (b == 1) umma_commit_elect(&sh.empty[g & 1][0]);
          }
          umma_commit_elect(&sh.empty[g & 1][1]);
          umma_commit_elect(&sh.o_done[g & 1]);
        }
      }
      ++it;
    }
    // every MMA this warp issued has completed before TMEM is released
    umma_commit_elect(&sh.mma_done);
    mbar_drain(&sh.mma_done, 0, 200000000ull);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == C::PV_WARP) tmem_dealloc(tmem, C::TMEM_COLS);
  if (threadIdx.x == 0) publish_faults(a, sh.faults);
}

// row_nt[t] = number of 64-slot tiles up to the last slot of idx row t holding an index >= 0; a block
// a row (2048 slots: one round of loads).
__global__ void __launch_bounds__(128) selected_tiles_kernel(const int32_t* idx, int topk, int32_t* row_nt) {
  __shared__ int top;
  grid_trigger();
  grid_wait();
  const int t = blockIdx.x;
  const int32_t* irow = idx + static_cast<size_t>(t) * topk;
  if (threadIdx.x == 0) top = -1;
  __syncthreads();
  int last = -1;
  if ((topk & 3) == 0 && (reinterpret_cast<uintptr_t>(idx) & 15) == 0) {
    const int4* v = reinterpret_cast<const int4*>(irow);
#pragma unroll 4
    for (int s = threadIdx.x; s < topk / 4; s += 128) {
      const int4 q = gload(v + s);
      if (q.x >= 0) last = 4 * s;
      if (q.y >= 0) last = 4 * s + 1;
      if (q.z >= 0) last = 4 * s + 2;
      if (q.w >= 0) last = 4 * s + 3;
    }
  } else {
#pragma unroll 4
    for (int s = threadIdx.x; s < topk; s += 128)
      if (gload(irow + s) >= 0) last = s;
  }
  last = __reduce_max_sync(0xffffffffu, last);
  if ((threadIdx.x & 31) == 0 && last >= 0) atomicMax(&top, last);
  __syncthreads();
  if (threadIdx.x == 0) row_nt[t] = (top + kRows) / kRows;
}

// Joins the partials of the rows that were split: block (b, y) takes the row that begins in group b's
// share and goes on in the next ones (by_row: row b, where there are fewer rows than groups), HPB heads,
// 8 / HPB warps a head; a warp takes every (8 / HPB)-th partial, a lane 16 dims, and the warps' sums meet
// in shared memory.  With M the largest of the partials' maxima m_s and w_s = 2^(m_s - M):
// out = sum w_s O_s / sum w_s lr_s, lse = ln 2 (M + log2 sum w_s l_s).  The order of the sums is fixed.
// Latency bounds it, so two round trips is all there is: every group's start, then the partials' maxima
// and sums and the first O rows together.  One block more puts the CTAs' fault words into the status.
// Few rows, each in many partials, take one head a block (eight warps on one row of 100K keys in 76
// partials, 128 heads: 10 us; 17 with a load of the starts, of the maxima and of the rows behind one
// another; one warp a head 56); many rows, most in two or three, take eight (48 rows, 16 heads: 7 us, 12).
template <int HPB>
__global__ void __launch_bounds__(256) latent_join_kernel(const __grid_constant__ LArgs a, bool by_row) {
  constexpr int kJoinWarps = 8 / HPB;
  constexpr int kAhead = 3;                      // O rows in flight per warp
  constexpr int kLaneGroups = kMostGroups / 32;
  __shared__ float4 sum[HPB][kJoinWarps > 1 ? kJoinWarps - 1 : 1][kJoinWarps > 1 ? kDv / 4 : 1];
  __shared__ float weight[8][kMostGroups];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int hw = warp / kJoinWarps, w = warp % kJoinWarps;
  const int h = blockIdx.y * HPB + hw;
  grid_trigger();
  grid_wait();
  if (blockIdx.x == gridDim.x - 1) {
    if (blockIdx.y != 0 || warp != 0) return;
    uint32_t bits = 0, count = 0;
#pragma unroll 5
    for (int i = lane; i < a.n_cta; i += 32) {
      bits |= a.err[2 * i];
      count += a.err[2 * i + 1];
    }
    bits = __reduce_or_sync(0xffffffffu, bits);
    count = __reduce_add_sync(0xffffffffu, count);
    if (lane == 0) {
      a.status[0] = bits;
      a.status[1] = count;
    }
    return;
  }
  int2 st[kLaneGroups];
#pragma unroll
  for (int k = 0; k < kLaneGroups; ++k)
    st[k] = lane + 32 * k < a.n_grp ? a.start[lane + 32 * k] : make_int2(0x7FFFFFFF, 0);
  int row = blockIdx.x;
  if (!by_row) {
    const int2 s0 = a.start[blockIdx.x], s1 = a.start[blockIdx.x + 1];
    if (s1.x == 0x7FFFFFFF || s1.y == 0 || (s0.x == s1.x && s0.y > 0)) return;   // no row goes on, or it began before
    row = s1.x;
  }
  // the row's groups: from the last that starts at its first tile or before, to the last that starts in it
  uint32_t below = 0;
#pragma unroll
  for (int k = 0; k < kLaneGroups; ++k) {
    below += st[k].x < row || (st[k].x == row && st[k].y == 0) ? 1u : 0u;
    below += st[k].x <= row ? 0x10000u : 0u;
  }
  below = __reduce_add_sync(0xffffffffu, below);
  const int b = static_cast<int>(below & 0xFFFFu) - 1, end = static_cast<int>(below >> 16);
  if (b < 0 || end - b < 2) return;                         // not split
  const size_t n = static_cast<size_t>(a.n_grp) * 2 * a.H;
  auto slot = [&](int c) { return (static_cast<size_t>(c) * 2 + (c == b ? 1 : 0)) * a.H + h; };
  const bool live = h < a.H;
  float M = -INFINITY, lr = 0.f, ls = 0.f;
  float4 acc[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (live) {
    float m[kLaneGroups], l1[kLaneGroups], l2[kLaneGroups];
#pragma unroll
    for (int k = 0; k < kLaneGroups; ++k) {
      const int c = b + lane + 32 * k;
      m[k] = -INFINITY;
      l1[k] = l2[k] = 0.f;
      if (c < end) {
        m[k] = gload(a.part_m + slot(c));
        l1[k] = gload(a.part_m + n + slot(c));
        l2[k] = gload(a.part_m + 2 * n + slot(c));
      }
    }
#pragma unroll 1
    for (int c0 = b + w; c0 < end; c0 += kAhead * kJoinWarps) {
      float4 o[kAhead][4];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int c = c0 + u * kJoinWarps;
        if (c < end) {
          const float4* src = reinterpret_cast<const float4*>(a.part_o + slot(c) * kDv) + lane;
#pragma unroll
          for (int k = 0; k < 4; ++k) o[u][k] = gload(src + 32 * k);
        }
      }
      if (c0 == b + w) {
        // (while the rows are on their way)  A partial without a key weighs nothing; one whose sum is NaN
        // (a NaN score) makes the row NaN even where its maximum says nothing.
#pragma unroll
        for (int k = 0; k < kLaneGroups; ++k) M = fmaxf(M, m[k]);
#pragma unroll
        for (int e = 16; e > 0; e >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, e));
#pragma unroll
        for (int k = 0; k < kLaneGroups; ++k) {
          const float f = m[k] == -INFINITY ? (l1[k] == l1[k] ? 0.f : l1[k]) : exp2f(m[k] - M);
          weight[warp][lane + 32 * k] = f;
          lr += f * l1[k];
          ls += f * l2[k];
        }
        __syncwarp();
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int c = c0 + u * kJoinWarps;
        if (c >= end) break;
        const float f = weight[warp][c - b];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          acc[k].x += f * o[u][k].x;
          acc[k].y += f * o[u][k].y;
          acc[k].z += f * o[u][k].z;
          acc[k].w += f * o[u][k].w;
        }
      }
    }
  }
  if (w > 0) {
#pragma unroll
    for (int k = 0; k < 4; ++k) sum[hw][w - 1][lane + 32 * k] = acc[k];
  }
  __syncthreads();
  if (w > 0 || !live) return;
#pragma unroll
  for (int e = 16; e > 0; e >>= 1) {
    lr += __shfl_xor_sync(0xffffffffu, lr, e);
    ls += __shfl_xor_sync(0xffffffffu, ls, e);
  }
  const float inv = lr == 0.f ? 0.f : 1.f / lr;
  const size_t orow = static_cast<size_t>(row) * a.H + h;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
#pragma unroll
    for (int v = 0; v < kJoinWarps - 1; ++v) {
      const float4 o = sum[hw][v][lane + 32 * k];
      acc[k].x += o.x;
      acc[k].y += o.y;
      acc[k].z += o.z;
      acc[k].w += o.w;
    }
    const __nv_bfloat162 x = __floats2bfloat162_rn(acc[k].x * inv, acc[k].y * inv);
    const __nv_bfloat162 y = __floats2bfloat162_rn(acc[k].z * inv, acc[k].w * inv);
    reinterpret_cast<uint2*>(a.out + orow * kDv)[lane + 32 * k] =
        make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
  }
  if (a.lse && lane == 0) a.lse[orow] = ls == 0.f ? -INFINITY : (M + log2f(ls)) * 0.69314718055994531f;
}

int head_block(int n_heads) { return n_heads <= 16 ? 16 : n_heads <= 32 ? 32 : 64; }

struct Layout {
  int n_hb, n_grp;
  size_t off_err, off_start, off_m, off_ring, off_o, total;
};
Layout latent_layout(int n_q, int n_heads, long long row_tiles_max) {
  Layout L{};
  L.n_hb = (n_heads + head_block(n_heads) - 1) / head_block(n_heads);
  const long long most = (static_cast<long long>(n_q) * row_tiles_max + kMinTiles - 1) / kMinTiles;
  int sms = device_sm_count();
  if (sms <= 0) sms = 152;
  L.n_grp = static_cast<int>(std::max(1LL, std::min<long long>(std::min(sms / L.n_hb, kMostGroups), most)));
  const auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
  size_t o = up(static_cast<size_t>(n_q) * sizeof(int32_t));           // row_nt (selected keys)
  L.off_err = o;
  o += up(static_cast<size_t>(L.n_grp) * L.n_hb * 2 * sizeof(uint32_t));
  L.off_start = o;
  o += up(static_cast<size_t>(L.n_grp) * sizeof(int2));
  L.off_m = o;
  o += up(static_cast<size_t>(L.n_grp) * 2 * n_heads * 3 * sizeof(float));
  L.off_ring = o;
  if (L.n_hb == 2) o += up(static_cast<size_t>(L.n_grp) * kRing * kRows * kDqk * sizeof(uint16_t));
  L.off_o = o;
  o += L.n_grp > 1 ? static_cast<size_t>(L.n_grp) * 2 * n_heads * kDv * sizeof(float) : 0;
  L.total = o;
  return L;
}

template <int HB, bool FP8, bool SEL>
cudaError_t launch_t(const CUtensorMap& tkv, const CUtensorMap& tv, const CUtensorMap& tq, const LArgs& a,
                     cudaStream_t st) {
  using C = LCfg<HB, FP8>;
  cudaError_t e = smem_attr_once<latent_attn_kernel<HB, FP8, SEL>>(C::DYN_SMEM);
  if (e != cudaSuccess) return e;
  return launch_pdl(latent_attn_kernel<HB, FP8, SEL>, dim3(a.n_cta), C::THREADS, C::DYN_SMEM, st, 1, tkv, tv, tq, a);
}
template <int HB>
cudaError_t launch_hb(bool fp8, bool sel, const CUtensorMap& tkv, const CUtensorMap& tv, const CUtensorMap& tq,
                      const LArgs& a, cudaStream_t st) {
  if (!fp8) return launch_t<HB, false, false>(tkv, tv, tq, a, st);
  return sel ? launch_t<HB, true, true>(tkv, tv, tq, a, st) : launch_t<HB, true, false>(tkv, tv, tq, a, st);
}

}  // namespace

namespace {
long long row_tiles_max(const PagedRows& pg, bool selected, int topk) {
  return selected ? (topk + kRows - 1) / kRows : pg.max_pages * 2LL;
}
}  // namespace

LatentRing latent_attn_ring(int n_q, int n_heads, const PagedRows& pg, bool selected, int topk) {
  const Layout L = latent_layout(n_q, n_heads, row_tiles_max(pg, selected, topk));
  return LatentRing{L.off_ring, L.n_hb == 2 ? L.n_grp * kRing * kRows : 0};
}

int latent_attn_q_box_rows(int n_heads) { return head_block(n_heads); }

size_t latent_attn_ws_bytes(int n_q, int n_heads) {
  // the most groups any block table can ask for
  return latent_layout(n_q, n_heads, 1LL << 24).total;
}

cudaError_t launch_latent_attn(const LatentCache& c, const CUtensorMap& tmap_kv, const CUtensorMap& tmap_v,
                               const CUtensorMap& tmap_q, const PagedRows& pg, const int32_t* idx, int n_q, int n_heads,
                               int topk, float scale, void* out, float* lse, uint32_t* status, void* scratch, cudaStream_t st) {
  const bool sel = idx != nullptr;
  const Layout L = latent_layout(n_q, n_heads, row_tiles_max(pg, sel, topk));
  uint8_t* base = static_cast<uint8_t*>(scratch);
  const PipelineDebug dbg = pipeline_debug();
  LArgs a{};
  a.latent = c.latent;
  a.scale = c.scale;
  a.rope = c.rope;
  a.idx = idx;
  a.row_nt = reinterpret_cast<int32_t*>(base);
  a.pg = pg;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.n_q = n_q;
  a.H = n_heads;
  a.topk = topk;
  a.n_grp = L.n_grp;
  a.n_hb = L.n_hb;
  a.n_cta = L.n_grp * L.n_hb;
  a.err = reinterpret_cast<uint32_t*>(base + L.off_err);
  a.scale_log2 = scale * 1.4426950408889634f;
  a.start = reinterpret_cast<int2*>(base + L.off_start);
  a.part_m = reinterpret_cast<float*>(base + L.off_m);
  a.ring = reinterpret_cast<uint16_t*>(base + L.off_ring);
  a.part_o = reinterpret_cast<float*>(base + L.off_o);
  a.status = status;
  a.wait_ns = dbg.wait_ns;
  a.stop_after = dbg.stop_after_tiles;
  cudaError_t e;
  if (sel) {
    const int ps = prof_begin(kProfAttnPrep, st);
    e = launch_pdl(selected_tiles_kernel, dim3(n_q), 128, 0, st, 1, idx, topk, reinterpret_cast<int32_t*>(base));
    prof_end(ps, st);
    if (e != cudaSuccess) return e;
  }
  const int ps = prof_begin(kProfAttn, st);
  if (L.n_hb == 2) {
    e = launch_latent_pair(c.fp8, sel, tmap_kv, tmap_v, tmap_q, a, st);
  } else switch (head_block(n_heads)) {
    case 16: e = launch_hb<16>(c.fp8, sel, tmap_kv, tmap_v, tmap_q, a, st); break;
    case 32: e = launch_hb<32>(c.fp8, sel, tmap_kv, tmap_v, tmap_q, a, st); break;
    default: e = launch_hb<64>(c.fp8, sel, tmap_kv, tmap_v, tmap_q, a, st); break;
  }
  if (e == cudaSuccess && a.n_cta > 1) {
    const int hpb = 8LL * n_q <= L.n_grp ? 1 : 8;      // eight partials a row and more, or fewer
    const bool by_row = n_q < L.n_grp;
    const dim3 grid(std::min(n_q, L.n_grp - 1) + 1, (n_heads + hpb - 1) / hpb);
    e = launch_pdl(hpb == 1 ? latent_join_kernel<1> : latent_join_kernel<8>, grid, 256, 0, st, 1, a, by_row);
  }
  prof_end(ps, st);
  return e;
}

}  // namespace dsa
