// Latent attention for 65 .. 128 heads: a pair of CTAs (a cluster of two on neighbouring SMs) walks the
// rows together, 64 heads each, on tcgen05 with cta_group::2.  See latent_attn.cu for the operator and
// the split over the length.
//
// Why a pair.  At these head counts the products, not the cache's bytes, are the larger part, and what
// bounds them is shared-memory bandwidth (128 bytes a clock): one CTA's transposed products read each
// row's 64-dim blocks once per M tile against only 64 columns.  Here the heads are on M, 64 in each
// CTA, and the tensor cores take half of the other operand from each CTA's shared memory:
//     S[h, r]  = Q[h, :576] . Rows[r, :576]      M = 2 x 64 heads, N = 64 rows (32 from each CTA), K = 576
//     O[h, d] += P[h, r] . Rows[r, d]            M = 2 x 64 heads, N = 256 dims (128 from each CTA) twice,
//                                                K = 64 rows
// Per 64-row tile a CTA's operand reads fall from 240 KB to 156 KB, the rows that it converts or loads
// from 72 KB to 68 KB (written) and 41 KB to 29 KB (fp8 codes read).
//
// Shared memory of a tile in CTA r (its dims: [256 r, 256 r + 256), its keys: rows 32 r .. 32 r + 31):
//   S part: its 32 keys, all 576 dims   (nine 64-dim blocks of 32 rows x 128 B)
//   V part: all 64 keys, its 256 dims   (four 64-dim blocks of 64 rows x 128 B)
// The two overlap in the values of its keys and dims, which lie in both: each part needs the same place
// in both CTAs (a descriptor holds for the pair) and its own row order.
//
// TMEM.  An M = 128 accumulator of a pair has head h of each CTA in lane h for the first half of the
// columns and in lane 64 + h for the second half: O is 2 x 128 columns, S 32 columns, double-buffered.
// A softmax thread owns one head and 16 of a tile's 64 keys, so the running maximum is a register and
// the slow path (a maximum that grew by more than 2^8) exchanges four values a head.
//
// The leader (the pair's even CTA) issues every product; the peer's warps signal its barriers.  Every
// wait is bounded; the CTAs leave together (a cluster barrier behind the last wait), so no signal goes
// to a CTA that has left.
#include "latent_attn.cuh"

namespace dsa {
namespace {

constexpr int kHeads = 64;                       // heads per CTA
constexpr int kSBlk = 32 * 128, kVBlk = 64 * 128;
constexpr int kSBytes = kKB * kSBlk, kVBytes = 4 * kVBlk;
constexpr int kStage = kSBytes + kVBytes;        // 68 KB
constexpr int kQBytes = kHeads * kDqk * 2;
constexpr int kPBytes = kHeads * kRows * 2;
constexpr int kOffStage = kQBytes, kOffP = kQBytes + 2 * kStage, kOffShared = kOffP + 2 * kPBytes;
constexpr uint32_t kTmemCols = 512;
constexpr int kSCol = 256;                       // O: columns 0 .. 255
constexpr int kSW = 8, kSoft = 256;              // softmax warps, threads

template <bool FP8>
struct PCfg {
  static constexpr int NP = FP8 ? 8 : 2;         // converters, or the TMA warp and the one behind it
  static constexpr int S_WARP = kSW + NP;
  static constexpr int PV_WARP = S_WARP + 1;
  // fp8: two idle warps complete the MMA warps' warpgroup, which pays for the converters' codes in
  // registers: 8 * 96 + 8 * 112 + 4 * 64 = 20 * 96.
  static constexpr bool REG_SPLIT = FP8;
  static constexpr int REG_LAUNCH = 96, REG_PROD = 112, REG_MMA = 64;
  static constexpr int THREADS = 32 * (PV_WARP + (REG_SPLIT ? 3 : 1));
  static_assert(8 * REG_LAUNCH + 8 * REG_PROD + 4 * REG_MMA <= 20 * REG_LAUNCH, "register split");
};

struct PShared {
  uint64_t full[2], ready[2], empty[2], q_full, q_ready, q_empty, s_full[2], s_empty[2], p_full[2], o_done[2], o_free,
      mma_done;
  uint32_t tmem_base, abort_flag, soft_abort;
  CtaFaults faults;
  Share share;
  float red[4][kHeads];
  float red2[4][kHeads];
};
constexpr int kDynSmem = kOffShared + sizeof(PShared);
static_assert(kDynSmem <= 232448, "shared memory");
static_assert(kOffStage % 1024 == 0 && kStage % 1024 == 0 && kSBytes % 1024 == 0, "swizzled blocks");

// ------------------------------------------------------------------------------- cluster, cta_group::2
__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Arrive on the leader's copy of `bar`.  What the arrival publishes lies in this CTA's own shared
// memory and TMEM and is read there by this SM's tensor core, so the order within the CTA is enough
// (fence.proxy.async, tcgen05 fences and the CTA-scope release before it); a cluster-scope release took
// about 1100 cycles on the path from one tile to the next.
__device__ __forceinline__ void arrive_leader(uint64_t* bar) {
  asm volatile(
      "{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %0, 0;\n mbarrier.arrive.shared::cluster.b64 _, [a];\n}\n" ::"r"(
          smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst_smem)), "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void tmem_relinquish_pair() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// Four K steps of a pair's product with one election (as umma_bf16_x4_elect).
template <int ASTEP, int BSTEP>
__device__ __forceinline__ void umma_pair_x4_elect(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                                   uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, e, t;\n .reg .b64 a1, a2, a3, b1, b2, b3;\n setp.ne.b32 p, %4, 0;\n setp.eq.b32 t, 0, 0;\n"
      " add.s64 a1, %1, %5;\n add.s64 a2, %1, %6;\n add.s64 a3, %1, %7;\n"
      " add.s64 b1, %2, %8;\n add.s64 b2, %2, %9;\n add.s64 b3, %2, %10;\n"
      " elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n"
      " @e tcgen05.mma.cta_group::2.kind::f16 [%0], a1, b1, %3, t;\n"
      " @e tcgen05.mma.cta_group::2.kind::f16 [%0], a2, b2, %3, t;\n"
      " @e tcgen05.mma.cta_group::2.kind::f16 [%0], a3, b3, %3, t;\n}\n" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "n"(ASTEP), "n"(2 * ASTEP), "n"(3 * ASTEP), "n"(BSTEP),
      "n"(2 * BSTEP), "n"(3 * BSTEP)
      : "memory");
}
// Arrive on this barrier in both CTAs when every product issued so far has completed.
__device__ __forceinline__ void commit_pair_elect(uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred e;\n .reg .b16 m;\n mov.b16 m, 3;\n elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n}\n" ::"r"(
          smem_u32(bar))
      : "memory");
}

// ------------------------------------------------------------------------------- the kernel
template <bool FP8, bool SEL>
__global__ void __launch_bounds__(PCfg<FP8>::THREADS, 1)
    latent_pair_kernel(const __grid_constant__ CUtensorMap tmap_s, const __grid_constant__ CUtensorMap tmap_v,
                       const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ LArgs a) {
  using C = PCfg<FP8>;
  extern __shared__ __align__(1024) uint8_t smem[];
  PShared& sh = *reinterpret_cast<PShared*>(smem + kOffShared);
  uint8_t* sQ = smem;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cta_rank();
  const int grp = blockIdx.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.ready[s], FP8 ? C::NP : 2);      // fp8: a group's four warps in each CTA
      mbar_init(&sh.empty[s], 1);
      mbar_init(&sh.s_full[s], 1);
      mbar_init(&sh.s_empty[s], 2 * kSW);
      mbar_init(&sh.p_full[s], 2 * kSW);
      mbar_init(&sh.o_done[s], 1);
    }
    mbar_init(&sh.q_full, 1);
    mbar_init(&sh.q_ready, 1);
    mbar_init(&sh.q_empty, 1);
    mbar_init(&sh.o_free, 2 * kSW);
    mbar_init(&sh.mma_done, 2);
    sh.abort_flag = 0;
    sh.soft_abort = 0;
    sh.faults.bits = sh.faults.count = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == C::PV_WARP) {
    tmem_alloc_pair(&sh.tmem_base, kTmemCols);
    tmem_relinquish_pair();
  }
  if constexpr (SEL) grid_wait();        // the tile counts of the selections
  grid_trigger();
  const long long share = find_share<SEL, C::THREADS>(a, grp, rank == 0, sh.share, sh.faults);
  __syncthreads();
  tc_fence_before();
  cluster_sync_all();                    // barriers and TMEM of both CTAs are there
  tc_fence_after();
  const uint32_t tmem = sh.tmem_base;
  Walk<SEL> walk(a, share > 0 ? sh.share.row0 : 0, share > 0 ? sh.share.tile0 : 0, share);
  Seg sg{};
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, mbar_wait_for(bar, parity, &sh.abort_flag, &sh.faults.bits, a.wait_ns));
  };

  // S warps: this CTA's 64 heads of a segment's row, once the previous ones have been read
  auto load_q = [&](uint32_t it) -> bool {
    if (it > 0 && !wait(&sh.q_empty, (it - 1) & 1)) return false;
    if (lane == 0) {
      mbar_arrive_expect_tx(&sh.q_full, kQBytes);
#pragma unroll 1
      for (int kb = 0; kb < kKB; ++kb)
        tma_load_2d(sQ + kb * (kHeads * 128), &tmap_q, &sh.q_full, kb * 64, sg.row * a.H + static_cast<int>(rank) * kHeads);
    }
    __syncwarp();
    const bool ok = wait(&sh.q_full, it & 1);
    if (!ok && lane == 0) mbar_drain(&sh.q_full, it & 1, 200000000ull);   // the copy lands before we leave
    return ok;
  };

  if (warp >= kSW && warp < C::S_WARP) {
    // ---------------------------------------------------------------- the rows
    if constexpr (C::REG_SPLIT) setmaxnreg_inc<C::REG_PROD>();
    const int pw = warp - kSW;
    uint32_t g = 0;
    bool ok = true;
    if constexpr (!FP8) {
      while (ok && walk.next(sg)) {
        const int32_t* bt = a.pg.block_table + static_cast<size_t>(sg.row) * a.pg.max_pages;
        const int len = row_len(a.pg, sg.row);
        int ahead = __ldg(bt + (sg.i0 >> 1));
        for (int n = 0; n < sg.n; ++n, ++g) {
          const int i = sg.i0 + n, page = ahead;
          if (n + 1 < sg.n) ahead = __ldg(bt + ((i + 1) >> 1));
          const int nv = tile_rows(a, len, i, page);
          uint8_t* st = smem + kOffStage + (g & 1) * kStage;
          if (pw == 0) {
            if (nv == 0 && lane == 0 && rank == 0) report(sh.faults, DEV_ERR_BAD_INDEX);
            if (a.stop_after >= 0 && g >= static_cast<uint32_t>(a.stop_after)) {
              ok = false;   // test hook: stop feeding the pipeline; the waits behind it run out
              break;
            }
            if (g >= 2 && !(ok = wait(&sh.empty[g & 1], ((g >> 1) - 1) & 1))) break;
            if (lane == 0) {
              const int row = nv == 0 ? 0 : (page << kPageShift) + (i & 1) * kRows;
              mbar_arrive_expect_tx(&sh.full[g & 1], kStage);
              tma_load_3d(st, &tmap_s, &sh.full[g & 1], 0, row + 32 * static_cast<int>(rank), 0);
              tma_load_3d(st + kSBytes, &tmap_v, &sh.full[g & 1], 0, row, 4 * static_cast<int>(rank));
            }
            __syncwarp();
          } else {
            // the warp behind the copies: zeros for rows without a key, then the leader may read
            if (!(ok = wait(&sh.full[g & 1], (g >> 1) & 1))) break;
            if (nv < kRows) {
              const uint32_t sp = smem_u32(st), vp = sp + kSBytes;
              const int s0 = max(0, min(32, nv - 32 * static_cast<int>(rank)));
              for (int e = lane; e < (32 - s0) * 8 * kKB; e += 32) {
                const int kb = e / ((32 - s0) * 8), w = e - kb * ((32 - s0) * 8);
                sts128(sp + kb * kSBlk + s0 * 128 + w * 16, 0u, 0u, 0u, 0u);
              }
              for (int e = lane; e < (kRows - nv) * 8 * 4; e += 32) {
                const int vb = e / ((kRows - nv) * 8), w = e - vb * ((kRows - nv) * 8);
                sts128(vp + vb * kVBlk + nv * 128 + w * 16, 0u, 0u, 0u, 0u);
              }
              fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) arrive_leader(&sh.ready[g & 1]);
          }
        }
      }
    } else {
      // Two groups of four warps take the tiles in turn (latent_attn.cu).  A warp takes eight of the
      // CTA's own keys (rows 8 (pw & 3) .. of the S part) and eight of the other 32: own keys x own dims
      // go to both parts, own keys x other dims to the S part, other keys x own dims to the V part.
      // Lane l looks after row l & 15 (own 0 .. 7, other 8 .. 15).
      const uint32_t turn = pw >> 2;                                      // tiles with g & 1 == turn, in slot `turn`
      const int rank_i = static_cast<int>(rank), row_base = 8 * (pw & 3);
      const int c = lane & 3, par = (lane >> 2) & 1, blk4 = lane >> 3;    // codes 16 c .. of block blk4, row parity
      const int my_key = (((lane & 8) != 0) == (rank_i != 0) ? 0 : 32) + row_base + (lane & 7);
      uint4 w[12], rp[2];
      uint32_t sc = 0;                       // scale word and cache row (-1: zeros) of row lane & 15
      int at = -1;
      Walk<SEL> aw(walk);
      Seg as;
      int ai = 0;
      bool alive = aw.next(as);
      int len0 = alive ? row_len(a.pg, as.row) : 0;
      int j1 = -1, row1 = 0, len1 = 0;       // offset known
      int j2 = -1, page2 = -1;               // page known
      bool past2 = false;
      auto advance = [&]() {
        if (alive && ++ai == as.n) {
          ai = 0;
          alive = aw.next(as);
          if (alive) len0 = row_len(a.pg, as.row);
        }
      };
      auto offset_step = [&]() {
        j1 = -1;
        if (!alive) return;
        row1 = as.row;
        len1 = len0;
        const int s = (as.i0 + ai) * kRows + my_key;
        j1 = !SEL ? s : s < a.topk ? __ldg(a.idx + static_cast<size_t>(row1) * a.topk + s) : -1;
        advance();
        advance();
      };
      auto page_step = [&]() {
        j2 = j1;
        past2 = j1 >= len1;
        page2 = -1;
        if (j1 >= 0 && !past2)
          page2 = __ldg(a.pg.block_table + static_cast<size_t>(row1) * a.pg.max_pages + (j1 >> kPageShift));
      };
      auto fetch_step = [&]() {
        const bool in = static_cast<uint32_t>(page2) < static_cast<uint32_t>(a.pg.n_pages);
        // a key on a page outside the cache, or (selected) past the end; the tile's tail is neither
        if (!in && j2 >= 0 && (SEL || (!past2 && my_key == 0)) && lane < 16 && rank == 0) report(sh.faults, DEV_ERR_BAD_INDEX);
        at = in ? (page2 << kPageShift) + (j2 & (kPageRows - 1)) : -1;
        const int safe = max(at, 0);           // a row of the cache in any case: no branch around the loads
        const int off = blk4 * 64 + c * 16;
        int from[8], rf[2];
#pragma unroll
        for (int k = 0; k < 8; ++k) from[k] = __shfl_sync(0xffffffffu, safe, 2 * k + par);   // own 0 .. 3, other 4 .. 7
#pragma unroll
        for (int k = 0; k < 2; ++k) rf[k] = __shfl_sync(0xffffffffu, safe, 4 * k + (lane >> 3));
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint8_t* own = a.latent + static_cast<size_t>(from[k]) * kDv + off;
          const uint8_t* oth = a.latent + static_cast<size_t>(from[4 + k]) * kDv + off;
          w[k] = ldg_once(own + 256 * rank_i);
          w[4 + k] = ldg_once(own + 256 * (1 - rank_i));
          w[8 + k] = ldg_once(oth + 256 * rank_i);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) rp[k] = ldg_once(a.rope + static_cast<size_t>(rf[k]) * 64 + (lane & 7) * 8);
        sc = __ldg(reinterpret_cast<const uint32_t*>(a.scale) + safe);
      };
      if (turn) advance();
      offset_step();
      page_step();
      offset_step();
      fetch_step();
      page_step();
      offset_step();
      const uint32_t sp = smem_u32(smem + kOffStage + turn * kStage), vp = sp + kSBytes;
      auto tile_step = [&]() -> bool {
        if (a.stop_after >= 0 && g >= static_cast<uint32_t>(a.stop_after)) return false;   // test hook
        if (g >= 2 && !wait(&sh.empty[turn], ((g >> 1) - 1) & 1)) return false;
#pragma unroll
        for (int e = 0; e < 12; ++e) {
          const int k = e & 3;
          const int r = row_base + 2 * k + par;                           // row of the S part, or of its half of the V part
          const int half = e >= 4 && e < 8 ? 1 - rank_i : rank_i;
          const int src = (e >= 8 ? 8 : 0) + 2 * k + par;
          const uint32_t rsc = __shfl_sync(0xffffffffu, sc, src);
          const bool in = __shfl_sync(0xffffffffu, at, src) >= 0;
          // dims block 4 half + blk4; a row without a key: times zero
          const uint32_t m = in ? fp8_mult((rsc >> (16 * half + 8 * (blk4 >> 1))) & 0xFFu) : 0u;
          const uint32_t ch0 = ((2 * c) ^ (r & 7)) << 4, ch1 = ((2 * c + 1) ^ (r & 7)) << 4;
          uint32_t o[8];
          fp8x4_to_bf16(w[e].x, m, o[0], o[1]);
          fp8x4_to_bf16(w[e].y, m, o[2], o[3]);
          fp8x4_to_bf16(w[e].z, m, o[4], o[5]);
          fp8x4_to_bf16(w[e].w, m, o[6], o[7]);
          if (e < 8) {
            const uint32_t d = sp + (4 * half + blk4) * kSBlk + r * 128;
            sts128(d + ch0, o[0], o[1], o[2], o[3]);
            sts128(d + ch1, o[4], o[5], o[6], o[7]);
          }
          if (e < 4 || e >= 8) {
            const int key = (e >= 8 ? 32 * (1 - rank_i) : 32 * rank_i) + r;   // key & 7 == r & 7
            const uint32_t d = vp + blk4 * kVBlk + key * 128;
            sts128(d + ch0, o[0], o[1], o[2], o[3]);
            sts128(d + ch1, o[4], o[5], o[6], o[7]);
          }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int q = 4 * k + (lane >> 3), r = row_base + q;
          const uint4 z = __shfl_sync(0xffffffffu, at, q) >= 0 ? rp[k] : make_uint4(0, 0, 0, 0);
          sts128(sp + 8 * kSBlk + r * 128 + (((lane & 7) ^ (r & 7)) << 4), z.x, z.y, z.z, z.w);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) arrive_leader(&sh.ready[turn]);
        fetch_step();
        page_step();
        offset_step();
        return true;
      };
      while (ok && walk.next(sg))
        for (int n = 0; n < sg.n && ok; ++n, ++g)
          if ((g & 1) == turn) ok = tile_step();
    }
    // let every copy this CTA started land before its shared memory can be released
    if constexpr (!FP8) {
      if (pw == 0 && lane == 0)
        for (uint32_t j = g > 2 ? g - 2 : 0; j < g; ++j) mbar_drain(&sh.full[j & 1], (j >> 1) & 1, 200000000ull);
    }
  } else if (warp < kSW) {
    // ---------------------------------------------------------------- softmax + epilogue
    const int qd = warp & 3, cw = warp >> 2;
    const int head = (qd & 1) * 32 + lane;                       // of this CTA's 64
    const int kbase = (qd >> 1) * 32 + cw * 16;                  // this thread's keys of a tile
    const int part = (qd >> 1) * 2 + cw;
    const uint32_t t_lane = static_cast<uint32_t>(qd * 32) << 16;
    const int ghead = static_cast<int>(rank) * kHeads + head;
    uint32_t g = 0;
    bool stop = false;
    while (!stop && walk.next(sg)) {
      const int len = row_len(a.pg, sg.row);
      const int32_t* bt = a.pg.block_table + static_cast<size_t>(sg.row) * a.pg.max_pages;
      const int32_t* irow = SEL ? a.idx + static_cast<size_t>(sg.row) * a.topk : nullptr;
      float m_used = -INFINITY, lp = 0.f, lu = 0.f;
      for (int n = 0; n < sg.n; ++n, ++g) {
        const int i = sg.i0 + n;
        const int sb = g & 1;
        uint32_t mask;                                           // bit c: key kbase + c holds a key
        if constexpr (SEL) {
          const int s = i * kRows + kbase + (lane & 15);
          const int j = s < a.topk ? __ldg(irow + s) : -1;
          bool v = j >= 0 && j < len;
          if (v) v = static_cast<uint32_t>(__ldg(bt + (j >> kPageShift))) < static_cast<uint32_t>(a.pg.n_pages);
          mask = __ballot_sync(0xffffffffu, v) & 0xFFFFu;
        } else {
          const int nv = max(0, min(16, tile_rows(a, len, i, __ldg(bt + (i >> 1))) - kbase));
          mask = (1u << nv) - 1u;
        }
        bool ok = wait(&sh.s_full[sb], (g >> 1) & 1);
        float x[16];
        float mx = -INFINITY;
        if (ok) {
          tc_fence_after();
          uint32_t v[16];
          tmem_ld16(tmem + t_lane + kSCol + sb * 32 + cw * 16, v);
          tmem_ld_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_leader(&sh.s_empty[sb]);
          if (mask == 0xFFFFu) {
#pragma unroll
            for (int c = 0; c < 16; ++c) x[c] = __uint_as_float(v[c]) * a.scale_log2;
          } else {
#pragma unroll
            for (int c = 0; c < 16; ++c) x[c] = (mask >> c) & 1u ? __uint_as_float(v[c]) * a.scale_log2 : -INFINITY;
          }
#pragma unroll
          for (int c = 0; c < 16; ++c) mx = fmaxf(mx, x[c]);
        }
        // the maximum in use follows only when it is outgrown by 2^8 (exact either way)
        if (!ok && lane == 0) sh.soft_abort = 1;
        if (bar_or(1, kSoft, mx > m_used + 8.f || !ok)) {
          sh.red[part][head] = mx;
          if (ok && n > 0) {
            // O may only be rescaled once the previous tile's product has finished
            ok = wait(&sh.o_done[(g - 1) & 1], ((g - 1) >> 1) & 1);
            if (!ok && lane == 0) sh.soft_abort = 1;
          }
          named_bar_sync(1, kSoft);
          stop = sh.soft_abort != 0;
          const float m = fmaxf(fmaxf(sh.red[0][head], sh.red[1][head]), fmaxf(sh.red[2][head], sh.red[3][head]));
          named_bar_sync(1, kSoft);
          if (stop) break;
          tc_fence_after();
          float al = 1.f;
          if (m > m_used + 8.f) {
            al = exp2f(m_used - m);                              // 0 when the old maximum is -inf
            m_used = m;
          }
          lp *= al;
          lu *= al;
          if (n > 0 && __any_sync(0xffffffffu, al != 1.f)) {
#pragma unroll 2
            for (int b = 0; b < 8; ++b) {
              uint32_t o[16];
              tmem_ld16(tmem + t_lane + cw * 128 + b * 16, o);
              tmem_ld_wait();
#pragma unroll
              for (int c = 0; c < 16; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * al);
              tmem_st16(tmem + t_lane + cw * 128 + b * 16, o);
            }
            tmem_st_wait();
          }
        }
        // P = 2^(s - m), rounded to bf16 (at most 2^-9 of each weight, no bias); the output is divided by
        // the sum of the rounded weights, the log-sum-exp takes the sum of the unrounded ones
        const float ms = m_used == -INFINITY ? 0.f : m_used;     // only masked entries so far: 2^(-inf - 0) = 0
        uint32_t pk[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const float p0 = ex2f(x[2 * c] - ms), p1 = ex2f(x[2 * c + 1] - ms);
          const __nv_bfloat162 pb = __floats2bfloat162_rn(p0, p1);
          pk[c] = *reinterpret_cast<const uint32_t*>(&pb);
          lp += __low2float(pb) + __high2float(pb);
          lu += p0 + p1;
        }
        // this P buffer's previous product (two tiles ago) has finished
        if (g >= 2) {
          ok = wait(&sh.o_done[sb], ((g >> 1) - 1) & 1);
          if (!ok && lane == 0) sh.soft_abort = 1;               // seen at the next barrier
        }
        const uint32_t prow = smem_u32(smem + kOffP + sb * kPBytes) + head * 128;
        sts128(prow + (((kbase / 8) ^ (head & 7)) << 4), pk[0], pk[1], pk[2], pk[3]);
        sts128(prow + (((kbase / 8 + 1) ^ (head & 7)) << 4), pk[4], pk[5], pk[6], pk[7]);
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_leader(&sh.p_full[sb]);
      }
      if (stop) break;
      // segment end
      sh.red[part][head] = lp;
      sh.red2[part][head] = lu;
      bool ok = wait(&sh.o_done[(g - 1) & 1], ((g - 1) >> 1) & 1);
      if (!ok && lane == 0) sh.soft_abort = 1;
      named_bar_sync(1, kSoft);
      stop = sh.soft_abort != 0;
      const float l = (sh.red[0][head] + sh.red[1][head]) + (sh.red[2][head] + sh.red[3][head]);
      const float l2 = (sh.red2[0][head] + sh.red2[1][head]) + (sh.red2[2][head] + sh.red2[3][head]);
      named_bar_sync(1, kSoft);                                  // red may be written again
      if (stop) break;
      tc_fence_after();
      const int dim0 = (qd >> 1) * 256 + cw * 128;               // this thread's 128 dims
      const size_t pslot = static_cast<size_t>(grp) * 2 + (sg.i0 > 0 ? 0 : 1);
      const float inv = l == 0.f ? 0.f : 1.f / l;                // a NaN sum stays NaN; no key: zeros
      uint16_t* orow = a.out + (static_cast<size_t>(sg.row) * a.H + ghead) * kDv + dim0;
      float* prow = a.part_o + (pslot * a.H + ghead) * kDv + dim0;
#pragma unroll 1
      for (int b = 0; b < 4; ++b) {
        uint32_t o[32];
        tmem_ld32(tmem + t_lane + cw * 128 + b * 32, o);
        tmem_ld_wait();
        if (ghead >= a.H) continue;
        if (sg.whole) {
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const __nv_bfloat162 ob = __floats2bfloat162_rn(__uint_as_float(o[8 * v + 2 * e]) * inv,
                                                              __uint_as_float(o[8 * v + 2 * e + 1]) * inv);
              w[e] = *reinterpret_cast<const uint32_t*>(&ob);
            }
            reinterpret_cast<uint4*>(orow + b * 32)[v] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        } else {
#pragma unroll
          for (int v = 0; v < 8; ++v)
            reinterpret_cast<uint4*>(prow + b * 32)[v] = make_uint4(o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]);
        }
      }
      if (part == 0 && ghead < a.H) {
        if (sg.whole) {
          if (a.lse)
            a.lse[static_cast<size_t>(sg.row) * a.H + ghead] =
                l2 == 0.f ? -INFINITY : (m_used + log2f(l2)) * 0.69314718055994531f;
        } else {
          const size_t n = static_cast<size_t>(a.n_grp) * 2 * a.H, at = pslot * a.H + ghead;
          a.part_m[at] = m_used;
          a.part_m[n + at] = l;
          a.part_m[2 * n + at] = l2;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_leader(&sh.o_free);
    }
  } else if (rank != 0) {
    // ---------------------------------------------------------------- the peer: tell the leader of its Q
    if constexpr (C::REG_SPLIT) setmaxnreg_dec<C::REG_MMA>();
    if (warp == C::S_WARP) {
      uint32_t it = 0;
      while (walk.next(sg)) {
        if (!load_q(it)) break;
        if (lane == 0) arrive_leader(&sh.q_ready);
        ++it;
      }
    }
  } else {
    // ---------------------------------------------------------------- MMA issuers (and idle warps)
    if constexpr (C::REG_SPLIT) setmaxnreg_dec<C::REG_MMA>();
    const bool issuer = warp <= C::PV_WARP;
    constexpr uint32_t id_qk = idesc_bf16_f32(128, kRows, 0, 0);
    constexpr uint32_t id_pv = idesc_bf16_f32(128, 256, 0, 1);
    uint32_t g = 0, it = 0;
    bool ok = true;
    const uint64_t dq = sdesc_sw128(smem_u32(sQ), 16, 1024);
    while (issuer && ok && walk.next(sg)) {
      if (warp == C::S_WARP) {
        ok = load_q(it) && wait(&sh.q_ready, it & 1);
        for (int n = 0; n < sg.n && ok; ++n, ++g) {
          const int sb = g & 1;
          if (g >= 2 && !(ok = wait(&sh.s_empty[sb], ((g >> 1) - 1) & 1))) break;
          if (!(ok = wait(&sh.ready[sb], (g >> 1) & 1))) break;
          tc_fence_after();
          const uint64_t dk = sdesc_sw128(smem_u32(smem + kOffStage + sb * kStage), 16, 1024);
#pragma unroll
          for (int kb = 0; kb < kKB; ++kb)
            umma_pair_x4_elect<2, 2>(tmem + kSCol + sb * 32, dq + static_cast<uint64_t>((kb * kHeads * 128) >> 4),
                                     dk + static_cast<uint64_t>((kb * kSBlk) >> 4), id_qk, kb ? 1u : 0u);
          commit_pair_elect(&sh.s_full[sb]);
        }
        if (ok) commit_pair_elect(&sh.q_empty);
      } else {
        for (int n = 0; n < sg.n && ok; ++n, ++g) {
          const int sb = g & 1;
          ok = wait(&sh.p_full[sb], (g >> 1) & 1);
          if (ok && n == 0 && it > 0) ok = wait(&sh.o_free, (it - 1) & 1);
          if (!ok) break;
          tc_fence_after();
          const uint64_t dp = sdesc_sw128(smem_u32(smem + kOffP + sb * kPBytes), 16, 1024);
          const uint64_t dv = sdesc_sw128(smem_u32(smem + kOffStage + sb * kStage + kSBytes), kVBlk, 1024);
#pragma unroll
          for (int h = 0; h < 2; ++h)
            umma_pair_x4_elect<2, 128>(tmem + h * 128, dp, dv + static_cast<uint64_t>((2 * h * kVBlk) >> 4), id_pv,
                                       n > 0 ? 1u : 0u);
          commit_pair_elect(&sh.empty[sb]);
          commit_pair_elect(&sh.o_done[sb]);
        }
      }
      ++it;
    }
    // every product this warp issued has completed before TMEM is released
    if (issuer) {
      commit_pair_elect(&sh.mma_done);
      mbar_drain(&sh.mma_done, 0, 200000000ull);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0) publish_faults(a, sh.faults);
  cluster_sync_all();                    // neither CTA signals, reads or is read any more
  tc_fence_after();
  if (warp == C::PV_WARP) tmem_dealloc_pair(tmem, kTmemCols);
}

template <bool FP8, bool SEL>
cudaError_t launch_t(const CUtensorMap& ts, const CUtensorMap& tv, const CUtensorMap& tq, const LArgs& a, cudaStream_t st) {
  cudaError_t e = smem_attr_once<latent_pair_kernel<FP8, SEL>>(kDynSmem);
  if (e != cudaSuccess) return e;
  if constexpr (PCfg<FP8>::REG_SPLIT) {
    // as in the one-CTA kernel: refuse a build whose setmaxnreg.inc could not be granted
    static const int regs = [] {
      cudaFuncAttributes fa{};
      return cudaFuncGetAttributes(&fa, latent_pair_kernel<FP8, SEL>) == cudaSuccess ? fa.numRegs : 0;
    }();
    if (regs < PCfg<FP8>::REG_LAUNCH) return cudaErrorInvalidConfiguration;
  }
  return launch_pdl(latent_pair_kernel<FP8, SEL>, dim3(a.n_cta), PCfg<FP8>::THREADS, kDynSmem, st, SEL, 2, ts, tv, tq, a);
}

}  // namespace

cudaError_t launch_latent_pair(bool fp8, bool sel, const CUtensorMap& tmap_s, const CUtensorMap& tmap_v,
                               const CUtensorMap& tmap_q, const LArgs& a, cudaStream_t st) {
  if (!fp8) return launch_t<false, false>(tmap_s, tmap_v, tmap_q, a, st);
  return sel ? launch_t<true, true>(tmap_s, tmap_v, tmap_q, a, st) : launch_t<true, false>(tmap_s, tmap_v, tmap_q, a, st);
}

}  // namespace dsa
