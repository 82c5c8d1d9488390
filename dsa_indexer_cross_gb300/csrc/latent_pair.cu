// Latent attention for 65 .. 128 heads: a pair of CTAs (a cluster of two on neighbouring SMs) walks the
// rows together, 64 heads each, on tcgen05 with cta_group::2.  See latent_attn.cu for the operator and
// the split over the length.
//
// Why a pair.  At these head counts the products, not the cache's bytes, are the larger part, and what
// they take most of is shared-memory bandwidth (128 bytes a clock): one CTA's transposed products read each
// row's 64-dim blocks once per M tile against only 64 columns.  Here the heads are on M, 64 in each
// CTA, and the tensor cores take half of the other operand from each CTA's shared memory:
//     S[h, r]  = Q[h, :576] . Rows[r, :576]      M = 2 x 64 heads, N = 64 rows (32 from each CTA), K = 576
//     O[h, d] += P[h, r] . Rows[r, d]            M = 2 x 64 heads, N = 256 dims (128 from each CTA) twice,
//                                                K = 64 rows
// Per 64-row tile a CTA's operand reads fall from 240 KB to 156 KB, the rows that it loads from 72 KB to
// 68 KB, the fp8 rows that it converts from 64 to 32.
//
// Shared memory of a tile in CTA r (its dims: [256 r, 256 r + 256), its keys: rows 32 r .. 32 r + 31):
//   S part: its 32 keys, all 576 dims   (nine 64-dim blocks of 32 rows x 128 B)
//   V part: all 64 keys, its 256 dims   (four 64-dim blocks of 64 rows x 128 B)
// The two overlap in the values of its keys and dims, which lie in both: each part needs the same place
// in both CTAs (a descriptor holds for the pair) and its own row order.  They are filled and freed
// apart: the S part of tile g + 2 as soon as S(g) is complete, the V part once PV(g) is, so the way
// of a tile from its rows to its product does not limit how often one begins (one barrier for both
// parts: 1487 us where the two take 1102, 64 rows of 8K to 131K keys, 128 heads, bf16).
//
// TMEM.  An M = 128 accumulator of a pair has head h of each CTA in lane h for the first half of the
// columns and in lane 64 + h for the second half: O is 2 x 128 columns, S 32 columns, double-buffered.
// A softmax thread owns one head and 16 of a tile's 64 keys, so the running maximum is a register and
// the slow path (a maximum that grew by more than 2^8) exchanges four values a head.
//
// fp8.  The two parts of a tile overlap, so converting into shared memory would convert (or write) the
// overlap twice.  Instead each CTA converts its 32 keys once, whole rows, into a ring of bf16 tiles in the
// workspace that stays in L2 (kRing tiles a pair, 0.6 MB; 45 MB in all), and both CTAs' TMA boxes pick
// their parts from there as they do from a bf16 cache (1900 us and more where converters wrote the parts
// into shared memory).
//
// What bounds it (64 rows of 8K to 131K keys, 4.8M in all).  bf16: 1102 to 1126 us, 1192 TFLOP/s of a measured
// 1924 and 4.9 TB/s of 6.78: operand reads and copies (224 KB a tile, at 128 bytes a clock) would take 80 %
// of that, though the counter of L1 and shared memory stands at 51 %, the tensor pipe at 44, DRAM at 54.
// fp8: 1470 us, 913 TFLOP/s, 2.1 TB/s: the same tiles, with the converters' loads and stores through L1 on
// top (53 %, 33, 24).  No unit is full in either: the rest is the chain from a tile's rows to S, softmax, P and
// the second product, two tiles under way, whose steps have not been measured apart.  (Scoring two tiles with
// one N = 128 product: bf16 1653, fp8 2008 us.)
//
// The leader (the pair's even CTA) issues every product; the peer's warps signal its barriers.  Every
// wait is bounded.  The CTAs leave together (a cluster barrier behind the last wait), so no thread
// signals a CTA that has left.  The leader's commits arrive in both CTAs by themselves, which no barrier
// between threads orders: each CTA waits for the last of them, mma_done, on its own copy before it leaves,
// and none is issued that nobody waits for (q_empty behind the last segment).
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
constexpr int kKT = 16, kOC = 128;               // keys of a tile, O columns per softmax thread
constexpr int kConv = 8;                         // fp8: converter warps = tiles of the ring (kRing)
static_assert(kConv == kRing, "a converter warp for each tile of the ring");

template <bool FP8>
struct PCfg {
  static constexpr int COPY = kSW;               // the TMA warp and the one behind it, for each part (fp8: for both)
  static constexpr int CONV = COPY + (FP8 ? 2 : 4);
  static constexpr int S_WARP = CONV + (FP8 ? kConv : 0);
  static constexpr int PV_WARP = S_WARP + 1;
  static constexpr int THREADS = 32 * (PV_WARP + 1);
};

struct PShared {
  // [2]: by tile parity.  full_*: copies have landed (this CTA); ready_*, s_empty, p_full, o_free, q_ready:
  // the leader's, both CTAs arrive; s_full, o_done, q_empty: S, PV, all of a segment's S complete (both CTAs;
  // q_empty where a segment follows); mma_done: every product complete (both CTAs)
  uint64_t full_s[2], full_v[2], ready_s[2], ready_v[2], q_full, q_ready, q_empty, s_full[2], s_empty[2], p_full[2],
      o_done[2], o_free, mma_done;
  uint64_t ring_full[kRing], ring_empty[kRing];   // fp8: both CTAs arrive on each CTA's
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
// Arrive on the copy of `bar` in the pair's CTA `rank` (0: the leader).  What the arrival publishes lies in
// this CTA's own shared memory and TMEM and is read there by this SM's tensor core, so the order within
// the CTA is enough (fence.proxy.async, tcgen05 fences and the CTA-scope release before it); a
// cluster-scope release took about 1100 cycles on the path from one tile to the next.  (The ring's rows in
// global memory are fenced at GPU scope by their writers.)
__device__ __forceinline__ void arrive_cta(uint64_t* bar, uint32_t rank) {
  asm volatile(
      "{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %0, %1;\n mbarrier.arrive.shared::cluster.b64 _, [a];\n}\n" ::"r"(
          smem_u32(bar)),
      "r"(rank)
      : "memory");
}
__device__ __forceinline__ void arrive_cta_n(uint64_t* bar, uint32_t rank, uint32_t n) {
  asm volatile(
      "{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %0, %1;\n mbarrier.arrive.shared::cluster.b64 _, [a], %2;\n}\n" ::"r"(
          smem_u32(bar)),
      "r"(rank), "r"(n)
      : "memory");
}
__device__ __forceinline__ void fence_proxy_async_global() { asm volatile("fence.proxy.async.global;" ::: "memory"); }
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
      mbar_init(&sh.full_s[s], 1);
      mbar_init(&sh.full_v[s], 1);
      mbar_init(&sh.ready_s[s], 2);
      mbar_init(&sh.ready_v[s], 2);
      mbar_init(&sh.s_full[s], 1);
      mbar_init(&sh.s_empty[s], 2 * kSW);
      mbar_init(&sh.p_full[s], 2 * kSW);
      mbar_init(&sh.o_done[s], 1);
    }
    for (int s = 0; s < kRing; ++s) {
      mbar_init(&sh.ring_full[s], 8);    // the CTAs' converters, for each quarter of their rows
      mbar_init(&sh.ring_empty[s], 3);   // its rows read: both of this CTA's parts, the other's V part
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
  if (threadIdx.x == 32) {
    tma_prefetch_desc(&tmap_q);
    tma_prefetch_desc(&tmap_s);
    tma_prefetch_desc(&tmap_v);
  }
  if (warp == C::PV_WARP) {
    tmem_alloc_pair(&sh.tmem_base, kTmemCols);
    tmem_relinquish_pair();
  }
  grid_trigger();
  grid_wait();
  const long long share = find_share<SEL, C::THREADS>(a, grp, rank == 0, sh.share, sh.faults);
  __syncthreads();
  tc_fence_before();
  cluster_sync_all();                    // barriers and TMEM of both CTAs are there
  tc_fence_after();
  const uint32_t tmem = sh.tmem_base;
  Walk<SEL> walk(a, share > 0 ? sh.share.row0 : 0, share > 0 ? sh.share.tile0 : 0, share);
  Seg sg{};
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, wait_bar(bar, parity, &sh.abort_flag, &sh.faults.bits, a.wait_ns));
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

  if (warp >= C::COPY && warp < C::CONV) {
    // ---------------------------------------------------------------- the rows
    // The first warp copies, the second, behind it, writes zeros for rows without a key (of the V part:
    // a masked score may come from anything, a zero weight does not cancel a NaN) and tells the
    // leader.  bf16: two warps for the S part, two for the V part; fp8: one pair for both, in turn.
    const int pw = warp - C::COPY;
    const bool copies = (pw & 1) == 0;
    const int part0 = FP8 ? 0 : pw >> 1, part1 = FP8 ? 2 : part0 + 1;   // 0: S part, 1: V part
    uint32_t g = 0, slot = 0, lap = 0;       // slot, lap: the tile's place in the ring
    bool ok = true;
    while (ok && walk.next(sg)) {
      const int32_t* bt = a.pg.block_table + static_cast<size_t>(sg.row) * a.pg.max_pages;
      const int len = row_len(a.pg, sg.row);
      int ahead = FP8 ? 0 : gload(bt + (sg.i0 >> 1));
      for (int n = 0; n < sg.n && ok; ++n, ++g) {
        const int i = sg.i0 + n, page = ahead, sb = g & 1;
        if (!FP8 && n + 1 < sg.n) ahead = gload(bt + ((i + 1) >> 1));
        const int nv = FP8 ? kRows : tile_rows(a, len, i, page);
        if (copies) {
          if (nv == 0 && lane == 0 && rank == 0 && part0 == 0) report(sh.faults, DEV_ERR_BAD_INDEX);
          if (a.stop_after >= 0 && g >= static_cast<uint32_t>(a.stop_after)) {
            ok = false;   // test hook: stop feeding the pipeline; the waits behind it run out
            break;
          }
          if constexpr (FP8) {
            if (!(ok = wait(&sh.ring_full[slot], lap & 1))) break;
          }
        }
#pragma unroll 1
        for (int part = part0; part < part1 && ok; ++part) {
          uint64_t* full = part ? &sh.full_v[sb] : &sh.full_s[sb];
          uint8_t* st = smem + kOffStage + sb * kStage + (part ? kSBytes : 0);
          if (copies) {
            if (g >= 2 && !(ok = wait(part ? &sh.o_done[sb] : &sh.s_full[sb], ((g >> 1) - 1) & 1))) break;
            if (lane == 0) {
              int row = nv == 0 ? 0 : (page << kPageShift) + (i & 1) * kRows;
              if constexpr (FP8) {
                row = (grp * kRing + static_cast<int>(slot)) * kRows;
                fence_proxy_async_global();    // the converters' stores, before the copies that read them
              }
              mbar_arrive_expect_tx(full, part ? kVBytes : kSBytes);
              if (part)
                tma_load_3d(st, &tmap_v, full, 0, row, 4 * static_cast<int>(rank));
              else
                tma_load_3d(st, &tmap_s, full, 0, row + 32 * static_cast<int>(rank), 0);
            }
            __syncwarp();
          } else {
            if (!(ok = wait(full, (g >> 1) & 1))) break;
            if (!FP8 && part && nv < kRows) {
#pragma unroll 1
              for (int vb = 0; vb < 4; ++vb) {
#pragma unroll 1
                for (uint32_t o = nv * 128 + lane * 16; o < kVBlk; o += 512) sts128(smem_u32(st) + vb * kVBlk + o, 0u, 0u, 0u, 0u);
              }
              fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) {
              arrive_cta(part ? &sh.ready_v[sb] : &sh.ready_s[sb], 0);
              if constexpr (FP8) {
                arrive_cta(&sh.ring_empty[slot], rank);
                if (part) arrive_cta(&sh.ring_empty[slot], rank ^ 1u);
              }
            }
          }
        }
        if (++slot == kRing) {
          slot = 0;
          ++lap;
        }
      }
    }
    // let every copy this CTA started land before its shared memory can be released (one more wait than
    // copies where the last tile's were not both started: bounded)
    if (copies && lane == 0)
      for (int part = part0; part < part1; ++part)
        for (uint32_t j = g > 2 ? g - 2 : 0; j < g; ++j)
          mbar_drain(part ? &sh.full_v[j & 1] : &sh.full_s[j & 1], (j >> 1) & 1, 200000000ull);
  } else if (FP8 && warp >= C::CONV && warp < C::S_WARP) {
    // ---------------------------------------------------------------- fp8: codes -> bf16 rows in the ring
    // Warp w converts the CTA's 32 keys of tiles w, w + kRing, ...: lane l looks up key l of the next tile
    // (offset, page) while this one is converted, eight rows at a time, a lane taking 16 codes (32 bytes
    // out) of each.  The first kRing tiles are spread instead, eight rows of four tiles a warp: the first
    // tile is there after one round of loads, not four (four selections of 2048: 30.8 -> 27.3 us).  The
    // loops stay rolled: the roles' code together has to stay in the instruction caches (all 32 rows
    // unrolled: 4826 us where this takes 1473).
    const uint32_t slot = warp - C::CONV;
    uint16_t* ring = a.ring + (static_cast<size_t>(grp * kRing) * kRows + 32 * rank) * kDqk;
    const uint32_t quarter = slot & 3, first = slot >> 2;      // spread: these rows of tiles first, first + 2, ...
    uint32_t my_row = 8 * quarter + (lane & 7), my_tile = first + 2 * (lane >> 3);
    Walk<SEL> aw(walk);
    Seg as;
    int ai = 0;
    bool alive = aw.next(as), ok = true;
    auto advance = [&](int by) {
      for (ai += by; alive && ai >= as.n;) {
        ai -= as.n;
        alive = aw.next(as);
      }
    };
    int j = -1, len = 0, page = -1;          // lane's key of the tile at ai
    auto find_offset = [&]() {
      j = -1;
      if (!alive) return;
      len = row_len(a.pg, as.row);
      const int s = (as.i0 + ai) * kRows + static_cast<int>(32 * rank + my_row);
      j = !SEL ? s : s < a.topk ? gload(a.idx + static_cast<size_t>(as.row) * a.topk + s) : -1;
    };
    auto find_page = [&]() {
      page = -1;
      if (j >= 0 && j < len)
        page = gload(a.pg.block_table + static_cast<size_t>(as.row) * a.pg.max_pages + (j >> kPageShift));
    };
    auto cache_row = [&]() -> int {          // -1: no key
      const bool in = static_cast<uint32_t>(page) < static_cast<uint32_t>(a.pg.n_pages);
      // a key on a page outside the cache, or a selected one past the end (the tile's tail is neither)
      if (!in && (SEL ? j >= 0 : j >= 0 && j < len && my_row == 0 && rank == 0)) report(sh.faults, DEV_ERR_BAD_INDEX);
      return in ? (page << kPageShift) + (j & (kPageRows - 1)) : -1;
    };
    const uint32_t n_tiles = a.stop_after >= 0 ? min(static_cast<uint32_t>(share), static_cast<uint32_t>(a.stop_after))
                                               : static_cast<uint32_t>(share);   // (test hook)
    advance(static_cast<int>(my_tile));
    find_offset();
    find_page();
    for (uint32_t lap = 0, t = slot; ok && (lap == 0 || t < n_tiles); t += kRing, ++lap) {
      const int at = cache_row();
      const uint32_t sc = gload(reinterpret_cast<const uint32_t*>(a.scale) + max(at, 0));
      advance(static_cast<int>(t + kRing - my_tile));
      my_tile = t + kRing;
      my_row = lane;
      find_offset();
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {
        const uint32_t at_tile = lap ? slot : first + 2 * q;
        if (lap == 0 && at_tile >= n_tiles) break;
        uint16_t* dst = ring + (at_tile * kRows + 8 * (lap ? q : quarter)) * kDqk;
        uint4 w[8], rope[2];
        int row[8], rr[2];
#pragma unroll
        for (int k = 0; k < 8; ++k) row[k] = __shfl_sync(0xffffffffu, at, 8 * q + k);
#pragma unroll
        for (int k = 0; k < 2; ++k) rr[k] = __shfl_sync(0xffffffffu, at, 8 * q + 4 * k + (lane >> 3));
        // (rows without a key read a row of the cache all the same: no branch around the loads)
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = gload_once(a.latent + static_cast<size_t>(max(row[k], 0)) * kDv + lane * 16);
#pragma unroll
        for (int k = 0; k < 2; ++k) rope[k] = gload_once(a.rope + static_cast<size_t>(max(rr[k], 0)) * 64 + (lane & 7) * 8);
        if (q == 0) {
          find_page();
          if (lap > 0 && !(ok = wait(&sh.ring_empty[slot], (lap - 1) & 1))) break;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t rsc = __shfl_sync(0xffffffffu, sc, 8 * q + k);
          const uint32_t m = row[k] >= 0 ? fp8_mult((rsc >> (8 * (lane >> 3))) & 0xFFu) : 0u;   // no key: times zero
          uint32_t o[8];
          fp8x4_to_bf16(w[k].x, m, o[0], o[1]);
          fp8x4_to_bf16(w[k].y, m, o[2], o[3]);
          fp8x4_to_bf16(w[k].z, m, o[4], o[5]);
          fp8x4_to_bf16(w[k].w, m, o[6], o[7]);
          stg256(dst + k * kDqk + lane * 16, o);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k)
          *reinterpret_cast<uint4*>(dst + (4 * k + (lane >> 3)) * kDqk + kDv + (lane & 7) * 8) =
              rr[k] >= 0 ? rope[k] : make_uint4(0, 0, 0, 0);
        if (lap == 0 || q == 3) {
          // the rows are visible to both CTAs' copies before they are told
          __threadfence();
          fence_proxy_async_global();
          __syncwarp();
          if (lane < 2) arrive_cta_n(&sh.ring_full[at_tile], lane, lap ? 4 : 1);
        }
      }
    }
  } else if (warp < kSW) {
    // ---------------------------------------------------------------- softmax + epilogue
    const int qd = warp & 3, cw = warp >> 2;
    const int head = (qd & 1) * 32 + lane;                       // of this CTA's 64
    const int kbase = (qd >> 1) * 32 + cw * kKT;               // this thread's keys of a tile
    const int part = (qd >> 1) * 2 + cw;
    const uint32_t t_lane = static_cast<uint32_t>(qd * 32) << 16;
    const int ghead = static_cast<int>(rank) * kHeads + head;
    constexpr uint32_t kAll = 0xFFFFu;
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
          const int s = i * kRows + kbase + (lane & (kKT - 1));
          const int j = s < a.topk ? gload(irow + s) : -1;
          bool v = j >= 0 && j < len;
          if (v) v = static_cast<uint32_t>(gload(bt + (j >> kPageShift))) < static_cast<uint32_t>(a.pg.n_pages);
          mask = __ballot_sync(0xffffffffu, v) & kAll;
        } else {
          const int nv = tile_rows(a, len, i, gload(bt + (i >> 1))) - kbase;
          mask = nv >= kKT ? kAll : nv <= 0 ? 0u : (1u << nv) - 1u;
        }
        bool ok = wait(&sh.s_full[sb], (g >> 1) & 1);
        float x[kKT];
        float mx = -INFINITY;
        if (ok) {
          tc_fence_after();
          uint32_t v[kKT];
          tmem_ld16(tmem + t_lane + kSCol + sb * 32 + cw * 16, v);
          tmem_ld_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_cta(&sh.s_empty[sb], 0);
          if (mask == kAll) {
#pragma unroll
            for (int c = 0; c < kKT; ++c) x[c] = __uint_as_float(v[c]) * a.scale_log2;
          } else {
#pragma unroll
            for (int c = 0; c < kKT; ++c) x[c] = (mask >> c) & 1u ? __uint_as_float(v[c]) * a.scale_log2 : -INFINITY;
          }
#pragma unroll
          for (int c = 0; c < kKT; ++c) mx = fmaxf(mx, x[c]);
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
            for (int b = 0; b < kOC / 16; ++b) {
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
        // P = 2^(s - m), rounded to bf16 (at most 2^-8 of each weight, no bias); the output is divided by
        // the sum of the rounded weights, the log-sum-exp takes the sum of the unrounded ones
        const float ms = m_used == -INFINITY ? 0.f : m_used;     // only masked entries so far: 2^(-inf - 0) = 0
        uint32_t pk[kKT / 2];
#pragma unroll
        for (int c = 0; c < kKT / 2; ++c) {
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
#pragma unroll
        for (int c = 0; c < kKT / 8; ++c)
          sts128(prow + (((kbase / 8 + c) ^ (head & 7)) << 4), pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_cta(&sh.p_full[sb], 0);
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
      const int dim0 = (qd >> 1) * 256 + cw * 128;               // this thread's OC dims
      const size_t pslot = static_cast<size_t>(grp) * 2 + (sg.i0 > 0 ? 0 : 1);
      const float inv = l == 0.f ? 0.f : 1.f / l;                // a NaN sum stays NaN; no key: zeros
      uint16_t* orow = a.out + (static_cast<size_t>(sg.row) * a.H + ghead) * kDv + dim0;
      float* prow = a.part_o + (pslot * a.H + ghead) * kDv + dim0;
#pragma unroll 1
      for (int b = 0; b < kOC / 32; ++b) {
        uint32_t o[32];
        tmem_ld32(tmem + t_lane + cw * 128 + b * 32, o);
        tmem_ld_wait();
        if (ghead >= a.H) continue;
        // a lane's dims are 32-byte pieces of its head's row
        if (sg.whole) {
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            uint32_t w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const __nv_bfloat162 ob = __floats2bfloat162_rn(__uint_as_float(o[16 * v + 2 * e]) * inv,
                                                              __uint_as_float(o[16 * v + 2 * e + 1]) * inv);
              w[e] = *reinterpret_cast<const uint32_t*>(&ob);
            }
            // (out is 16-byte aligned)
            reinterpret_cast<uint4*>(orow + b * 32)[2 * v] = make_uint4(w[0], w[1], w[2], w[3]);
            reinterpret_cast<uint4*>(orow + b * 32)[2 * v + 1] = make_uint4(w[4], w[5], w[6], w[7]);
          }
        } else {
#pragma unroll
          for (int v = 0; v < 4; ++v) stg256(prow + b * 32 + 8 * v, o + 8 * v);
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
      if (lane == 0) arrive_cta(&sh.o_free, 0);
    }
  } else if (rank != 0) {
    // ---------------------------------------------------------------- the peer: tell the leader of its Q
    if (warp == C::S_WARP) {
      uint32_t it = 0;
      while (walk.next(sg)) {
        if (!load_q(it)) break;
        if (lane == 0) arrive_cta(&sh.q_ready, 0);
        ++it;
      }
    }
  } else {
    // ---------------------------------------------------------------- MMA issuers
    constexpr uint32_t id_qk = idesc_bf16_f32(128, kRows, 0, 0);
    constexpr uint32_t id_pv = idesc_bf16_f32(128, 256, 0, 1);
    uint32_t g = 0, it = 0;
    bool ok = true;
    const uint64_t dq = sdesc_sw128(smem_u32(sQ), 16, 1024);
    while (ok && walk.next(sg)) {
      if (warp == C::S_WARP) {
        ok = load_q(it) && wait(&sh.q_ready, it & 1);
        for (int n = 0; n < sg.n && ok; ++n, ++g) {
          const int sb = g & 1;
          if (g >= 2 && !(ok = wait(&sh.s_empty[sb], ((g >> 1) - 1) & 1))) break;
          if (!(ok = wait(&sh.ready_s[sb], (g >> 1) & 1))) break;
          tc_fence_after();
          const uint64_t dk = sdesc_sw128(smem_u32(smem + kOffStage + sb * kStage), 16, 1024);
          // (fp8: rolled -- 36 products in line, behind the other roles' code, came out of the instruction cache
          // too slowly for the tensor core: 1913 us where the loop takes 1473)
#pragma unroll FP8 ? 1 : kKB
          for (int kb = 0; kb < kKB; ++kb)
            umma_pair_x4_elect<2, 2>(tmem + kSCol + sb * 32, dq + static_cast<uint64_t>((kb * kHeads * 128) >> 4),
                                     dk + static_cast<uint64_t>((kb * kSBlk) >> 4), id_qk, kb ? 1u : 0u);
          commit_pair_elect(&sh.s_full[sb]);
        }
        if (ok && walk.left > 0) commit_pair_elect(&sh.q_empty);
      } else {
        for (int n = 0; n < sg.n && ok; ++n, ++g) {
          const int sb = g & 1;
          ok = wait(&sh.ready_v[sb], (g >> 1) & 1) && wait(&sh.p_full[sb], (g >> 1) & 1);
          if (ok && n == 0 && it > 0) ok = wait(&sh.o_free, (it - 1) & 1);
          if (!ok) break;
          tc_fence_after();
          const uint64_t dp = sdesc_sw128(smem_u32(smem + kOffP + sb * kPBytes), 16, 1024);
          const uint64_t dv = sdesc_sw128(smem_u32(smem + kOffStage + sb * kStage + kSBytes), kVBlk, 1024);
#pragma unroll FP8 ? 1 : 2
          for (int h = 0; h < 2; ++h)
            umma_pair_x4_elect<2, 128>(tmem + h * 128, dp, dv + static_cast<uint64_t>((2 * h * kVBlk) >> 4), id_pv,
                                       n > 0 ? 1u : 0u);
          commit_pair_elect(&sh.o_done[sb]);
        }
      }
      ++it;
    }
    // every product this warp issued has completed before TMEM is released
    commit_pair_elect(&sh.mma_done);
    mbar_drain(&sh.mma_done, 0, 200000000ull);
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0) publish_faults(a, sh.faults);
  cluster_sync_all();                    // no thread of either CTA signals, reads or is read any more
  // The leader has issued every commit and seen its own copy of mma_done.  The peer's shared memory may only be
  // given up when its copy is there too: both issuing warps' last commit, behind all others of theirs.
  if (rank != 0 && threadIdx.x == 0) mbar_drain(&sh.mma_done, 0, 200000000ull);
  tc_fence_after();
  if (warp == C::PV_WARP) tmem_dealloc_pair(tmem, kTmemCols);
}

template <bool FP8, bool SEL>
cudaError_t launch_t(const CUtensorMap& ts, const CUtensorMap& tv, const CUtensorMap& tq, const LArgs& a, cudaStream_t st) {
  cudaError_t e = smem_attr_once<latent_pair_kernel<FP8, SEL>>(kDynSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(latent_pair_kernel<FP8, SEL>, dim3(a.n_cta), PCfg<FP8>::THREADS, kDynSmem, st, 2, ts, tv, tq, a);
}

}  // namespace

cudaError_t launch_latent_pair(bool fp8, bool sel, const CUtensorMap& tmap_s, const CUtensorMap& tmap_v,
                               const CUtensorMap& tmap_q, const LArgs& a, cudaStream_t st) {
  if (!fp8) return launch_t<false, false>(tmap_s, tmap_v, tmap_q, a, st);
  return sel ? launch_t<true, true>(tmap_s, tmap_v, tmap_q, a, st) : launch_t<true, false>(tmap_s, tmap_v, tmap_q, a, st);
}

}  // namespace dsa
