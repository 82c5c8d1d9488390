// Shared by the latent attention kernels: arguments, the split of the work over the cache's length,
// and small helpers.
#pragma once

#include <cuda_bf16.h>

#include "fp8.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace dsa {

constexpr int kRows = 64;              // latent rows per tile
constexpr int kDqk = 576;
constexpr int kDv = 512;
constexpr int kKB = kDqk / 64;         // 64-dim blocks per row
// A share holds at least this many tiles, four where two would leave the rows in more than 64 partials each.
// One row of 1000, 8000, 12000, 20000 keys, 16 heads: 13.6, 14.8, 16.7, 20.8 us with shares of two or more,
// 15.6, 16.8, 16.8, 18.8 with four; eight rows of 2500: 16.7 and 18.7; 4000 keys, 64 heads, fp8: 20.9 and 22.9.
constexpr int kMinTiles = 2;
constexpr int kMostGroups = 160;       // groups of CTAs (the join holds five per lane)
__device__ __forceinline__ int min_share(long long total, int n_q) { return total > 128LL * n_q ? 4 : kMinTiles; }
// The first tile of group g's share, g <= groups <= kMostGroups: total * g / groups, to the nearest 2^s tiles
// below where that passes 32 bits (a 64-bit division takes hundreds of cycles on every call's way).
__device__ __forceinline__ long long share_start(long long total, int g, int groups) {
  if (g == groups) return total;
  const int s = max(0, 40 - __clzll(total));           // total >> s < 2^24
  return static_cast<long long>(static_cast<uint32_t>(total >> s) * static_cast<uint32_t>(g) / static_cast<uint32_t>(groups))
         << s;
}

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ bool bar_or(uint32_t id, uint32_t n, bool p) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred pi, po;\n setp.ne.u32 pi, %1, 0;\n bar.red.or.pred po, %2, %3, pi;\n selp.u32 %0, 1, 0, po;\n}\n"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(p)), "r"(id), "r"(n)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void sts32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
// gload of what is read once.
__device__ __forceinline__ uint4 gload_once(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ void stg256(void* p, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
// One thread of the warp, the same each time.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n selp.u32 %0, 1, 0, e;\n}\n" : "=r"(one));
  return one != 0;
}
// A shared-memory matrix descriptor's low word; the high word (sdesc_sw128's, SBO = 1024) is the same for all.
constexpr uint32_t kDescHi = 0x40004040u;
__device__ __forceinline__ uint32_t sdesc_lo(uint32_t saddr, uint32_t lbo_bytes) {
  return ((saddr & 0x3FFFFu) >> 4) | ((lbo_bytes >> 4) << 16);
}
// x, as a value the compiler cannot carry around a loop (addresses derived from it are formed where they
// are used instead of being held in registers).
__device__ __forceinline__ uint32_t opaque(uint32_t x) {
  uint32_t y;
  asm volatile("mov.u32 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void lrow16(float (&r)[16], const float* p) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 v = *reinterpret_cast<const float4*>(p + 4 * i);
    r[4 * i] = v.x;
    r[4 * i + 1] = v.y;
    r[4 * i + 2] = v.z;
    r[4 * i + 3] = v.w;
  }
}

// What a row of the line is: a query row with every key of its sequence, or with its selected ones; an item of a
// shared-prefix call (latent_shared.cu): some columns, (row, head) pairs that follow one another in q, over some
// tiles of one row's table; a query row whose keys' weights are wanted.
enum WalkMode : int { kEvery = 0, kSelected = 1, kItems = 2, kWeights = 3 };

// An item: {first column, columns | flags, table row, first tile}.
constexpr int kItemSole = 1 << 16;     // nothing else adds to its columns
constexpr int kItemOwn = 1 << 17;      // a row's own keys (clear: a group's prefix)

struct LArgs {
  const uint8_t* latent;       // bf16 rows (unused by the kernel: TMA), or e4m3 codes
  const uint8_t* scale;
  const uint16_t* rope;
  const int32_t* idx;          // selected offsets [n_q][topk], or nullptr
  const int32_t* row_nt;       // selected keys: 64-slot tiles of each row; items: tiles of each
  const int4* items;           // kItems
  const int4* shares;          // kItems: {first item, its first tile, tiles} of each group
  float* whole_o;              // kItems: an item that one share holds, by column: [prefix, own][n_q * H][512]
  float4* whole_m;             // [prefix, own][n_q * H]: a column's {max in use, rounded, plain sum} (as part_m)
  float4* item_m;              // [n_grp * 2][part_cols]: the same of partials
  int2* pieces;                // kItems: the first group of each item, and the one behind its last
  PagedRows pg;
  uint16_t* out;
  float* lse;
  int n_q, H, topk, n_grp, n_hb;
  float scale_log2;
  int2* start;                 // [n_grp]: (row, tile) each group starts at; groups without a share: row INT_MAX
  uint16_t* ring;              // fp8, CTA pairs: [n_grp][kRing][64][576] bf16
  float* part_o;               // [n_grp * 2][H][512]        (kItems: part_cols columns for H)
  float* part_m;               // [3][n_grp * 2][H]: max in use (log2), sum of the rounded weights, plain sum
  int part_cols;
  const float* lse_in;         // kWeights: [n_q][H]
  const float* w_in;           // [n_q] rows w_stride apart; nullptr: zeros
  float* w_out;
  long long w_stride;
  const int32_t* group_start;  // groups of rows that the call names without sharing anything (latent_shared.cu):
  const int32_t* prefix_len;   // the join checks them; nullptr: none
  int n_groups;
  uint32_t* status;
  uint32_t* err;               // [CTAs][2]: error bits, bad-index count
  int n_cta;
  unsigned long long wait_ns;
  int stop_after;
};

__device__ __forceinline__ int row_len(const PagedRows& pg, int row) {
  return max(0, min(gload(pg.seq_len + row), pg.max_pages << kPageShift));
}
template <int MODE>
__device__ __forceinline__ int row_tiles(const LArgs& a, int row) {
  if constexpr (MODE == kSelected || MODE == kItems) return gload(a.row_nt + row);
  return (row_len(a.pg, row) + kRows - 1) / kRows;
}

// Splitting rows evenly costs writing and joining partials; a CTA pair per row costs the tiles that the
// longest row has above the even share.  128 heads, 64 rows of 8 selected tiles over 76 pairs: 54.8 us
// split, 40.9 whole; of 32 tiles, 87.8 and 78.6; 48 rows of 32 (12 above the share), 76.8 and 75.3; 20 rows
// of 16 (12 above it), 41.9 and 46.4.  Up to 8 extra tiles are taken at 76 pairs, where all of this was
// measured; 12 gain or lose with the rows' length.  Fewer groups, whose partials are fewer, take fewer in
// proportion (not measured).  Single CTAs, whose partials are smaller, gain nothing (64 heads, 128 rows of 32:
// 112 and 118).  Extra tiles that are taken:
__device__ __forceinline__ int whole_row_extra(int groups) { return groups / 9; }

// The segments (consecutive tiles of one row) of this CTA's share, in order.
struct Seg {
  int row, i0, n;    // row: of the block table; i0: its tile
  bool begins;       // with the row's first tile
  bool whole;        // the row's every tile
  int col0, ncol;    // columns of q and out; kItems: ncol with the item's flags
  int item;          // kItems
  bool ends;         // kItems: with the item's last tile
};
template <int MODE>
struct Walk {
  const LArgs& a;
  int row, tile;
  long long left;
  __device__ __forceinline__ Walk(const LArgs& args, int r, int t, long long n) : a(args), row(r), tile(t), left(n) {}
  __device__ __forceinline__ bool next(Seg& s) {
    if (left <= 0) return false;
    int T = row_tiles<MODE>(a, row);
#pragma unroll 1
    while (T == 0) T = row_tiles<MODE>(a, ++row);
    s.row = row;
    s.i0 = tile;
    s.n = static_cast<int>(min(static_cast<long long>(T - tile), left));
    s.begins = tile == 0;
    s.whole = tile == 0 && s.n == T;
    if constexpr (MODE == kItems) {
      const int4 it = gload(a.items + row);
      s.col0 = it.x;
      s.ncol = it.y;
      s.item = row;
      s.ends = tile + s.n == T;
      s.row = it.z;
      s.i0 += it.w;
    } else {
      s.col0 = row * a.H;
      s.ncol = a.H;
    }
    left -= s.n;
    ++row;
    tile = 0;
    return true;
  }
};
// Keys of the row that a segment belongs to.  (A prefix's item has whole tiles, and no length of its own.)
template <int MODE>
__device__ __forceinline__ int seg_len(const LArgs& a, const Seg& s) {
  if (MODE == kItems && !(s.ncol & kItemOwn)) return 0x7FFFFFFF;
  return row_len(a.pg, s.row);
}
// Where a segment's unnormalised columns go: the first's row of O, and (column c) its three numbers.
template <int MODE>
struct Partial {
  float* o;
  float* m;
  size_t step;
  __device__ __forceinline__ Partial(const LArgs& a, const Seg& s, int grp) {
    const int cols = MODE == kItems ? a.part_cols : a.H;
    const size_t slot = static_cast<size_t>(grp) * 2 + (s.begins ? 1 : 0);
    o = a.part_o + slot * cols * kDv;
    if constexpr (MODE == kItems) {
      m = reinterpret_cast<float*>(a.item_m + slot * cols);
      if (s.whole) {
        const size_t at = (s.ncol & kItemOwn ? static_cast<size_t>(a.n_q) * a.H : 0) + s.col0;
        o = a.whole_o + at * kDv;
        m = reinterpret_cast<float*>(a.whole_m + at);
      }
    } else {
      m = a.part_m + slot * cols;
      step = static_cast<size_t>(a.n_grp) * 2 * cols;
    }
  }
  __device__ __forceinline__ void sums(int c, float max, float rounded, float plain) const {
    if constexpr (MODE == kItems) {
      reinterpret_cast<float4*>(m)[c] = make_float4(max, rounded, plain, 0.f);
    } else {
      m[c] = max;
      m[step + c] = rounded;
      m[2 * step + c] = plain;
    }
  }
};
// (one thread of a group, for each of its segments)
template <int MODE>
__device__ __forceinline__ void note_piece(const LArgs& a, const Seg& s, int grp) {
  if constexpr (MODE == kItems) {
    if (s.begins) a.pieces[s.item].x = grp;
    if (s.ends) a.pieces[s.item].y = grp + 1;
  }
}
template <int MODE>
__device__ __forceinline__ bool writes_out(const Seg& s) {
  return s.whole && (MODE != kItems || (s.ncol & kItemSole));
}
template <int MODE>
__device__ __forceinline__ int columns(const Seg& s) {
  return MODE == kItems ? s.ncol & 0xFFFF : s.ncol;
}

// Error bits of entry g of n_groups groups of rows, g <= n_groups: starts ascending within [0, n_q], no prefix below 0.
__device__ __forceinline__ uint32_t group_errors(const int32_t* start, const int32_t* prefix, int n_groups, int n_q, int g) {
  // (the loads side by side)
  const bool last = g == n_groups;
  const int s = gload(start + g), next = last ? s : gload(start + g + 1), len = last ? 0 : gload(prefix + g);
  return s < 0 || s > n_q || next < s || len < 0 ? DEV_ERR_RANGE : 0u;
}

// Faults are collected per CTA; the CTAs' words are put together by the join kernel (or, when
// there is one CTA, written as they are), so no clearing pass runs before the kernel.
struct CtaFaults {
  uint32_t bits, count;
};
__device__ __forceinline__ void report(CtaFaults& f, uint32_t bits) {
  atomicOr(&f.bits, bits);
  atomicAdd(&f.count, 1u);
}
template <int MODE>
__device__ __forceinline__ void publish_faults(const LArgs& a, const CtaFaults& f) {
  uint32_t* w = MODE != kItems && gridDim.x == 1 ? a.status : a.err + 2 * blockIdx.x;
  w[0] = f.bits;
  w[1] = f.count;
}

// The share of group `grp` (of items: as it was listed): a scan over the rows' tile counts (the whole block calls it;
// a block-wide barrier is needed behind it before row0 / tile0 are read).
struct Share {
  long long wsum[32];
  int wmax[32];
  int row0, tile0;
};
// Groups in use, and whether they take a row each.
template <int MODE>
__device__ __forceinline__ int share_groups(int n_grp, int n_hb, int n_rows, long long total, int tallest, bool& by_row) {
  const long long most = min_share(total, n_rows) == 4 ? (total + 3) >> 2 : (total + 1) >> 1;
  const int groups = static_cast<int>(min(static_cast<long long>(n_grp), most));
  by_row = MODE != kWeights && n_hb == 2 && n_rows <= n_grp &&
           tallest <= share_start(total, 1, max(groups, 1)) + whole_row_extra(groups);
  return by_row ? n_rows : groups;
}
__device__ __forceinline__ bool bad_length(const PagedRows& pg, int row) {
  const int want = gload(pg.seq_len + row);
  return want < 0 || want > (pg.max_pages << kPageShift);
}
template <int MODE, int THREADS>
__device__ __forceinline__ long long find_share(const LArgs& a, int grp, bool writes_start, Share& sh, CtaFaults& faults) {
  if constexpr (MODE == kItems) {
    const int4 r = gload(a.shares + grp);
    if (threadIdx.x == 0) {
      sh.row0 = r.x;
      sh.tile0 = r.y;
    }
    return r.z;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  long long share = 0;
  int groups;
  if (a.n_q <= 32) {
    // A row a lane, each warp for itself: no barrier, no trip through shared memory (300 keys, 16 heads: 11.6 ->
    // 10.8 us).
    const int T = lane < a.n_q ? row_tiles<MODE>(a, lane) : 0;
    const uint32_t total = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(T));     // 32 x 2^25 at most
    bool by_row;
    groups = share_groups<MODE>(a.n_grp, a.n_hb, a.n_q, total, __reduce_max_sync(0xffffffffu, T), by_row);
    uint32_t pre = T;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, pre, o);
      if (lane >= o) pre += v;
    }
    pre -= T;
    int row0 = grp, tile0 = 0;
    if (grp < groups) {
      if (by_row) {
        share = __shfl_sync(0xffffffffu, T, grp);
      } else {
        const uint32_t first = static_cast<uint32_t>(share_start(total, grp, groups));
        share = share_start(total, grp + 1, groups) - first;
        row0 = __ffs(static_cast<int>(__ballot_sync(0xffffffffu, pre <= first && first < pre + T))) - 1;
        tile0 = static_cast<int>(first - __shfl_sync(0xffffffffu, pre, row0));
      }
    }
    if (threadIdx.x == 0) {
      sh.row0 = row0;
      sh.tile0 = tile0;
      if (writes_start && grp < groups) a.start[grp] = make_int2(row0, tile0);
    }
    if (blockIdx.x == 0 && warp == 0) {
      __syncwarp();        // (thread 0 has set faults)
      if (lane < a.n_q && bad_length(a.pg, lane)) report(faults, DEV_ERR_RANGE);
    }
  } else {
    const int per = (a.n_q + THREADS - 1) / THREADS;
    const int ra = min(a.n_q, static_cast<int>(threadIdx.x) * per), rb = min(a.n_q, ra + per);
    long long mine = 0;
    int tallest = 0;
    bool bad_len = false;
#pragma unroll 1
    for (int r = ra; r < rb; ++r) {
      const int T = row_tiles<MODE>(a, r);
      mine += T;
      tallest = max(tallest, T);
      if (blockIdx.x == 0 && bad_length(a.pg, r)) bad_len = true;
    }
    long long pre = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, pre, o);
      if (lane >= o) pre += v;
    }
    if (lane == 31) sh.wsum[warp] = pre;
    tallest = __reduce_max_sync(0xffffffffu, tallest);
    if (lane == 0) sh.wmax[warp] = tallest;
    __syncthreads();
    if (bad_len) report(faults, DEV_ERR_RANGE);
    long long total = 0;
    pre -= mine;
#pragma unroll 1
    for (int w = 0; w < THREADS / 32; ++w) {
      if (w < warp) pre += sh.wsum[w];
      total += sh.wsum[w];
      tallest = max(tallest, sh.wmax[w]);
    }
    bool by_row;
    groups = share_groups<MODE>(a.n_grp, a.n_hb, a.n_q, total, tallest, by_row);
    if (by_row) {
      share = grp < groups ? row_tiles<MODE>(a, grp) : 0;
      if (threadIdx.x == 0 && grp < groups) {
        sh.row0 = grp;
        sh.tile0 = 0;
        if (writes_start) a.start[grp] = make_int2(grp, 0);
      }
    } else {
      const long long first = grp < groups ? share_start(total, grp, groups) : 0;
      share = grp < groups ? share_start(total, grp + 1, groups) - first : 0;
      if (share > 0 && pre <= first && first < pre + mine) {
        long long at = pre;
        int r = ra;
        while (true) {
          const int T = row_tiles<MODE>(a, r);
          if (first < at + T) break;
          at += T;
          ++r;
        }
        sh.row0 = r;
        sh.tile0 = static_cast<int>(first - at);
        if (writes_start) a.start[grp] = make_int2(r, static_cast<int>(first - at));
      }
    }
  }
  if (writes_start && threadIdx.x == 0 && grp >= groups) a.start[grp] = make_int2(0x7FFFFFFF, 0);
  // rows without keys: zeros and -inf
  if constexpr (MODE != kWeights) {
#pragma unroll 1
    for (int t = blockIdx.x; t < a.n_q; t += gridDim.x) {
      if (row_tiles<MODE>(a, t) != 0) continue;
      uint4* o = reinterpret_cast<uint4*>(a.out + static_cast<size_t>(t) * a.H * kDv);
#pragma unroll 1
      for (int e = threadIdx.x; e < a.H * (kDv / 8); e += THREADS) o[e] = make_uint4(0, 0, 0, 0);
      if (a.lse)
        for (int h = threadIdx.x; h < a.H; h += THREADS) a.lse[static_cast<size_t>(t) * a.H + h] = -INFINITY;
    }
  }
  return share;
}

// Bounded mbarrier wait, as mbar_wait_for, but out of line behind the first try: the warp roles' code
// together has to stay in the instruction caches, and the waits are most of its copies.
static __device__ __noinline__ bool wait_more(uint64_t* bar, uint32_t parity, volatile uint32_t* abort_flag, uint32_t* bits,
                                       unsigned long long limit_ns) {
  const uint64_t t0 = globaltimer_ns();
  while (true) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (globaltimer_ns() - t0 > limit_ns) {
      *abort_flag = 1u;
      atomicOr(bits, DEV_ERR_TIMEOUT);
      return false;
    }
  }
}
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile uint32_t* abort_flag, uint32_t* bits,
                                         unsigned long long limit_ns) {
  return mbar_try_wait(bar, parity) || wait_more(bar, parity, abort_flag, bits, limit_ns);
}

// Valid rows of tile i of a row of `len` keys: none on a page outside the cache.
__device__ __forceinline__ int tile_rows(const LArgs& a, int len, int i, int page) {
  if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(a.pg.n_pages)) return 0;
  return max(0, min(kRows, len - i * kRows));
}

// Columns of a CTA of the kernel for up to 64 heads.
inline int head_block(int n_heads) { return n_heads <= 16 ? 16 : n_heads <= 32 ? 32 : 64; }
// That kernel, with hb columns a CTA (latent_attn.cu).  tmap_kv / tmap_v: a bf16 cache in boxes {64, 64, 1}
// and {64, 64, 4}.
cudaError_t launch_latent_single(int hb, bool fp8, int mode, const CUtensorMap& tmap_kv, const CUtensorMap& tmap_v,
                                 const CUtensorMap& tmap_q, const LArgs& a, cudaStream_t st);

// The CTA-pair kernel for 65 .. 128 heads (latent_pair.cu).  tmap_s / tmap_v: a bf16 cache in boxes
// {64, 32, 9} and {64, 64, 4}.
cudaError_t launch_latent_pair(bool fp8, int mode, const CUtensorMap& tmap_s, const CUtensorMap& tmap_v,
                               const CUtensorMap& tmap_q, const LArgs& a, cudaStream_t st);

}  // namespace dsa
