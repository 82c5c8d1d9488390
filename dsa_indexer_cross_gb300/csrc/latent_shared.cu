// Latent attention of query rows that share a prefix (a batch behind one system prompt, drafts of one
// sequence): the prefix's tiles are walked once for all heads of all rows of a group.
//
//   o[t, h] = sum over j of the group's prefix and of the row's own keys, softmax over both together
//
// In the latent cache every head reads the same rows, so a group's (row, head) pairs are all columns of one
// product with the prefix: 64 rows of 16 heads are 1024 columns, where the walk of one row by itself fills 16
// and is bound by the rows' bytes.  The kernels are those of dsa_latent_attn_paged (latent_attn.cu,
// latent_pair.cu); what differs is the line of tiles that is cut into shares.  It holds items: some columns
// (consecutive (row, head) pairs of q) and some tiles of one block-table row.  A group of rows gives one item
// per block of columns over its prefix's whole tiles of 64 keys, each row one item over the rest of its keys.  The
// lengths are device data, so a kernel of one block lists the items first.
//
// Which kernel.  Up to 64 columns a group: one launch of the single-CTA kernel takes every item.  More than 64
// heads: one launch of the CTA-pair kernel (128 columns).  In between two launches, the pair kernel for the
// prefixes, the single-CTA one for the rows' own keys, which are bound by bytes; where these are few, the pair
// kernel takes them too and the second launch finds nothing.
//
// Staging (fp8).  A walk converts a prefix's codes once for each block of 128 columns.  Where there are many
// blocks, the prefixes are first brought to bf16 once, in pages of the workspace that stay mostly in L2, and the
// pair kernel takes them from there as from a bf16 cache, in a walk of its own.
//
// The line counts an item as a few tiles more than it has, for what it costs by itself (32 rows of 64 heads
// behind 100K keys, fp8, one walk: the pairs at the line's end had sixteen short items each; 599 -> 525 us).
//
// A column's result comes from its prefix item and its own item, each whole or in partials where shares were
// cut: latent_shared_join_kernel puts them together with one softmax.  A row that is the only thing its columns
// come from is written by the walk itself.
//
// What bounds it.  32 rows of 64 heads behind 100K keys, fp8, 340 us (the unshared call 640): some 250 of them the staged
// walk, 1.8 PFLOP/s (latent_pair.cu); 22 staging; 24 own keys; the rest list and join.  37 rows of 128 heads behind four
// documents, 262 us (318): the staged walk, 45 own keys, 22 staging.  48 rows of 16 heads behind 8000 keys, bf16, 39 us (58): 18
// tiles a pair, some 24 us with fill and segments' ends, the list 5, the join 7.  Small calls: launches and loads one behind
// the other, so those that gain nothing are not shared.
//
// A group is walked by rows, not shared, where that takes no more items (128 heads, or few rows of more than 64) and
// nothing is staged; calls that can have no other group run the unshared kernels, as those too small to gain do.
#include <cuda_bf16.h>

#include <algorithm>

#include "latent_attn.cuh"

namespace dsa {
namespace {

// A prefix of fewer tiles than this is left to the rows.
constexpr int kMinShared = 2;
// What an item costs apart from its tiles, in tiles: its columns of q are loaded and its sums written while the
// products wait.  A pair takes a tile of bf16 rows in less time.  3, 4, 6, 8 tiles: 48 rows of 64 heads behind 8000 keys with
// 50..150 of their own, bf16, 83, 76, 64, 62 us; 40 groups of 5 behind 5000..8000, 191, 166, 141, 139; the same of 16 heads, fp8,
// 124, 126, 132, 137.
constexpr int kItemCost = 3, kItemCostPairBf16 = 6;

// Up to this many tiles of the rows' own keys go with the prefixes through the pair kernel, which a second walk's
// launch, fill and partials cost more than: 48 rows behind 8000 keys, own tiles 266, 811, 2121, 5916, 22575: bf16, 16 heads,
// one walk 36, 42, 56, 102, 305 us, two 46, 54, 72, 114, 285.  fp8 where nothing is staged: 16 rows of 16 heads, own
// tiles 16, 802, 3231: 34, 51, 95 and 41, 50, 76; 8 rows of 64 heads, 348, 1404: 37, 70 and 37, 79.
constexpr int kMostOwnBf16 = 12000, kMostOwnFp8 = 1500;

// Calls of up to this many tiles, as the table's width allows, share nothing: listing the items and joining them costs
// more.  Drafts of one sequence, 16 heads, bf16, rows x keys: 4 x 5000 (320 tiles) 19.5 us shared, 13.9 alone; 8 x 8000
// (1008) 25.0 and 17.7; 16 x 8000 (2016) 25.9 and 25.1; 48 x 8000 and more (7000) 39 and 58.
constexpr int kAloneTiles = 2000;

// Staging: prefixes of up to this many pages in all (151 MB), walked by this many blocks of columns each and more, on
// average.  A tile costs some 0.02 us to stage, its walks 0.005 us more each where they convert.
constexpr int kStagePages = 1024, kStageBlocks = 6, kStageTiles = 64;
constexpr int kStageParts = 4;         // of a page, a block each

struct PlanArgs {
  const int32_t* start;      // [n_groups + 1]
  const int32_t* prefix;     // [n_groups]
  PagedRows pg;
  int n_groups, n_q, H, cols;     // cols: columns of a prefix item
  bool two;                  // there is a second walk, for own items of more than most_own tiles in all
  int most_own;
  int32_t* tiles;            // [n_groups]: the shared tiles
  int32_t* table;            // [n_groups]: the row whose table names their pages
  int32_t* base;             // [n_groups]: first item, and the line before it
  long long* base_at;
  int32_t* nt[3];            // by list: 0 prefixes (and own items), 1 own items, 2 staged prefixes
  int4* items[3];
  int4* rows;                // [n_q]: first prefix item (-1), its first column, own item (-1), and the lists: of the
                             // own item + 4 that of the prefix item
  long long* at[3];          // the line before each item
  int4* shares[3];           // [n_grp]
  int n_grp[3];
  bool pair[3];
  int cost[3];               // what an item costs, in tiles
  uint32_t* faults;          // [2]
  int stage_pages;           // room for staged pages, 0: none
  int32_t* stage_at;         // [n_groups + 1]: first staged page of each group, then their number
};

struct Count {
  int items;
  long long line;
};
// Exclusive sums over the block's threads, and the totals.
template <int kPlanThreads>
__device__ __forceinline__ Count block_excl(Count x, Count* warp_sum, Count& total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const auto incl = [&](Count c) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int i = __shfl_up_sync(0xffffffffu, c.items, o);
      const long long t = __shfl_up_sync(0xffffffffu, c.line, o);
      if (lane >= o) {
        c.items += i;
        c.line += t;
      }
    }
    return c;
  };
  const Count mine = incl(x);
  __syncthreads();
  if (lane == 31) warp_sum[warp] = mine;
  __syncthreads();
  const Count w = lane < kPlanThreads / 32 ? warp_sum[lane] : Count{0, 0}, all = incl(w);
  total = Count{__shfl_sync(0xffffffffu, all.items, 31), __shfl_sync(0xffffffffu, all.line, 31)};
  return Count{__shfl_sync(0xffffffffu, all.items - w.items, warp) + mine.items - x.items,
               __shfl_sync(0xffffffffu, all.line - w.line, warp) + mine.line - x.line};
}
// The last of the n ascending values at v that is <= x; v[0] <= x.
template <typename T>
__device__ __forceinline__ int last_not_above(const T* v, int n, T x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (gload(v + mid) <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

template <int kPlanThreads>
__global__ void __launch_bounds__(kPlanThreads) latent_plan_kernel(const __grid_constant__ PlanArgs p) {
  __shared__ Count warp_sum[32];
  __shared__ CtaFaults faults;
  __shared__ int tallest[3];
  __shared__ unsigned long long stage_sum[3];      // pages, tiles, and tiles times blocks
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  grid_trigger();
  if (tid == 0) {
    faults.bits = faults.count = tallest[0] = tallest[1] = tallest[2] = 0;
    stage_sum[0] = stage_sum[1] = stage_sum[2] = 0;
  }
  grid_wait();
  // groups that do not lie in order within the rows, or a prefix of less than no key: none is shared (a call without
  // groups does not get here, and may have no arrays of them)
  bool bad = false;
  for (int g = tid; p.n_groups > 0 && g <= p.n_groups; g += kPlanThreads)
    if (group_errors(p.start, p.prefix, p.n_groups, p.n_q, g)) {
      bad = true;
      report(faults, DEV_ERR_RANGE);
    }
  bad = __syncthreads_or(bad);
  const int n_groups = bad ? 0 : p.n_groups;
  // A group's longest row, and its second longest, whose keys bound what is shared: a warp a group, or eight lanes
  // where there are more groups than warps.
  const int lanes = n_groups > kPlanThreads / 32 ? 8 : 32, sub = lane & (lanes - 1);
  for (int g0 = warp * (32 / lanes); g0 < n_groups; g0 += kPlanThreads / lanes) {
    const int g = g0 + lane / lanes;
    int n = 0, want = 0, longest = -1, second = -1, at = 0x7FFFFFFF;
    if (g < n_groups) {
      const int s = gload(p.start + g);
      n = gload(p.start + g + 1) - s;
      want = gload(p.prefix + g);
      for (int r = sub; r < n; r += lanes) {
        const int len = row_len(p.pg, s + r);
        second = max(second, min(len, longest));
        if (len > longest) {
          longest = len;
          at = s + r;
        }
      }
    }
    __syncwarp();
    for (int o = lanes >> 1; o > 0; o >>= 1) {
      const int l = __shfl_xor_sync(0xffffffffu, longest, o), r = __shfl_xor_sync(0xffffffffu, at, o);
      second = max(max(second, __shfl_xor_sync(0xffffffffu, second, o)), min(longest, l));
      if (l > longest || (l == longest && r < at)) {
        longest = l;
        at = r;
      }
    }
    if (sub == 0 && g < n_groups) {
      const long long blocks = (static_cast<long long>(n) * p.H + p.cols - 1) / p.cols;
      int tiles = min(want, max(second, 0)) / kRows;
      if (n < 2 || tiles < kMinShared || blocks > n) tiles = 0;
      const bool only_staged = blocks >= n;
      if (only_staged && (p.stage_pages == 0 || blocks < kStageBlocks)) tiles = 0;
      if (tiles > 0 && p.stage_pages > 0) {
        atomicAdd(&stage_sum[0], static_cast<unsigned long long>((tiles + 1) >> 1));
        atomicAdd(&stage_sum[1], static_cast<unsigned long long>(tiles));
        atomicAdd(&stage_sum[2], static_cast<unsigned long long>(tiles * blocks));
      }
      p.tiles[g] = only_staged ? -tiles : tiles;
      p.table[g] = at;
    }
  }
  __syncthreads();
  const bool staged = p.stage_pages > 0 && stage_sum[0] <= static_cast<unsigned long long>(p.stage_pages) &&
                      stage_sum[1] >= kStageTiles && stage_sum[2] >= kStageBlocks * stage_sum[1];
  if (p.stage_pages > 0) {
    // the tiles that are shared after all, and their pages
    int pages = 0;
    for (int g0 = 0; g0 < n_groups; g0 += kPlanThreads) {
      const int g = g0 + tid;
      int tiles = g < n_groups ? p.tiles[g] : 0;
      tiles = staged ? abs(tiles) : max(tiles, 0);
      Count total;
      const Count before = block_excl<kPlanThreads>(Count{staged ? (tiles + 1) >> 1 : 0, 0}, warp_sum, total);
      if (g < n_groups) {
        p.tiles[g] = tiles;
        p.stage_at[g] = pages + before.items;
      }
      pages += total.items;
    }
    if (tid == 0) p.stage_at[p.n_groups] = pages;
    __syncthreads();
  }
  const int pre_list = staged ? 2 : 0;
  // prefix items
  Count pre{0, 0};
  int most_tiles = 0;
  for (int g0 = 0; g0 < n_groups; g0 += kPlanThreads) {
    const int g = g0 + tid;
    Count mine{0, 0};
    if (g < n_groups && p.tiles[g] > 0) {
      const long long cols = static_cast<long long>(gload(p.start + g + 1) - gload(p.start + g)) * p.H;
      mine.items = static_cast<int>((cols + p.cols - 1) / p.cols);
      mine.line = static_cast<long long>(mine.items) * (p.tiles[g] + p.cost[pre_list]);
      most_tiles = max(most_tiles, p.tiles[g]);
    }
    Count total;
    const Count before = block_excl<kPlanThreads>(mine, warp_sum, total);
    if (g < n_groups) {
      p.base[g] = pre.items + before.items;
      p.base_at[g] = pre.line + before.line;
    }
    pre.items += total.items;
    pre.line += total.line;
  }
  __syncthreads();
  for (int i = tid; i < pre.items; i += kPlanThreads) {
    const int g = last_not_above(p.base, n_groups, i);       // (the last of equal ones: the one with items)
    const int s = gload(p.start + g), e = gload(p.start + g + 1), b = i - p.base[g];
    p.items[pre_list][i] = make_int4(s * p.H + b * p.cols, min(p.cols, (e - s) * p.H - b * p.cols),
                                     staged ? p.stage_at[g] : p.table[g], 0);
    p.nt[pre_list][i] = p.tiles[g];
    p.at[pre_list][i] = p.base_at[g] + static_cast<long long>(b) * (p.tiles[g] + p.cost[pre_list]);
  }
  // the rows' own items
  const int first = n_groups > 0 ? gload(p.start) : 0, end = n_groups > 0 ? gload(p.start + n_groups) : 0;
  const auto own_tiles = [&](int t, int& shared, int4& info) {
    const int len = row_len(p.pg, t);
    shared = 0;
    info = make_int4(-1, 0, -1, 0);
    if (t >= first && t < end) {
      const int g = last_not_above(p.start, n_groups, t);
      if (p.tiles[g] > 0 && len >= p.tiles[g] * kRows) {
        shared = p.tiles[g];
        info.x = p.base[g];
        info.y = gload(p.start + g) * p.H;
      }
    }
    return (len + kRows - 1) / kRows - shared;
  };
  int list = 0;
  if (p.two && staged) {       // (their prefixes are not in list 0 either)
    list = 1;
  } else if (p.two) {          // in a walk of their own, where they are many
    Count mine{0, 0}, total;
    int shared;
    int4 info;
    for (int t = tid; t < p.n_q; t += kPlanThreads) mine.line += own_tiles(t, shared, info);
    block_excl<kPlanThreads>(mine, warp_sum, total);
    list = total.line > p.most_own ? 1 : 0;
  }
  Count own = list == pre_list ? pre : Count{0, 0};
  int most_own = 0;
  for (int t0 = 0; t0 < p.n_q; t0 += kPlanThreads) {
    const int t = t0 + tid;
    int4 info = make_int4(-1, 0, -1, 0);
    int tiles = 0, shared = 0;
    if (t < p.n_q) {
      if (bad_length(p.pg, t)) report(faults, DEV_ERR_RANGE);
      tiles = own_tiles(t, shared, info);
      info.w = list + 4 * pre_list;
      most_own = max(most_own, tiles);
    }
    Count total;
    const Count before = block_excl<kPlanThreads>(tiles > 0 ? Count{1, tiles + p.cost[list]} : Count{0, 0}, warp_sum, total);
    if (t < p.n_q) {
      if (tiles > 0) {
        const int i = own.items + before.items;
        info.z = i;
        p.items[list][i] = make_int4(t * p.H, p.H | kItemOwn | (shared ? 0 : kItemSole), t, shared);
        p.nt[list][i] = tiles;
        p.at[list][i] = own.line + before.line;
      }
      p.rows[t] = info;
    }
    own.items += total.items;
    own.line += total.line;
  }
  most_tiles = __reduce_max_sync(0xffffffffu, most_tiles);
  most_own = __reduce_max_sync(0xffffffffu, most_own);
  if (lane == 0) {
    atomicMax(&tallest[pre_list], most_tiles);
    atomicMax(&tallest[list], most_own);
  }
  __syncthreads();
  // each group's share
  for (int k = 0; k < 3; ++k) {
    if (p.n_grp[k] == 0) continue;             // no such walk
    const int cost = p.cost[k];
    const Count c = k == list ? own : k == pre_list ? pre : Count{0, 0};
    bool by_row;
    const int groups = share_groups<kItems>(p.n_grp[k], p.pair[k] ? 2 : 1, c.items, c.line, tallest[k] + cost, by_row);
    // Where share g begins: an item, and the tiles before it in the item and in the list.  A cut that would leave a
    // piece of one tile is moved to the item's end or beginning.
    const auto cut = [&](int g, int& i, int& tile) -> long long {
      if (g == groups) {
        i = c.items;
        tile = 0;
        return c.line - static_cast<long long>(cost) * c.items;
      }
      const long long at = share_start(c.line, g, groups);
      i = last_not_above(p.at[k], c.items, at);
      const int nt = p.nt[k][i];
      const long long before = p.at[k][i] - static_cast<long long>(cost) * i;
      tile = static_cast<int>(at - p.at[k][i]) - cost;
      if (tile < 2) {
        tile = 0;
      } else if (nt - tile < 2) {
        ++i;
        tile = 0;
        return before + nt;
      }
      return before + tile;
    };
    for (int g = tid; g < p.n_grp[k]; g += kPlanThreads) {
      int4 r = make_int4(0, 0, 0, 0);
      if (g < groups && by_row) {
        r = make_int4(g, 0, p.nt[k][g], 0);
      } else if (g < groups) {
        int i, tile;
        const long long from = cut(g, r.x, r.y), to = cut(g + 1, i, tile);
        r.z = static_cast<int>(to - from);
      }
      p.shares[k][g] = r;
    }
  }
  if (tid == 0) {
    p.faults[0] = faults.bits;
    p.faults[1] = faults.count;
  }
}

// The staged pages: codes of each group's shared tiles to bf16 rows, and the table that names them (-1: a page outside
// the cache, which the walk reports).  A block takes a part of a page, a warp four
// rows of it at a time.  (Whole pages, some blocks two of them and some one: 344 us for a call that takes 340.)
__global__ void __launch_bounds__(256) latent_stage_kernel(const LatentCache c, const PagedRows pg, const int32_t* stage_at,
                                                           const int32_t* table, int n_groups, uint16_t* rows,
                                                           int32_t* stage_table) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_trigger();
  grid_wait();
  const int parts = gload(stage_at + n_groups) * kStageParts;
#pragma unroll 1
  for (int u = blockIdx.x; u < parts; u += gridDim.x) {
    constexpr int kPartRows = kPageRows / kStageParts;
    const int p = u / kStageParts, part = u % kStageParts;
    const int g = last_not_above(stage_at, n_groups, p), k = p - gload(stage_at + g);
    const int page = gload(pg.block_table + static_cast<size_t>(gload(table + g)) * pg.max_pages + k);
    const bool in = static_cast<uint32_t>(page) < static_cast<uint32_t>(pg.n_pages);
    if (threadIdx.x == 0 && part == 0) stage_table[p] = in ? p : -1;
    if (!in) continue;
#pragma unroll 1
    for (int r0 = part * kPartRows + warp * 4; r0 < (part + 1) * kPartRows; r0 += 32) {
      const size_t row = (static_cast<size_t>(page) << kPageShift) + r0;
      uint4 w[4];
      uint32_t sc[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        w[u] = gload_once(c.latent + (row + u) * kDv + lane * 16);
        sc[u] = gload(reinterpret_cast<const uint32_t*>(c.scale) + row + u);
      }
      const uint4 rope = gload_once(c.rope + (row + (lane >> 3)) * 64 + (lane & 7) * 8);
      uint16_t* dst = rows + ((static_cast<size_t>(p) << kPageShift) + r0) * kDqk;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint32_t m = fp8_mult((sc[u] >> (8 * (lane >> 3))) & 0xFFu);
        uint32_t o[8];
        fp8x4_to_bf16(w[u].x, m, o[0], o[1]);
        fp8x4_to_bf16(w[u].y, m, o[2], o[3]);
        fp8x4_to_bf16(w[u].z, m, o[4], o[5]);
        fp8x4_to_bf16(w[u].w, m, o[6], o[7]);
        stg256(dst + u * kDqk + lane * 16, o);
      }
      *reinterpret_cast<uint4*>(dst + (lane >> 3) * kDqk + kDv + (lane & 7) * 8) = rope;
    }
  }
}

struct JoinArgs {
  LArgs walk[3];             // by list; n_cta 0: no such walk
  const int4* rows;
  const uint32_t* plan_faults;
  int cols;
};

// The pieces of an item's column: one, whole, or the partials of groups b .. b + n - 1, of which the first is in the
// second slot of its group and the others in the first of theirs.
struct Pieces {
  const float* o;
  const float4* m;
  size_t first, next, pitch;
  int n;
  __device__ __forceinline__ size_t at(int k) const { return k == 0 ? first : next + (k - 1) * pitch; }
};
__device__ __forceinline__ Pieces find_pieces(const LArgs& a, int2 groups, int col_in_item, size_t col) {
  Pieces p{};
  // (a walk whose wait ran out has left items unnoted: what is found there then is any number, and no piece)
  if (groups.x < 0 || groups.y > a.n_grp || groups.x >= groups.y) return p;
  p.n = groups.y - groups.x;
  if (p.n == 1) {
    p.o = a.whole_o;
    p.m = a.whole_m;
    p.first = col;
  } else {
    p.o = a.part_o;
    p.m = a.item_m;
    p.pitch = 2 * static_cast<size_t>(a.part_cols);
    p.first = (static_cast<size_t>(groups.x) * 2 + 1) * a.part_cols + col_in_item;
    p.next = static_cast<size_t>(groups.x + 1) * p.pitch + col_in_item;
  }
  return p;
}

// One column's pieces put together, HPB columns a block, 8 / HPB warps each: a warp takes every (8 / HPB)-th
// piece, a lane 16 dims.  With M the largest of the pieces' maxima m_s and w_s = 2^(m_s - M), out = sum w_s O_s /
// sum w_s lr_s and lse = ln 2 (M + log2 sum w_s l_s); the order of the sums is fixed.  Four trips to L2, one behind
// the other: the row, its items' groups, the maxima and sums together with the first O rows, the other O rows.
// One block more puts the fault words together.
template <int HPB>
__global__ void __launch_bounds__(256) latent_shared_join_kernel(const __grid_constant__ JoinArgs j) {
  constexpr int kJoinWarps = 8 / HPB;
  constexpr int kMost = 2 * kMostGroups;
  __shared__ float4 sum[HPB][kJoinWarps > 1 ? kJoinWarps - 1 : 1][kJoinWarps > 1 ? kDv / 4 : 1];
  __shared__ float weight[8][kMost];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int hw = warp / kJoinWarps, w = warp % kJoinWarps;
  const LArgs& out = j.walk[0];
  grid_trigger();
  grid_wait();
  if (blockIdx.x == gridDim.x - 1) {
    if (warp != 0) return;
    uint32_t bits = lane == 0 ? j.plan_faults[0] : 0, count = lane == 0 ? j.plan_faults[1] : 0;
    for (int k = 0; k < 3; ++k)
      for (int i = lane; i < j.walk[k].n_cta; i += 32) {
        bits |= j.walk[k].err[2 * i];
        count += j.walk[k].err[2 * i + 1];
      }
    bits = __reduce_or_sync(0xffffffffu, bits);
    count = __reduce_add_sync(0xffffffffu, count);
    if (lane == 0) {
      out.status[0] = bits;
      out.status[1] = count;
    }
    return;
  }
  const int H = out.H;
  const long long col = static_cast<long long>(blockIdx.x) * HPB + hw, all = static_cast<long long>(out.n_q) * H;
  const bool live = col < all;
  float M = -INFINITY, lr = 0.f, ls = 0.f;
  float4 acc[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  bool done = !live;
  if (live) {
    const int t = static_cast<int>(col / H), h = static_cast<int>(col - static_cast<long long>(t) * H);
    const int4 info = gload(j.rows + t);
    const int in_group = static_cast<int>(col - info.y);
    int2 pre_groups = make_int2(0, 0), own_groups = make_int2(0, 0);
    const LArgs &own_walk = j.walk[info.w & 3], &pre_walk = j.walk[info.w >> 2];
    if (info.x >= 0) pre_groups = gload(pre_walk.pieces + info.x + in_group / j.cols);
    if (info.z >= 0) own_groups = gload(own_walk.pieces + info.z);
    const Pieces pre = find_pieces(pre_walk, pre_groups, in_group % j.cols, col);
    const Pieces own = find_pieces(own_walk, own_groups, h, all + col);
    done = pre.n == 0 && own.n == 1;           // written by the walk
    const int n = done ? 0 : pre.n + own.n;
    const auto meta = [&](int k) { return k < pre.n ? gload(pre.m + pre.at(k)) : gload(own.m + own.at(k - pre.n)); };
    constexpr int kAhead = 3;                  // O rows in flight
    bool weighed = false;
#pragma unroll 1
    for (int k0 = w; k0 < n || (!weighed && n > 0); k0 += kAhead * kJoinWarps) {
      float4 o[kAhead][4];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int k = k0 + u * kJoinWarps;
        if (k < n) {
          const float* row = k < pre.n ? pre.o + pre.at(k) * kDv : own.o + own.at(k - pre.n) * kDv;
          const float4* src = reinterpret_cast<const float4*>(row) + lane;
#pragma unroll
          for (int v = 0; v < 4; ++v) o[u][v] = gload(src + 32 * v);
        }
      }
      if (!weighed) {
        // (while the rows are on their way)  A piece without a key weighs nothing; one whose sum is NaN makes the
        // column NaN even where its maximum says nothing.
        weighed = true;
        const auto weigh = [&](const float4& m, int k) {
          const float f = m.x == -INFINITY ? (m.y == m.y ? 0.f : m.y) : exp2f(m.x - M);
          weight[warp][k] = f;
          lr += f * m.y;
          ls += f * m.z;
        };
        float4 m[2];                           // (more than 64 pieces are loaded twice)
#pragma unroll
        for (int u = 0; u < 2; ++u) m[u] = lane + 32 * u < n ? meta(lane + 32 * u) : make_float4(-INFINITY, 0.f, 0.f, 0.f);
        M = fmaxf(m[0].x, m[1].x);
        for (int k = lane + 64; k < n; k += 32) M = fmaxf(M, meta(k).x);
#pragma unroll
        for (int e = 16; e > 0; e >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, e));
#pragma unroll
        for (int u = 0; u < 2; ++u) weigh(m[u], lane + 32 * u);
        for (int k = lane + 64; k < n; k += 32) weigh(meta(k), k);
        __syncwarp();
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int k = k0 + u * kJoinWarps;
        if (k >= n) break;
        const float f = weight[warp][k];
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          acc[v].x += f * o[u][v].x;
          acc[v].y += f * o[u][v].y;
          acc[v].z += f * o[u][v].z;
          acc[v].w += f * o[u][v].w;
        }
      }
    }
  }
  if (w > 0) {
#pragma unroll
    for (int k = 0; k < 4; ++k) sum[hw][w - 1][lane + 32 * k] = acc[k];
  }
  __syncthreads();
  if (w > 0 || done) return;
#pragma unroll
  for (int e = 16; e > 0; e >>= 1) {
    lr += __shfl_xor_sync(0xffffffffu, lr, e);
    ls += __shfl_xor_sync(0xffffffffu, ls, e);
  }
  const float inv = lr == 0.f ? 0.f : 1.f / lr;
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
    reinterpret_cast<uint2*>(out.out + static_cast<size_t>(col) * kDv)[lane + 32 * k] =
        make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
  }
  if (out.lse && lane == 0) out.lse[col] = ls == 0.f ? -INFINITY : (M + log2f(ls)) * 0.69314718055994531f;
}

struct WalkLayout {
  bool used, pair;
  int cols, n_grp, n_items;
  size_t off_nt, off_items, off_at, off_pieces, off_err, off_shares, off_m, off_o, off_ring;
};
struct Layout {
  WalkLayout walk[3];        // by list
  size_t off_tiles, off_table, off_base, off_base_at, off_rows, off_faults, off_whole_m, off_whole_o, off_stage_at, off_stage_table,
      off_stage, total;
};
// Whether an fp8 cache's prefixes of groups of that many columns may have enough blocks to be staged.
bool may_stage(long long group_cols) { return group_cols > (kStageBlocks - 1) * 128; }
Layout shared_layout(int n_q, int n_heads, int n_groups, int max_rows) {
  Layout L{};
  int sms = device_sm_count();
  if (sms <= 0) sms = 152;
  const long long group_cols = static_cast<long long>(std::max(1, std::min(max_rows, n_q))) * n_heads;
  const bool pair = group_cols > 64;
  L.walk[0].used = true;
  L.walk[0].pair = pair;
  L.walk[0].cols = pair ? 128 : head_block(static_cast<int>(group_cols));
  L.walk[1].used = pair && n_heads <= 64;
  L.walk[1].cols = head_block(std::min(n_heads, 64));
  L.walk[2].used = n_groups > 0 && may_stage(group_cols);
  L.walk[2].pair = true;
  L.walk[2].cols = 128;
  const long long all = static_cast<long long>(n_q) * n_heads, pre = all / L.walk[0].cols + n_groups;
  const auto items = [](long long n) { return static_cast<int>(std::min<long long>(n, 0x7FFFFFFF)); };
  L.walk[0].n_items = items(pre + n_q);
  L.walk[1].n_items = n_q;
  L.walk[2].n_items = items(pre);
  size_t o = 0;
  const auto take = [&](size_t n, size_t bytes) {
    const size_t at = o;
    o += (n * bytes + 255) & ~size_t(255);
    return at;
  };
  const size_t groups = static_cast<size_t>(n_groups);
  L.off_faults = take(2, sizeof(uint32_t));
  L.off_tiles = take(groups, sizeof(int32_t));
  L.off_table = take(groups, sizeof(int32_t));
  L.off_base = take(groups, sizeof(int32_t));
  L.off_base_at = take(groups, sizeof(long long));
  L.off_rows = take(n_q, sizeof(int4));
  for (WalkLayout& w : L.walk) {
    if (!w.used) continue;
    w.n_grp = std::max(1, std::min(w.pair ? sms / 2 : sms, kMostGroups));
    const size_t n = static_cast<size_t>(w.n_items), slots = static_cast<size_t>(w.n_grp) * 2 * w.cols;
    w.off_nt = take(n, sizeof(int32_t));
    w.off_items = take(n, sizeof(int4));
    w.off_pieces = take(n, sizeof(int2));
    w.off_at = take(n, sizeof(long long));
    w.off_err = take(static_cast<size_t>(w.n_grp) * 2, 2 * sizeof(uint32_t));
    w.off_shares = take(w.n_grp, sizeof(int4));
    w.off_m = take(slots, sizeof(float4));
    w.off_o = take(slots, kDv * sizeof(float));
    if (&w == &L.walk[2]) {
      L.off_stage_at = take(groups + 1, sizeof(int32_t));
      L.off_stage_table = take(kStagePages, sizeof(int32_t));
      L.off_stage = take(static_cast<size_t>(kStagePages) * kPageRows * kDqk, sizeof(uint16_t));
    } else if (w.pair) {
      w.off_ring = take(static_cast<size_t>(w.n_grp) * kRing * kRows * kDqk, sizeof(uint16_t));
    }
  }
  L.off_whole_m = take(static_cast<size_t>(all) * 2, sizeof(float4));
  L.off_whole_o = take(static_cast<size_t>(all) * 2 * kDv, sizeof(float));
  L.total = o;
  return L;
}

}  // namespace

bool latent_shared_alone(bool fp8, int n_q, int n_heads, const PagedRows& pg, const SharedRows& groups) {
  if (groups.n_groups == 0) return true;                                   // no groups to check either
  if (!latent_attn_joins(n_q, n_heads, pg)) return false;                  // (it is the join that checks them)
  // A group of m rows is walked by rows where its columns fill as many blocks of 128: from 65 heads on, up to that many
  // rows.  Then only staged prefixes are worth a list.  (128 heads, fp8, with a list that shares
  // nothing and without, us: 32 sequences of five rows and 8000 keys 421, 413; 512 of 1000 keys 1103, 941.)
  const long long m = std::max(1, std::min(groups.max_rows, n_q));
  if (n_heads > 64 && m * (128 - n_heads) < 128 && !(fp8 && may_stage(m * n_heads))) return true;
  return 2LL * n_q * pg.max_pages <= kAloneTiles;
}

size_t latent_shared_ws_bytes(int n_q, int n_heads, int n_groups, int max_rows) {
  return shared_layout(n_q, n_heads, n_groups, max_rows).total;
}

SharedWalks latent_shared_walks(int n_q, int n_heads, int n_groups, int max_rows) {
  const Layout L = shared_layout(n_q, n_heads, n_groups, max_rows);
  SharedWalks s{};
  for (int k = 0; k < 3; ++k) {
    const WalkLayout& w = L.walk[k];
    s.used[k] = w.used;
    s.pair[k] = w.pair;
    s.q_rows[k] = w.pair ? 64 : w.cols;
    if (k == 2) {
      s.rows_offset[k] = L.off_stage;
      s.rows[k] = kStagePages * kPageRows;
    } else if (w.pair) {
      s.rows_offset[k] = w.off_ring;
      s.rows[k] = w.n_grp * kRing * kRows;
    }
  }
  return s;
}

cudaError_t launch_latent_shared(const LatentCache& c, const CUtensorMap* tmap_kv, const CUtensorMap* tmap_v,
                                 const CUtensorMap* tmap_q, const PagedRows& pg, const SharedRows& groups, int n_q,
                                 int n_heads, float scale, void* out, float* lse, uint32_t* status, void* scratch,
                                 cudaStream_t st) {
  const Layout L = shared_layout(n_q, n_heads, groups.n_groups, groups.max_rows);
  uint8_t* base = static_cast<uint8_t*>(scratch);
  const PipelineDebug dbg = pipeline_debug();
  const auto i32 = [&](size_t at) { return reinterpret_cast<int32_t*>(base + at); };
  const bool stage = c.fp8 && L.walk[2].used;
  PlanArgs p{};
  p.start = groups.start;
  p.prefix = groups.prefix;
  p.pg = pg;
  p.n_groups = groups.n_groups;
  p.n_q = n_q;
  p.H = n_heads;
  p.cols = L.walk[0].cols;
  p.two = L.walk[1].used;
  p.most_own = c.fp8 ? kMostOwnFp8 : kMostOwnBf16;
  p.tiles = i32(L.off_tiles);
  p.table = i32(L.off_table);
  p.base = i32(L.off_base);
  p.base_at = reinterpret_cast<long long*>(base + L.off_base_at);
  p.rows = reinterpret_cast<int4*>(base + L.off_rows);
  p.faults = reinterpret_cast<uint32_t*>(base + L.off_faults);
  p.stage_pages = stage ? kStagePages : 0;
  p.stage_at = i32(L.off_stage_at);
  JoinArgs j{};
  j.rows = p.rows;
  j.plan_faults = p.faults;
  j.cols = p.cols;
  for (int k = 0; k < 3; ++k) {
    const WalkLayout& w = L.walk[k];
    if (!w.used || (k == 2 && !stage)) continue;
    p.nt[k] = i32(w.off_nt);
    p.items[k] = reinterpret_cast<int4*>(base + w.off_items);
    p.at[k] = reinterpret_cast<long long*>(base + w.off_at);
    p.shares[k] = reinterpret_cast<int4*>(base + w.off_shares);
    p.n_grp[k] = w.n_grp;
    p.pair[k] = w.pair;
    p.cost[k] = w.pair && (!c.fp8 || k == 2) ? kItemCostPairBf16 : kItemCost;
    LArgs& a = j.walk[k];
    a.latent = c.latent;
    a.scale = c.scale;
    a.rope = c.rope;
    a.row_nt = p.nt[k];
    a.items = p.items[k];
    a.shares = p.shares[k];
    a.whole_o = reinterpret_cast<float*>(base + L.off_whole_o);
    a.whole_m = reinterpret_cast<float4*>(base + L.off_whole_m);
    a.pieces = reinterpret_cast<int2*>(base + w.off_pieces);
    a.pg = pg;
    a.out = static_cast<uint16_t*>(out);
    a.lse = lse;
    a.n_q = n_q;
    a.H = n_heads;
    a.n_grp = w.n_grp;
    a.n_hb = w.pair ? 2 : 1;
    a.n_cta = w.n_grp * a.n_hb;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.err = reinterpret_cast<uint32_t*>(base + w.off_err);
    a.item_m = reinterpret_cast<float4*>(base + w.off_m);
    a.part_o = reinterpret_cast<float*>(base + w.off_o);
    a.part_cols = w.cols;
    a.ring = reinterpret_cast<uint16_t*>(base + w.off_ring);
    a.status = status;
    a.wait_ns = dbg.wait_ns;
    a.stop_after = dbg.stop_after_tiles;
  }
  // a staged prefix's "table row" is its first page: rows of one entry, one behind the other
  if (stage) j.walk[2].pg = PagedRows{i32(L.off_stage_table), nullptr, 1, kStagePages};
  int ps = prof_begin(kProfAttnPrep, st);
  // (fewer threads, cheaper barriers: 4 rows 19.2 us with 128, 20.8 with 1024; 200 rows in 40 groups 31.2 with 512, 35.7
  // with 128; 900 in 300 93 with 1024, 99 with 512)
  const int most = std::max(n_q, 16 * groups.n_groups);
  cudaError_t e = most <= 128    ? launch_pdl(latent_plan_kernel<128>, dim3(1), 128, 0, st, 1, p)
                  : most <= 1024 ? launch_pdl(latent_plan_kernel<512>, dim3(1), 512, 0, st, 1, p)
                                 : launch_pdl(latent_plan_kernel<1024>, dim3(1), 1024, 0, st, 1, p);
  if (e == cudaSuccess && stage) {
    int sms = device_sm_count();
    if (sms <= 0) sms = 152;
    e = launch_pdl(latent_stage_kernel, dim3(16 * sms), 256, 0, st, 1, c, pg, p.stage_at, p.table, p.n_groups,
                   reinterpret_cast<uint16_t*>(base + L.off_stage), i32(L.off_stage_table));
  }
  prof_end(ps, st);
  if (e != cudaSuccess) return e;
  ps = prof_begin(kProfAttn, st);
  for (int k = 2; k >= 0 && e == cudaSuccess; --k) {
    const LArgs& a = j.walk[k];
    if (a.n_cta == 0) continue;
    e = L.walk[k].pair ? launch_latent_pair(c.fp8 && k != 2, kItems, tmap_kv[k], tmap_v[k], tmap_q[k], a, st)
                       : launch_latent_single(L.walk[k].cols, c.fp8, kItems, tmap_kv[k], tmap_v[k], tmap_q[k], a, st);
  }
  if (e == cudaSuccess) {
    const long long all = static_cast<long long>(n_q) * n_heads;
    // Warps a column by the pieces that it may be in: 64 columns in 40, one column a block 22.0 us, four 26.1, eight
    // 30.6; 768 in some 13, 54.0, 53.0, 61.3; 8192 in two or three, 378, 353, 349.
    const long long pieces = static_cast<long long>(L.walk[0].n_grp) * L.walk[0].cols / all;
    const int hpb = pieces > 32 ? 1 : pieces > 8 ? 4 : 8;
    e = launch_pdl(hpb == 1 ? latent_shared_join_kernel<1> : hpb == 4 ? latent_shared_join_kernel<4> : latent_shared_join_kernel<8>,
                   dim3(static_cast<unsigned>((all + hpb - 1) / hpb + 1)), 256, 0, st, 1, j);
  }
  prof_end(ps, st);
  return e;
}

}  // namespace dsa
