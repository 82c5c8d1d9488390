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
// prefixes, the single-CTA one for the rows' own keys, which are bound by bytes.
//
// A column's result comes from its prefix item and its own item, each whole or in partials where shares were
// cut: latent_shared_join_kernel puts them together with one softmax.  A row that is the only thing its columns
// come from is written by the walk itself.
//
// A group is walked by rows, not shared, where that takes no more items: from 128 heads on.
#include <cuda_bf16.h>

#include <algorithm>

#include "latent_attn.cuh"

namespace dsa {
namespace {

constexpr int kPlanThreads = 1024;
// A prefix of fewer tiles than this is left to the rows.
constexpr int kMinShared = 2;

struct PlanArgs {
  const int32_t* start;      // [n_groups + 1]
  const int32_t* prefix;     // [n_groups]
  PagedRows pg;
  int n_groups, n_q, H, cols;     // cols: columns of a prefix item
  bool two;                  // own items in a list of their own
  int32_t* tiles;            // [n_groups]: the shared tiles
  int32_t* table;            // [n_groups]: the row whose table names their pages
  int32_t* base;             // [n_groups + 1]: first item
  int32_t* nt[2];
  int4* items[2];
  int4* rows;                // [n_q]: first prefix item (-1), its first column, own item (-1)
  int32_t* n_items;          // [2]
  uint32_t* faults;          // [2]
};

// Exclusive sum over the block's threads; total: the sum.
__device__ __forceinline__ int block_excl(int x, int* warp_sum, int& total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  const int w = warp_sum[lane];
  int before = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += y;
  }
  total = __shfl_sync(0xffffffffu, before, 31);
  before -= w;
  return __shfl_sync(0xffffffffu, before, warp) + incl - x;
}
// The last of the n ascending values at v that is <= x; v[0] <= x.
__device__ __forceinline__ int last_not_above(const int32_t* v, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (gload(v + mid) <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kPlanThreads) latent_plan_kernel(const __grid_constant__ PlanArgs p) {
  __shared__ int warp_sum[32];
  __shared__ CtaFaults faults;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  grid_trigger();
  if (tid == 0) faults.bits = faults.count = 0;
  grid_wait();
  // groups that do not lie in order within the rows: none is shared
  bool bad = false;
  for (int g = tid; g <= p.n_groups; g += kPlanThreads) {
    const int s = gload(p.start + g);
    bad |= s < 0 || s > p.n_q || (g < p.n_groups && gload(p.start + g + 1) < s);
  }
  bad = __syncthreads_or(bad);
  if (bad && tid == 0) report(faults, DEV_ERR_RANGE);
  const int n_groups = bad ? 0 : p.n_groups;
  // a warp a group: its longest row
  for (int g = warp; g < n_groups; g += kPlanThreads / 32) {
    const int s = gload(p.start + g), n = gload(p.start + g + 1) - s, want = gload(p.prefix + g);
    int longest = -1, at = 0;
    for (int r = lane; r < n; r += 32) {
      const int len = row_len(p.pg, s + r);
      if (len > longest) {
        longest = len;
        at = s + r;
      }
    }
    const int most = __reduce_max_sync(0xffffffffu, longest);
    at = __reduce_min_sync(0xffffffffu, longest == most ? at : 0x7FFFFFFF);
    if (lane == 0) {
      const long long blocks = (static_cast<long long>(n) * p.H + p.cols - 1) / p.cols;
      int tiles = min(max(want, 0), max(most, 0)) / kRows;
      if (n < 2 || tiles < kMinShared || blocks >= n) tiles = 0;
      if (want < 0) report(faults, DEV_ERR_RANGE);
      p.tiles[g] = tiles;
      p.table[g] = at;
    }
  }
  __syncthreads();
  // prefix items
  int n_pre = 0;
  for (int g0 = 0; g0 < n_groups; g0 += kPlanThreads) {
    const int g = g0 + tid;
    int blocks = 0;
    if (g < n_groups && p.tiles[g] > 0) {
      const long long cols = static_cast<long long>(gload(p.start + g + 1) - gload(p.start + g)) * p.H;
      blocks = static_cast<int>((cols + p.cols - 1) / p.cols);
    }
    int total;
    const int at = n_pre + block_excl(blocks, warp_sum, total);
    if (g < n_groups) p.base[g] = at;
    n_pre += total;
  }
  __syncthreads();
  for (int i = tid; i < n_pre; i += kPlanThreads) {
    const int g = last_not_above(p.base, n_groups, i);       // (the last of equal ones: the one with items)
    const int s = gload(p.start + g), e = gload(p.start + g + 1), b = i - p.base[g];
    p.items[0][i] = make_int4(s * p.H + b * p.cols, min(p.cols, (e - s) * p.H - b * p.cols), p.table[g], 0);
    p.nt[0][i] = p.tiles[g];
  }
  // the rows' own items
  const int list = p.two ? 1 : 0;
  int n_own = p.two ? 0 : n_pre;
  const int first = n_groups > 0 ? gload(p.start) : 0, end = n_groups > 0 ? gload(p.start + n_groups) : 0;
  for (int t0 = 0; t0 < p.n_q; t0 += kPlanThreads) {
    const int t = t0 + tid;
    int4 info = make_int4(-1, 0, -1, 0);
    int own = 0, shared = 0;
    if (t < p.n_q) {
      const int want = gload(p.pg.seq_len + t), len = row_len(p.pg, t);
      if (want != len) report(faults, DEV_ERR_RANGE);
      if (t >= first && t < end) {
        const int g = last_not_above(p.start, n_groups, t);
        if (p.tiles[g] > 0 && len >= p.tiles[g] * kRows) {
          shared = p.tiles[g];
          info.x = p.base[g];
          info.y = gload(p.start + g) * p.H;
        }
      }
      own = (len + kRows - 1) / kRows - shared;
    }
    int total;
    const int at = n_own + block_excl(own > 0 ? 1 : 0, warp_sum, total);
    if (t < p.n_q) {
      if (own > 0) {
        info.z = at;
        p.items[list][at] = make_int4(t * p.H, p.H | kItemOwn | (shared ? 0 : kItemSole), t, shared);
        p.nt[list][at] = own;
      }
      p.rows[t] = info;
    }
    n_own += total;
  }
  __syncthreads();
  if (tid == 0) {
    p.n_items[0] = p.two ? n_pre : n_own;
    p.n_items[1] = n_own;
    p.faults[0] = faults.bits;
    p.faults[1] = faults.count;
  }
}

struct JoinArgs {
  LArgs walk[2];             // the walks of prefix items and of own items (one launch: the same)
  const int4* rows;
  const uint32_t* plan_faults;
  int n_walks, cols;
};

// The pieces of an item: `n` partials from `o` on, each `pitch` columns behind the one before (the first is in
// the second slot of its group, the others in the first of theirs), or one, whole.
struct Pieces {
  const float *o, *m;
  size_t step, first, next;      // column of the first piece, of the second; the third lies pitch behind that
  size_t pitch;
  int n;
  __device__ __forceinline__ size_t at(int k) const { return k == 0 ? first : next + (k - 1) * pitch; }
};
__device__ __forceinline__ Pieces find_pieces(const LArgs& a, int item, int col_in_item, size_t col, bool own) {
  const int lane = threadIdx.x & 31;
  Pieces p{};
  if (item < 0) return p;
  uint32_t below = 0;
#pragma unroll
  for (int k = 0; k < kMostGroups / 32; ++k) {
    const int c = lane + 32 * k;
    if (c >= a.n_grp) continue;
    const int2 st = gload(a.start + c);
    below += st.x < item || (st.x == item && st.y == 0) ? 1u : 0u;
    below += st.x <= item ? 0x10000u : 0u;
  }
  below = __reduce_add_sync(0xffffffffu, below);
  const int b = static_cast<int>(below & 0xFFFFu) - 1, end = static_cast<int>(below >> 16);
  if (end - b < 2) {
    const size_t all = static_cast<size_t>(a.n_q) * a.H, k = own ? 1 : 0;
    p.o = a.whole_o + k * all * kDv;
    p.m = a.whole_m + k * 3 * all;
    p.step = all;
    p.first = col;
    p.n = 1;
  } else {
    p.o = a.part_o;
    p.m = a.part_m;
    p.pitch = 2 * static_cast<size_t>(a.part_cols);
    p.step = static_cast<size_t>(a.n_grp) * p.pitch;
    p.first = (static_cast<size_t>(b) * 2 + 1) * a.part_cols + col_in_item;
    p.next = static_cast<size_t>(b + 1) * 2 * a.part_cols + col_in_item;
    p.n = end - b;
  }
  return p;
}

// One column's pieces put together, HPB columns a block, 8 / HPB warps each: a warp takes every (8 / HPB)-th
// piece, a lane 16 dims.  With M the largest of the pieces' maxima m_s and w_s = 2^(m_s - M), out = sum w_s O_s /
// sum w_s lr_s and lse = ln 2 (M + log2 sum w_s l_s); the order of the sums is fixed.  One block more puts the
// fault words together.
template <int HPB>
__global__ void __launch_bounds__(256) latent_shared_join_kernel(const __grid_constant__ JoinArgs j) {
  constexpr int kJoinWarps = 8 / HPB;
  constexpr int kMost = 2 * kMostGroups;
  __shared__ float4 sum[HPB][kJoinWarps > 1 ? kJoinWarps - 1 : 1][kJoinWarps > 1 ? kDv / 4 : 1];
  __shared__ float weight[8][kMost];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int hw = warp / kJoinWarps, w = warp % kJoinWarps;
  const LArgs& own_walk = j.walk[j.n_walks - 1];
  grid_trigger();
  grid_wait();
  if (blockIdx.x == gridDim.x - 1) {
    if (warp != 0) return;
    uint32_t bits = lane == 0 ? j.plan_faults[0] : 0, count = lane == 0 ? j.plan_faults[1] : 0;
    for (int k = 0; k < j.n_walks; ++k)
      for (int i = lane; i < j.walk[k].n_cta; i += 32) {
        bits |= j.walk[k].err[2 * i];
        count += j.walk[k].err[2 * i + 1];
      }
    bits = __reduce_or_sync(0xffffffffu, bits);
    count = __reduce_add_sync(0xffffffffu, count);
    if (lane == 0) {
      own_walk.status[0] = bits;
      own_walk.status[1] = count;
    }
    return;
  }
  const int H = own_walk.H;
  const long long col = static_cast<long long>(blockIdx.x) * HPB + hw;
  const bool live = col < static_cast<long long>(own_walk.n_q) * H;
  float M = -INFINITY, lr = 0.f, ls = 0.f;
  float4 acc[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  bool done = !live;
  if (live) {
    const int t = static_cast<int>(col / H), h = static_cast<int>(col - static_cast<long long>(t) * H);
    const int4 info = gload(j.rows + t);
    const int in_group = static_cast<int>(col - info.y);
    const Pieces pre = find_pieces(j.walk[0], info.x < 0 ? -1 : info.x + in_group / j.cols, in_group % j.cols, col, false);
    const Pieces own = find_pieces(own_walk, info.z, h, col, true);
    done = pre.n == 0 && own.n == 1;           // written by the walk
    const int n = done ? 0 : pre.n + own.n;
    const auto piece = [&](int k, const float*& m, size_t& step) -> const float4* {
      const bool first = k < pre.n;
      const size_t at = first ? pre.at(k) : own.at(k - pre.n);
      m = (first ? pre.m : own.m) + at;
      step = first ? pre.step : own.step;
      return reinterpret_cast<const float4*>((first ? pre.o : own.o) + at * kDv) + lane;
    };
    const float* pm;
    size_t step;
    constexpr int kAhead = 3;                  // O rows in flight
    bool weighed = false;
#pragma unroll 1
    for (int k0 = w; k0 < n || (!weighed && n > 0); k0 += kAhead * kJoinWarps) {
      float4 o[kAhead][4];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int k = k0 + u * kJoinWarps;
        if (k < n) {
          const float4* src = piece(k, pm, step);
#pragma unroll
          for (int v = 0; v < 4; ++v) o[u][v] = gload(src + 32 * v);
        }
      }
      if (!weighed) {
        // (while the rows are on their way)  A piece without a key weighs nothing; one whose sum is NaN makes the
        // column NaN even where its maximum says nothing.
        weighed = true;
        for (int k = lane; k < n; k += 32) {
          piece(k, pm, step);
          M = fmaxf(M, gload(pm));
        }
#pragma unroll
        for (int e = 16; e > 0; e >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, e));
        for (int k = lane; k < n; k += 32) {
          piece(k, pm, step);
          const float m = gload(pm), l1 = gload(pm + step), l2 = gload(pm + 2 * step);
          const float f = m == -INFINITY ? (l1 == l1 ? 0.f : l1) : exp2f(m - M);
          weight[warp][k] = f;
          lr += f * l1;
          ls += f * l2;
        }
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
    reinterpret_cast<uint2*>(own_walk.out + static_cast<size_t>(col) * kDv)[lane + 32 * k] =
        make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
  }
  if (own_walk.lse && lane == 0) own_walk.lse[col] = ls == 0.f ? -INFINITY : (M + log2f(ls)) * 0.69314718055994531f;
}

struct WalkLayout {
  bool pair;
  int cols, n_grp;
  size_t off_err, off_start, off_m, off_o, off_ring;
};
struct Layout {
  WalkLayout walk[2];
  int n_walks, n_items[2];
  size_t off_tiles, off_table, off_base, off_nt[2], off_items[2], off_rows, off_counts, off_whole_m, off_whole_o, total;
};
Layout shared_layout(int n_q, int n_heads, int n_groups, int max_rows) {
  Layout L{};
  int sms = device_sm_count();
  if (sms <= 0) sms = 152;
  const long long group_cols = static_cast<long long>(std::max(1, std::min(max_rows, n_q))) * n_heads;
  L.n_walks = group_cols > 64 && n_heads <= 64 ? 2 : 1;
  L.walk[0].pair = group_cols > 64;
  L.walk[0].cols = group_cols > 64 ? 128 : head_block(static_cast<int>(group_cols));
  L.walk[1].pair = false;
  L.walk[1].cols = head_block(std::min(n_heads, 64));
  const long long all = static_cast<long long>(n_q) * n_heads;
  const long long pre = all / L.walk[0].cols + n_groups;
  L.n_items[0] = static_cast<int>(std::min<long long>(pre + (L.n_walks == 1 ? n_q : 0), 0x7FFFFFFF));
  L.n_items[1] = L.n_walks == 2 ? n_q : 0;
  size_t o = 0;
  const auto take = [&](size_t bytes) {
    const size_t at = o;
    o += (bytes + 255) & ~size_t(255);
    return at;
  };
  L.off_counts = take(4 * sizeof(int32_t));
  L.off_tiles = take(static_cast<size_t>(n_groups) * sizeof(int32_t));
  L.off_table = take(static_cast<size_t>(n_groups) * sizeof(int32_t));
  L.off_base = take((static_cast<size_t>(n_groups) + 1) * sizeof(int32_t));
  L.off_rows = take(static_cast<size_t>(n_q) * sizeof(int4));
  for (int k = 0; k < L.n_walks; ++k) {
    WalkLayout& w = L.walk[k];
    w.n_grp = std::max(1, std::min(w.pair ? sms / 2 : sms, kMostGroups));
    L.off_nt[k] = take(static_cast<size_t>(L.n_items[k]) * sizeof(int32_t));
    L.off_items[k] = take(static_cast<size_t>(L.n_items[k]) * sizeof(int4));
    w.off_err = take(static_cast<size_t>(w.n_grp) * 2 * 2 * sizeof(uint32_t));
    w.off_start = take(static_cast<size_t>(w.n_grp) * sizeof(int2));
    w.off_m = take(static_cast<size_t>(w.n_grp) * 2 * w.cols * 3 * sizeof(float));
    w.off_o = take(static_cast<size_t>(w.n_grp) * 2 * w.cols * kDv * sizeof(float));
    w.off_ring = w.pair ? take(static_cast<size_t>(w.n_grp) * kRing * kRows * kDqk * sizeof(uint16_t)) : 0;
  }
  L.off_whole_m = take(static_cast<size_t>(all) * 2 * 3 * sizeof(float));
  L.off_whole_o = take(static_cast<size_t>(all) * 2 * kDv * sizeof(float));
  L.total = o;
  return L;
}

}  // namespace

size_t latent_shared_ws_bytes(int n_q, int n_heads, int n_groups, int max_rows) {
  return shared_layout(n_q, n_heads, n_groups, max_rows).total;
}

SharedWalks latent_shared_walks(int n_q, int n_heads, int n_groups, int max_rows) {
  const Layout L = shared_layout(n_q, n_heads, n_groups, max_rows);
  SharedWalks w{};
  w.n = L.n_walks;
  for (int k = 0; k < L.n_walks; ++k) {
    w.pair[k] = L.walk[k].pair;
    w.q_rows[k] = L.walk[k].pair ? 64 : L.walk[k].cols;
    w.ring_offset[k] = L.walk[k].off_ring;
    w.ring_rows[k] = L.walk[k].pair ? L.walk[k].n_grp * kRing * kRows : 0;
  }
  return w;
}

cudaError_t launch_latent_shared(const LatentCache& c, const CUtensorMap* tmap_kv, const CUtensorMap* tmap_v,
                                 const CUtensorMap* tmap_q, const PagedRows& pg, const SharedRows& groups, int n_q,
                                 int n_heads, float scale, void* out, float* lse, uint32_t* status, void* scratch,
                                 cudaStream_t st) {
  const Layout L = shared_layout(n_q, n_heads, groups.n_groups, groups.max_rows);
  uint8_t* base = static_cast<uint8_t*>(scratch);
  const PipelineDebug dbg = pipeline_debug();
  const auto i32 = [&](size_t at) { return reinterpret_cast<int32_t*>(base + at); };
  PlanArgs p{};
  p.start = groups.start;
  p.prefix = groups.prefix;
  p.pg = pg;
  p.n_groups = groups.n_groups;
  p.n_q = n_q;
  p.H = n_heads;
  p.cols = L.walk[0].cols;
  p.two = L.n_walks == 2;
  p.tiles = i32(L.off_tiles);
  p.table = i32(L.off_table);
  p.base = i32(L.off_base);
  p.rows = reinterpret_cast<int4*>(base + L.off_rows);
  p.n_items = i32(L.off_counts);
  p.faults = reinterpret_cast<uint32_t*>(p.n_items + 2);
  for (int k = 0; k < L.n_walks; ++k) {
    p.nt[k] = i32(L.off_nt[k]);
    p.items[k] = reinterpret_cast<int4*>(base + L.off_items[k]);
  }
  int ps = prof_begin(kProfAttnPrep, st);
  cudaError_t e = launch_pdl(latent_plan_kernel, dim3(1), kPlanThreads, 0, st, 1, p);
  prof_end(ps, st);
  if (e != cudaSuccess) return e;
  JoinArgs j{};
  j.rows = p.rows;
  j.plan_faults = p.faults;
  j.n_walks = L.n_walks;
  j.cols = p.cols;
  ps = prof_begin(kProfAttn, st);
  for (int k = 0; k < L.n_walks && e == cudaSuccess; ++k) {
    const WalkLayout& w = L.walk[k];
    LArgs& a = j.walk[k];
    a.latent = c.latent;
    a.scale = c.scale;
    a.rope = c.rope;
    a.row_nt = p.nt[k];
    a.items = p.items[k];
    a.n_items = p.n_items + k;
    a.whole_o = reinterpret_cast<float*>(base + L.off_whole_o);
    a.whole_m = reinterpret_cast<float*>(base + L.off_whole_m);
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
    a.start = reinterpret_cast<int2*>(base + w.off_start);
    a.part_m = reinterpret_cast<float*>(base + w.off_m);
    a.part_o = reinterpret_cast<float*>(base + w.off_o);
    a.part_cols = w.cols;
    a.ring = reinterpret_cast<uint16_t*>(base + w.off_ring);
    a.status = status;
    a.wait_ns = dbg.wait_ns;
    a.stop_after = dbg.stop_after_tiles;
    e = w.pair ? launch_latent_pair(c.fp8, kItems, tmap_kv[k], tmap_v[k], tmap_q[k], a, st)
               : launch_latent_single(w.cols, c.fp8, kItems, tmap_kv[k], tmap_v[k], tmap_q[k], a, st);
  }
  if (e == cudaSuccess) {
    const long long all = static_cast<long long>(n_q) * n_heads;
    const int hpb = all <= 1024 ? 1 : 8;
    e = launch_pdl(hpb == 1 ? latent_shared_join_kernel<1> : latent_shared_join_kernel<8>,
                   dim3(static_cast<unsigned>((all + hpb - 1) / hpb + 1)), 256, 0, st, 1, j);
  }
  prof_end(ps, st);
  return e;
}

}  // namespace dsa
