// Eviction from a paged latent cache: the keys that stay, chosen by the attention weight they have received,
// and the copy of their rows to other pages.
//
// A sequence of L keys that is longer than n_keep keeps its first n_first, its last n_last and, of the keys
// between, the K = n_keep - n_first - n_last heaviest (ties: the lower position), all in order.
//
// Choosing.  A cluster of CTAs takes a sequence, each warp a run of consecutive keys.  The K-th heaviest
// weight is found by a radix select on order-preserving 32-bit keys, 11, 11 and 10 bits at a time: a histogram
// per CTA, summed over the cluster through distributed shared memory, one bin of which goes on.  Then each warp
// counts the keys above and at the limit, a scan over the cluster's warps says where its own go, and it writes
// them in order by ballots.  A CTA reads its keys once where it can hold them, up to 8192 in registers, up to 24576 in
// shared memory; of longer sequences they are read again in every pass, out of L2.
//
// Copying.  A warp takes eight rows; HBM bounds it.
//
// What bounds the call.  24 sequences of 8K to 65K keys cut to 16384, fp8: 95 us, of which the copy moves 490 MB in 72
// (6.8 TB/s, what a copy reaches), behind some 20 of choosing: three trips to memory and, a pass, two cluster barriers and
// a scan of 2048 bins.  Two of 3000 to 5000, bf16: 10 us, the same trips without a cluster and one launch more.  Keys
// read again in every pass: 104 us where they are held (15.4 for the small call); a clearing launch and always three
// passes: 97 and 11.7.
#include <cuda_bf16.h>

#include <algorithm>

#include "kernels.h"
#include "ptx.cuh"
#include "status.cuh"

namespace dsa {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMostCtas = 8;
constexpr int kBins = 2048;
// Where a CTA holds its keys: sixteen a lane in registers, 48 in shared memory, or nowhere.
enum Hold : int { kRegisters = 0, kShared = 1, kNowhere = 2 };
constexpr int kHeld = 16, kSharedHeld = 48;

// Larger weights have larger keys, -0 that of 0; a NaN has the smallest.
__device__ __forceinline__ uint32_t weight_key(float w) { return w == w ? float_key(w) : 0u; }

__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t load_cta(const uint32_t* p, uint32_t rank) {
  uint32_t v;
  asm volatile("{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %1, %2;\n ld.shared::cluster.u32 %0, [a];\n}\n"
               : "=r"(v)
               : "r"(smem_u32(p)), "r"(rank)
               : "memory");
  return v;
}
__device__ __forceinline__ void store_cta(uint32_t* p, uint32_t rank, uint32_t v) {
  asm volatile("{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %0, %1;\n st.shared::cluster.u32 [a], %2;\n}\n" ::"r"(smem_u32(p)),
               "r"(rank), "r"(v)
               : "memory");
}

struct Smem {
  // This CTA's histogram; behind the last pass, where nobody reads it any more, the keys above and at the limit of each
  // warp of the cluster.  (Beside each other, two CTAs that hold their keys in shared memory did not fit on an SM.)
  union {
    uint32_t mine[kBins];
    struct {
      uint32_t above[kMostCtas * kWarps], at[kMostCtas * kWarps];
    };
  };
  uint32_t all[kBins];               // the cluster's histogram
  uint32_t warp_sum[kWarps];
  uint32_t bin, before, count;       // the limit's bin, the entries above it and its own
};
constexpr int kSharedBytes = kThreads * kSharedHeld * static_cast<int>(sizeof(float));
// Two CTAs an SM, as the launch counts them: 228 KB, of which each CTA takes 1 KB more than it asks for, in steps of 128 B.
static_assert(2 * ((sizeof(Smem) + kSharedBytes + 1024 + 127) / 128 * 128) <= 228 * 1024, "two CTAs an SM");

// Inclusive sum over the lanes.
__device__ __forceinline__ uint32_t warp_incl(uint32_t x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

template <int HOLD>
__global__ void __launch_bounds__(kThreads, 2) evict_select_kernel(const __grid_constant__ Evict e, int n_cta, uint32_t* status) {
  __shared__ Smem sh;
  extern __shared__ float in_shared[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x / n_cta, rank = blockIdx.x - t * n_cta;
  const auto sync = [&]() {
    if (n_cta > 1) cluster_sync_all();
    else __syncthreads();
  };
  grid_trigger();
  grid_wait();
  const int want = gload(e.from.seq_len + t);
  const int L = max(0, min(want, e.from.max_pages << kPageShift));
  const int n = min(L, e.n_keep);
  const float* w = e.weight + t * e.weight_stride;
  float* w_out = e.weight_out ? e.weight_out + t * e.weight_out_stride : nullptr;
  int32_t* kept = e.kept + static_cast<long long>(t) * e.n_keep;
  const bool all = L <= e.n_keep;
  const int head = all ? L : e.n_first, tail = all ? 0 : e.n_last;
  const int K = n - head - tail;
  // the warp's run [lo, hi) of the keys between
  const int from = head, to = L - tail;
  const int run = (to - from + n_cta * kWarps - 1) / (n_cta * kWarps);
  const int lo = min(to, from + (rank * kWarps + warp) * run), hi = K > 0 ? min(to, lo + run) : lo;
  float held[HOLD == kRegisters ? kHeld : 1];
  float* mine = in_shared + warp * (32 * kSharedHeld) + lane;
  if constexpr (HOLD == kRegisters) {
#pragma unroll
    for (int u = 0; u < kHeld; ++u) held[u] = lo + 32 * u + lane < hi ? gload(w + lo + 32 * u + lane) : 0.f;
  } else if constexpr (HOLD == kShared) {
#pragma unroll 8
    for (int j = lo + lane; j < hi; j += 32) mine[j - lo - lane] = gload(w + j);
  }
  // each(j, weight of key j, whether there is one) for 32 keys after another
  const auto keys = [&](auto&& each) {
    if constexpr (HOLD == kRegisters) {
#pragma unroll
      for (int u = 0; u < kHeld; ++u)
        if (lo + 32 * u < hi) each(lo + 32 * u + lane, held[u], lo + 32 * u + lane < hi);
    } else {
#pragma unroll 4
      for (int j0 = lo; j0 < hi; j0 += 32) {
        const bool there = j0 + lane < hi;
        const float x = !there ? 0.f : HOLD == kShared ? mine[j0 - lo] : gload(w + j0 + lane);
        each(j0 + lane, x, there);
      }
    }
  };
  if (rank == 0 && threadIdx.x == 0) e.new_len[t] = n;
  if (blockIdx.x == 0 && threadIdx.x < 2) status[threadIdx.x] = 0u;      // (faults are the next kernel's to report)
  // those that stay in any case, and the unused end of kept
  const int stride = n_cta * kThreads, me = rank * kThreads + static_cast<int>(threadIdx.x);
  const auto keep = [&](int place, int j) {
    kept[place] = j;
    if (w_out) w_out[place] = gload(w + j);
  };
  for (int i = me; i < head; i += stride) keep(i, i);
  for (int i = me; i < tail; i += stride) keep(n - tail + i, L - tail + i);
  for (int i = n + me; i < e.n_keep; i += stride) kept[i] = -1;
  if (K == 0) return;                                          // (the whole cluster)

  uint32_t limit = 0;                // bits of the limit found so far, those from `shift` on
  uint32_t need = static_cast<uint32_t>(K);
  int shift = 0;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const int bits = pass == 2 ? 10 : 11;
    for (int b = threadIdx.x; b < kBins; b += kThreads) sh.mine[b] = 0;
    __syncthreads();
    keys([&](int, float x, bool there) {
      const uint32_t key = weight_key(x);
      if (there && (pass == 0 || (key >> (shift + bits)) == limit)) atomicAdd(&sh.mine[(key >> shift) & ((1u << bits) - 1u)], 1u);
    });
    sync();
    if (n_cta > 1) {
      // a part of the bins each, summed over the cluster, to every CTA
      const int part = kBins / n_cta + 1;
      for (int b = rank * part + static_cast<int>(threadIdx.x); b < min(kBins, (rank + 1) * part); b += kThreads) {
        uint32_t c[kMostCtas], s = 0;
#pragma unroll
        for (int k = 0; k < kMostCtas; ++k) c[k] = k < n_cta ? load_cta(&sh.mine[b], k) : 0u;
#pragma unroll
        for (int k = 0; k < kMostCtas; ++k) s += c[k];
        for (int k = 0; k < n_cta; ++k) store_cta(&sh.all[b], k, s);
      }
      cluster_sync_all();
    }
    // the bin that holds the need-th entry from above: thread i takes the four bins from the top
    const uint32_t* hist = n_cta > 1 ? sh.all : sh.mine;
    constexpr int PER = kBins / kThreads;
    uint32_t c[PER], sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      c[i] = hist[kBins - 1 - (static_cast<int>(threadIdx.x) * PER + i)];
      sum += c[i];
    }
    const uint32_t incl = warp_incl(sum);
    if (lane == 31) sh.warp_sum[warp] = incl;
    __syncthreads();
    const uint32_t warps = warp_incl(lane < kWarps ? sh.warp_sum[lane] : 0u);
    uint32_t before = __shfl_sync(0xffffffffu, warps, max(warp - 1, 0));
    before = (warp ? before : 0u) + incl - sum;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (before < need && need <= before + c[i]) {
        sh.bin = kBins - 1 - (static_cast<uint32_t>(threadIdx.x) * PER + i);
        sh.before = before;
        sh.count = c[i];
      }
      before += c[i];
    }
    __syncthreads();
    limit = (limit << bits) | sh.bin;
    need -= sh.before;
    if (need == sh.count) break;       // the whole bin stays (as a rule one key, after the second pass)
  }
  // limit: the K-th heaviest weight, or its upper bits; need: how many with these stay
  uint32_t above = 0, at = 0;
  keys([&](int, float x, bool there) {
    const uint32_t key = weight_key(x) >> shift;
    above += there && key > limit ? 1u : 0u;
    at += there && key == limit ? 1u : 0u;
  });
  above = __reduce_add_sync(0xffffffffu, above);
  at = __reduce_add_sync(0xffffffffu, at);
  if (lane < n_cta) {
    store_cta(&sh.above[rank * kWarps + warp], lane, above);
    store_cta(&sh.at[rank * kWarps + warp], lane, at);
  }
  sync();
  // what the warps before this one hold
  uint32_t above_before = 0, at_before = 0;
  for (int g = lane; g < rank * kWarps + warp; g += 32) {
    above_before += sh.above[g];
    at_before += sh.at[g];
  }
  above_before = __reduce_add_sync(0xffffffffu, above_before);
  at_before = __reduce_add_sync(0xffffffffu, at_before);
  keys([&](int j, float x, bool there) {
    const uint32_t key = weight_key(x) >> shift;
    const uint32_t a = __ballot_sync(0xffffffffu, there && key > limit), q = __ballot_sync(0xffffffffu, there && key == limit);
    const uint32_t lower = (1u << lane) - 1u;
    const uint32_t at_here = at_before + __popc(q & lower);
    const bool stays = ((a >> lane) & 1u) || (((q >> lane) & 1u) && at_here < need);
    if (stays) {
      const int place = from + static_cast<int>(above_before + __popc(a & lower) + min(at_here, need));
      kept[place] = j;
      if (w_out) w_out[place] = x;
    }
    above_before += __popc(a);
    at_before += __popc(q);
  });
}

// kCopyRows rows a warp: lane l looks one of them up, a trip each for its place and its page, then all rows' loads
// are in flight before the first store (bf16: half of them).  Eight rows where there are many, else two.
template <bool FP8, int kCopyRows>
__global__ void __launch_bounds__(256) evict_copy_kernel(const __grid_constant__ Evict e, const LatentCache src,
                                                         const LatentCache dst, int per_seq, uint32_t* status) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_trigger();
  grid_wait();
  const int t = blockIdx.x / per_seq;
  const int i0 = ((blockIdx.x - t * per_seq) * 8 + warp) * kCopyRows;
  const int n = gload(e.new_len + t);
  if (i0 == 0 && lane == 0) {
    const int want = gload(e.from.seq_len + t);
    if (want < 0 || want > (e.from.max_pages << kPageShift)) report(status, false, DEV_ERR_RANGE);
  }
  if (i0 >= n) return;
  const int i = i0 + (lane & (kCopyRows - 1));
  int from = -1, to = -1;
  if (i < n) {
    const int j = gload(e.kept + static_cast<long long>(t) * e.n_keep + i);
    const int to_page = gload(e.to.block_table + static_cast<long long>(t) * e.to.max_pages + (i >> kPageShift));
    const int page = gload(e.from.block_table + static_cast<long long>(t) * e.from.max_pages + (j >> kPageShift));
    if (static_cast<uint32_t>(page) < static_cast<uint32_t>(e.from.n_pages) &&
        static_cast<uint32_t>(to_page) < static_cast<uint32_t>(e.to.n_pages)) {
      from = (page << kPageShift) + (j & (kPageRows - 1));
      to = (to_page << kPageShift) + (i & (kPageRows - 1));
    } else if (lane < kCopyRows) {
      report(status, false, DEV_ERR_BAD_INDEX);
    }
  }
  if constexpr (FP8) {
    constexpr int kRope = (kCopyRows + 3) / 4;       // four rows' rotary dims an instruction
    uint4 v[kCopyRows], r[kRope];
    uint32_t sc = 0;
#pragma unroll
    for (int k = 0; k < kCopyRows; ++k) {
      const int row = __shfl_sync(0xffffffffu, from, k);
      if (row >= 0) v[k] = gload(reinterpret_cast<const uint4*>(src.latent + static_cast<size_t>(row) * 512) + lane);
    }
#pragma unroll
    for (int k = 0; k < kRope; ++k) {
      const int q = 4 * k + (lane >> 3), row = __shfl_sync(0xffffffffu, from, q);
      if (q < kCopyRows && row >= 0)
        r[k] = gload(reinterpret_cast<const uint4*>(src.rope + static_cast<size_t>(row) * 64) + (lane & 7));
    }
    if (lane < kCopyRows && from >= 0) sc = gload(reinterpret_cast<const uint32_t*>(src.scale) + from);
#pragma unroll
    for (int k = 0; k < kCopyRows; ++k) {
      const int row = __shfl_sync(0xffffffffu, to, k);
      if (row >= 0) reinterpret_cast<uint4*>(dst.latent + static_cast<size_t>(row) * 512)[lane] = v[k];
    }
#pragma unroll
    for (int k = 0; k < kRope; ++k) {
      const int q = 4 * k + (lane >> 3), row = __shfl_sync(0xffffffffu, to, q);
      if (q < kCopyRows && row >= 0) reinterpret_cast<uint4*>(dst.rope + static_cast<size_t>(row) * 64)[lane & 7] = r[k];
    }
    if (lane < kCopyRows && to >= 0) reinterpret_cast<uint32_t*>(dst.scale)[to] = sc;
  } else {
    // 72 vectors a row
    constexpr int kVec = 72, kAll = (kCopyRows * kVec + 31) / 32, kPart = kCopyRows > 4 ? (kAll + 1) / 2 : kAll;
#pragma unroll 1
    for (int h = 0; h < kAll; h += kPart) {
      uint4 v[kPart];
#pragma unroll
      for (int k = 0; k < kPart; ++k) {
        const int x = (h + k) * 32 + lane, row = __shfl_sync(0xffffffffu, from, x / kVec);
        if (x < kCopyRows * kVec && row >= 0)
          v[k] = gload(reinterpret_cast<const uint4*>(src.latent + static_cast<size_t>(row) * 1152) + x % kVec);
      }
#pragma unroll
      for (int k = 0; k < kPart; ++k) {
        const int x = (h + k) * 32 + lane, row = __shfl_sync(0xffffffffu, to, x / kVec);
        if (x < kCopyRows * kVec && row >= 0)
          reinterpret_cast<uint4*>(dst.latent + static_cast<size_t>(row) * 1152)[x % kVec] = v[k];
      }
    }
  }
}

}  // namespace

cudaError_t launch_evict(const Evict& a, const LatentCache& src, const LatentCache& dst, uint32_t* status, cudaStream_t st) {
  cudaError_t e;
  int sms = device_sm_count();
  if (sms <= 0) sms = 152;
  // As many CTAs a sequence as hold the longest that the table allows in registers, while all sequences are resident at
  // once; fewer for that only where their keys are held as before (60000 .. 65536 keys cut to 2048, fp8: 40 sequences,
  // clusters of seven 64.6 us, of six 54.4; 48, of six 72.9, of five 63.6; 100, of three 122, of two, which hold
  // nothing, 157).
  const int width = a.from.max_pages * kPageRows;
  const int fit = 2 * sms / std::max(1, std::min(a.n_seq, 2 * sms));
  int ctas = std::max(1, std::min({kMostCtas, fit, (width + kHeld * kThreads - 1) / (kHeld * kThreads)}));
  const auto form = [&](int n) -> Hold {       // (a warp's run is the CTA's sixteenth, rounded up)
    const long long run = (static_cast<long long>(width) + n * kWarps - 1) / (n * kWarps);
    return run <= 32 * kHeld ? kRegisters : run <= 32 * kSharedHeld ? kShared : kNowhere;
  };
  const Hold hold = form(ctas);
  if (hold == kShared && (e = smem_attr_once<evict_select_kernel<kShared>>(kSharedBytes)) != cudaSuccess) return e;
  const auto select = [&](auto kern, int smem) {
    constexpr auto k = decltype(kern)::value;
    while (ctas > 1 && form(ctas - 1) == hold && resident_clusters<k>(ctas, kThreads, smem) < a.n_seq) --ctas;
    const dim3 grid(static_cast<unsigned>(a.n_seq) * static_cast<unsigned>(ctas));
    return launch_pdl(k, grid, kThreads, static_cast<size_t>(smem), st, ctas, a, ctas, status);
  };
  e = hold == kRegisters ? select(Kernel<evict_select_kernel<kRegisters>>{}, 0)
      : hold == kShared  ? select(Kernel<evict_select_kernel<kShared>>{}, kSharedBytes)
                         : select(Kernel<evict_select_kernel<kNowhere>>{}, 0);
  if (e != cudaSuccess) return e;
  const int rows = std::min(a.n_keep, width);
  const int each = static_cast<long long>(a.n_seq) * rows > 64LL * sms ? 8 : 2;
  const int per_seq = (rows + 8 * each - 1) / (8 * each);
  const auto go = [&](auto kern) {
    return launch_pdl(kern, dim3(static_cast<unsigned>(a.n_seq) * static_cast<unsigned>(per_seq)), 256, 0, st, 1, a, src, dst,
                      per_seq, status);
  };
  if (each == 8) return src.fp8 ? go(evict_copy_kernel<true, 8>) : go(evict_copy_kernel<false, 8>);
  return src.fp8 ? go(evict_copy_kernel<true, 2>) : go(evict_copy_kernel<false, 2>);
}

}  // namespace dsa
