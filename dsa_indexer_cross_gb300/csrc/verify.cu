// Verification of drafted tokens against the target's probabilities, from given uniform numbers.
//
// Sequence t drafted x_0 .. x_{n-1} from q_0 .. q_{n-1}.  Draft i is taken when u_i q_i(x_i) < p_i(x_i)
// (probability min(1, p / q)); a is the first draft that is not, or n.  The token at place a is drawn from
//     r(v) = max(p_a(v) - q_a(v), 0)   a < n        r(v) = p_n(v)   a = n
// by inverting its distribution: the lowest v with sum_{w <= v} r(w) > u sum_w r(w).  The tokens then follow
// p, whatever q is.
//
// A cluster of CTAs takes a sequence: its warps own consecutive regions of the vocabulary, sum them in one
// pass, and exchange the sums through distributed shared memory; the CTA whose regions hold the drawn
// token reads that one region again (out of L2) and finds it.  One launch, one row of p and at most one of
// q read, and every sum in a fixed order.
//
// Sums.  A drawn token hangs on where u R falls among the running sums of up to 2^17 values, some 1e-5
// apart, so single precision would draw a neighbour now and then.  Every sum is kept as two floats (the
// error of each addition, and of p - q, is known exactly from a few more additions), good to some 2^-45.
// Double precision would do, but this GPU has few units for it: sums by warps and CTAs in double, with
// two-float sums inside a thread only, took 13.9 us where this takes 6.2 (one sequence, a vocabulary of 32000).
//
// What bounds it.  One sequence, 6.2 us in a graph: a chain of five trips to memory (lengths, tokens, their
// probabilities, the rows, the region again), the launch and one cluster barrier.  64 sequences, a vocabulary
// of 131072, fp32: 14.4 us for the 55 MB of a floor of 8.2, that chain and the loads behind it.  200 of 50257,
// bf16, no draft probabilities: 13.8 us.  The additions are made two at a time and, as 0 <= q <= p, with three
// for p - q (15.8 and 20.3 us one at a time).
#include <cuda_bf16.h>

#include <algorithm>
#include <climits>

#include "kernels.h"
#include "ptx.cuh"
#include "status.cuh"

namespace dsa {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMostCtas = 8;            // a cluster's CTAs
constexpr int kSoleMost = 4096;         // drafts of a call whose status one block writes

template <typename T>
struct Prob;
template <>
struct Prob<float> {
  static constexpr int PER = 4;
  static __device__ __forceinline__ float load(const float* p) { return gload(p); }
  static __device__ __forceinline__ float get(const uint4& v, int i) {
    return __uint_as_float(i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w);
  }
};
template <>
struct Prob<__nv_bfloat16> {
  static constexpr int PER = 8;
  static __device__ __forceinline__ float load(const __nv_bfloat16* p) {
    return __uint_as_float(static_cast<uint32_t>(gload(reinterpret_cast<const uint16_t*>(p))) << 16);
  }
  static __device__ __forceinline__ float get(const uint4& v, int i) {
    const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
    return __uint_as_float(i & 1 ? w & 0xFFFF0000u : w << 16);
  }
};

// A sum kept as two floats, good to some 2^-45 of it.
struct F2 {
  float hi, lo;
};
// p - q where it is positive (a NaN weighs nothing), with the error of the subtraction: 0 <= q <= p.
__device__ __forceinline__ F2 weight(float p, float q) {
  p = fmaxf(p, 0.f);
  q = fminf(q, p);
  const float r = p - q;
  return F2{r, (p - r) - q};
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
  const float s = a.hi + b.hi, c = s - a.hi;
  const float e = (a.hi - (s - c)) + (b.hi - c) + (a.lo + b.lo);
  const float hi = s + e;
  return F2{hi, e - (hi - s)};
}
__device__ __forceinline__ bool operator>(F2 a, F2 b) { return a.hi > b.hi || (a.hi == b.hi && a.lo > b.lo); }
// Two floats at once.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t x;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a), "f"(b));
  return x;
}
__device__ __forceinline__ float2 unpair(uint64_t x) {
  float2 v;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(x));
  return v;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// Two sums, the low parts not yet carried over.
struct Sums {
  uint64_t hi, lo;
  __device__ __forceinline__ void add(uint64_t w, uint64_t w_lo) {
    const uint64_t s = add2(hi, w), c = sub2(s, hi);
    lo = add2(lo, add2(add2(sub2(hi, sub2(s, c)), sub2(w, c)), w_lo));
    hi = s;
  }
  __device__ __forceinline__ void add(uint64_t w) {
    const uint64_t s = add2(hi, w), c = sub2(s, hi);
    lo = add2(lo, add2(sub2(hi, sub2(s, c)), sub2(w, c)));
    hi = s;
  }
};
__device__ __forceinline__ F2 shfl(F2 x, int from) {
  return F2{__shfl_sync(0xffffffffu, x.hi, from), __shfl_sync(0xffffffffu, x.lo, from)};
}
__device__ __forceinline__ F2 warp_incl(F2 x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const F2 y{__shfl_up_sync(0xffffffffu, x.hi, o), __shfl_up_sync(0xffffffffu, x.lo, o)};
    if (lane >= o) x = x + y;
  }
  return x;
}
// From inclusive to exclusive sums over the lanes.
__device__ __forceinline__ F2 before_lane(F2 incl) {
  const F2 y{__shfl_up_sync(0xffffffffu, incl.hi, 1), __shfl_up_sync(0xffffffffu, incl.lo, 1)};
  return (threadIdx.x & 31) ? y : F2{};
}
// u R (the product of the high parts without error)
__device__ __forceinline__ F2 scaled(F2 r, float u) {
  const float p = u * r.hi;
  return F2{p, 0.f} + F2{fmaf(u, r.hi, -p) + u * r.lo, 0.f};
}
// u q < p, exactly
__device__ __forceinline__ bool takes(float u, float q, float p) {
  const float x = u * q;
  if (fabsf(x) < 1e-25f) return static_cast<double>(u) * static_cast<double>(q) < static_cast<double>(p);
  return x < p || (x == p && fmaf(u, q, -x) < 0.f);      // (the product's error is a float)
}

constexpr int kMostRegions = kMostCtas * kWarps, kPerLane = kMostRegions / 32;
struct Smem {
  F2 region[2][kMostRegions];     // by round: the sums of the cluster's warps
  F2 block[kWarps];
  int found, last;
};

__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void store_to_cta(F2* p, uint32_t rank, F2 x) {
  asm volatile("{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %0, %1;\n st.shared::cluster.v2.f32 [a], {%2, %3};\n}\n" ::"r"(
                   smem_u32(p)),
               "r"(rank), "f"(x.hi), "f"(x.lo)
               : "memory");
}

// A vocabulary row as 16-byte vectors: vector k holds values k PER - m .. k PER - m + PER - 1, where m is
// the row's distance from a 16-byte boundary.
template <typename T>
struct Row {
  const T* p;
  int V, m;
  bool wide;         // vectors lie on 16-byte boundaries
  // vector k; zeros outside the row
  __device__ __forceinline__ uint4 vec(int k) const {
    constexpr int PER = Prob<T>::PER;
    const int v0 = k * PER - m;
    if (wide && v0 >= 0 && v0 + PER <= V) return gload(reinterpret_cast<const uint4*>(p + v0));
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int v = v0 + i;
      if (v < 0 || v >= V) continue;
      const uint32_t bits = __float_as_uint(Prob<T>::load(p + v));
      if constexpr (PER == 4) w[i] = bits;
      else w[i / 2] |= i & 1 ? bits : bits >> 16;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

template <typename T, bool DRAFT>
__global__ void __launch_bounds__(kThreads) verify_kernel(const __grid_constant__ Verify a, int n_cta, int sole,
                                                          uint32_t* status) {
  constexpr int PER = Prob<T>::PER;
  __shared__ Smem sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x / n_cta, rank = blockIdx.x - t * n_cta;
  const int d = a.n_draft;
  grid_trigger();
  grid_wait();
  const auto length = [&](int seq, uint32_t& bits) {
    const int n = a.draft_len ? gload(a.draft_len + seq) : d;
    if (n < 0 || n > d) bits |= DEV_ERR_RANGE;
    return max(0, min(n, d));
  };
  if (t == a.n_seq) {          // the cluster that checks
    if (rank == 0)
      sole_status(status, sole, [&](int i) {
        uint32_t bits = 0;
        const int seq = d ? i / d : i, k = d ? i - seq * d : 0;
        const int n = length(seq, bits);
        if (k != 0) bits = 0;                  // (counted once)
        if (k < n && static_cast<uint32_t>(gload(a.tokens + i)) >= static_cast<uint32_t>(a.vocab)) bits |= DEV_ERR_BAD_INDEX;
        return bits;
      });
    return;
  }
  const T* target = static_cast<const T*>(a.target) + static_cast<size_t>(t) * (d + 1) * a.target_stride;
  const T* draft = DRAFT ? static_cast<const T*>(a.draft) + static_cast<size_t>(t) * d * a.draft_stride : nullptr;
  const int32_t* tokens = a.tokens + static_cast<size_t>(t) * d;
  uint32_t bits = 0;
  const int len = length(t, bits);

  // the drafts that are taken, each warp for itself
  int n_ok = 0, x_end = -1;
#pragma unroll 1
  for (int i0 = 0; i0 < len; i0 += 32) {
    const int i = i0 + lane;
    bool ok = true;
    int x = -1;
    if (i < len) {
      x = gload(tokens + i);
      const float u = gload(a.u_accept + static_cast<size_t>(t) * d + i);
      ok = static_cast<uint32_t>(x) < static_cast<uint32_t>(a.vocab);
      if (ok) {
        const float p = Prob<T>::load(target + i * a.target_stride + x);
        const float q = DRAFT ? Prob<T>::load(draft + i * a.draft_stride + x) : 1.f;
        ok = takes(u, q, p);
      } else {
        bits |= DEV_ERR_BAD_INDEX;
      }
    }
    const uint32_t no = __ballot_sync(0xffffffffu, !ok);
    n_ok = min(len, i0 + 32);
    if (no) {
      n_ok = i0 + __ffs(no) - 1;
      x_end = __shfl_sync(0xffffffffu, x, __ffs(no) - 1);
      break;
    }
  }
  const bool rejected = n_ok < len;
  if (!sole && rank == 0 && warp == 0) {
    // (one more look, at every draft: those behind the first that is refused are not looked at above)
    uint32_t count = lane == 0 && (bits & DEV_ERR_RANGE) ? 1u : 0u;
    bits &= DEV_ERR_RANGE;
#pragma unroll 1
    for (int i = lane; i < len; i += 32)
      if (static_cast<uint32_t>(gload(tokens + i)) >= static_cast<uint32_t>(a.vocab)) {
        bits |= DEV_ERR_BAD_INDEX;
        ++count;
      }
    if (count) {
      atomicOr(status, bits);
      atomicAdd(status + 1, count);
    }
  }
  int32_t* out = a.tokens_out + static_cast<size_t>(t) * (d + 1);
  if (rank == 0) {
    if (threadIdx.x == 0) a.n_accepted[t] = n_ok;
#pragma unroll 1
    for (int i = threadIdx.x; i <= d; i += kThreads)
      if (i != n_ok) out[i] = i < n_ok ? gload(tokens + i) : -1;
  }

  // the row that the last token is drawn from
  Row<T> P{target + static_cast<size_t>(n_ok) * a.target_stride, a.vocab, 0, true}, Q{nullptr, a.vocab, 0, false};
  P.m = static_cast<int>((reinterpret_cast<uintptr_t>(P.p) & 15) / sizeof(T));
  bool use_q = DRAFT && rejected;
  if (use_q) {
    Q.p = draft + static_cast<size_t>(n_ok) * a.draft_stride;
    Q.m = P.m;
    Q.wide = ((reinterpret_cast<uintptr_t>(Q.p) ^ reinterpret_cast<uintptr_t>(P.p)) & 15) == 0;
  }
  int skip = !DRAFT && rejected ? x_end : -1;      // a draft without probabilities: all of its weight on its token
  const int n_vec = (a.vocab + P.m + PER - 1) / PER;
  const int per = (n_vec + n_cta * kWarps - 1) / (n_cta * kWarps);      // vectors of a region
  const float u = gload(a.u_sample + t);
  // Vector k of the target's row, without the token that takes no part.
  const auto target_vec = [&](int k) {
    uint4 v = P.vec(k);
    if constexpr (!DRAFT) {
      const int i = skip + P.m - k * PER;
      if (skip >= 0 && i >= 0 && i < PER) {
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < PER; ++j)
          if (j == i) w[j * 4 / PER] &= PER == 4 ? 0u : j & 1 ? 0xFFFFu : 0xFFFF0000u;
        v = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    return v;
  };

  // Twice where the draft's distribution covers the target's and no weight is left: then from the target's.
#pragma unroll 1
  for (int round = 0; round < 2; ++round) {
    const int lo = min(n_vec, (rank * kWarps + warp) * per), hi = min(n_vec, lo + per);
    Sums sums{};
    constexpr int U = 4;                 // vectors in flight
#pragma unroll 1
    for (int k0 = lo + lane; k0 < hi; k0 += 32 * U) {
      uint4 pv[U], qv[U];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        pv[j] = qv[j] = make_uint4(0u, 0u, 0u, 0u);
        const int k = k0 + 32 * j;
        if (k < hi) {
          pv[j] = target_vec(k);
          if (DRAFT && use_q) qv[j] = Q.vec(k);
        }
      }
#pragma unroll
      for (int j = 0; j < U; ++j) {
#pragma unroll
        for (int i = 0; i < PER; i += 2) {
          const float p0 = fmaxf(Prob<T>::get(pv[j], i), 0.f), p1 = fmaxf(Prob<T>::get(pv[j], i + 1), 0.f);
          const uint64_t p = pair(p0, p1);
          if constexpr (DRAFT) {               // (weight, twice)
            const uint64_t q = pair(fminf(Prob<T>::get(qv[j], i), p0), fminf(Prob<T>::get(qv[j], i + 1), p1));
            const uint64_t r = sub2(p, q);
            sums.add(r, sub2(sub2(p, r), q));
          } else {
            sums.add(p);
          }
        }
      }
    }
    const float2 hi2 = unpair(sums.hi), lo2 = unpair(sums.lo);
    F2 sum = (F2{hi2.x, 0.f} + F2{hi2.y, 0.f}) + (F2{lo2.x, 0.f} + F2{lo2.y, 0.f});
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      sum = sum + F2{__shfl_xor_sync(0xffffffffu, sum.hi, o), __shfl_xor_sync(0xffffffffu, sum.lo, o)};
    if (lane < n_cta) store_to_cta(&sh.region[round][rank * kWarps + warp], lane, sum);
    if (threadIdx.x == 0) {
      sh.found = INT_MAX;
      sh.last = -1;
    }
    cluster_sync_all();
    // The region that holds the first point above u R: every warp for itself, a lane kPerLane regions.  Where
    // rounding leaves none, the last region of any weight.
    F2 incl[kPerLane], run{};
    bool some[kPerLane];
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      const int g = lane * kPerLane + i;
      const F2 x = g < n_cta * kWarps ? sh.region[round][g] : F2{};
      some[i] = !(x.hi == 0.f);          // (a NaN: an infinite probability)
      run = run + x;
      incl[i] = run;
    }
    const F2 all = warp_incl(run), before = before_lane(all);
    const F2 R = shfl(all, 31);
    const F2 at = u > 0.f ? scaled(R, u) : F2{};
    int first = kPerLane, last_some = -1;
#pragma unroll
    for (int i = kPerLane - 1; i >= 0; --i) {
      if (some[i] && before + incl[i] > at) first = i;
      if (some[i] && last_some < 0) last_some = i;
    }
    const uint32_t over = __ballot_sync(0xffffffffu, first < kPerLane), any = __ballot_sync(0xffffffffu, last_some >= 0);
    if (any == 0) {
      if (round == 0 && (use_q || skip >= 0)) {
        use_q = false;
        skip = -1;
        continue;
      }
      if (rank == 0 && threadIdx.x == 0) out[n_ok] = -1;
      return;
    }
    if (!(R.hi < INFINITY)) {            // no draw
      if (rank == 0 && threadIdx.x == 0) out[n_ok] = -1;
      return;
    }
    const int owner = over ? __ffs(over) - 1 : 31 - __clz(any);
    const int pick = over ? first : last_some;
    const int region = owner * kPerLane + __shfl_sync(0xffffffffu, pick, owner);
    if (region / kWarps != rank) return;
    F2 mine = before;
#pragma unroll
    for (int i = 0; i < kPerLane - 1; ++i)
      if (i == pick - 1) mine = before + incl[i];
    F2 base = shfl(mine, owner);           // what lies before the region
    const int from = min(n_vec, region * per), to = min(n_vec, from + per);
#pragma unroll 1
    for (int b = from; b < to; b += kThreads) {
      const int k = b + static_cast<int>(threadIdx.x);
      uint4 pv = make_uint4(0u, 0u, 0u, 0u), qv = pv;
      if (k < to) {
        pv = target_vec(k);
        if (DRAFT && use_q) qv = Q.vec(k);
      }
      const auto at_place = [&](int i) { return weight(Prob<T>::get(pv, i), DRAFT ? Prob<T>::get(qv, i) : 0.f); };
      F2 here{};
#pragma unroll
      for (int i = 0; i < PER; ++i) here = here + at_place(i);
      const F2 in_warp = warp_incl(here), skipped = before_lane(in_warp);
      if (lane == 31) sh.block[warp] = in_warp;
      __syncthreads();
      const F2 blocks = warp_incl(lane < kWarps ? sh.block[lane] : F2{});
      F2 at_here = base + skipped;
      if (warp > 0) at_here = at_here + shfl(blocks, warp - 1);
      int found = INT_MAX, last = -1;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const F2 w = at_place(i);
        if (w.hi > 0.f) {
          at_here = at_here + w;
          last = k * PER - P.m + i;
          if (found == INT_MAX && at_here > at) found = last;
        }
      }
      found = __reduce_min_sync(0xffffffffu, found);
      last = __reduce_max_sync(0xffffffffu, last);
      if (lane == 0) {
        if (found != INT_MAX) atomicMin(&sh.found, found);
        if (last >= 0) atomicMax(&sh.last, last);
      }
      base = base + shfl(blocks, 31);
      __syncthreads();
      if (sh.found != INT_MAX) break;
    }
    if (threadIdx.x == 0) out[n_ok] = sh.found != INT_MAX ? sh.found : sh.last;
    return;
  }
}

template <typename T>
cudaError_t launch_t(const Verify& a, uint32_t* status, cudaStream_t st) {
  const int n = std::max(a.n_draft, 1);
  const bool sole = static_cast<long long>(a.n_seq) * n <= kSoleMost;
  const cudaError_t e = sole ? cudaSuccess : clear_status(status, st);
  if (e != cudaSuccess) return e;
  // As many CTAs a sequence as leave all sequences resident at once, so that none waits for another's chain of loads
  // (131072 values, fp32: 40 sequences, clusters of seven 25.8 us, of six 19.6; 64, of four 23.7, of five 29.8; 100, of
  // three 37.0, of two 31.9), and 4096 values or more each.
  int sms = device_sm_count();
  if (sms <= 0) sms = 152;
  const int fit = 2 * sms / std::max(1, std::min(a.n_seq, 2 * sms));
  int ctas = std::max(1, std::min({kMostCtas, fit, (a.vocab + 4095) / 4096}));
  const auto go = [&](auto kern) {
    constexpr auto k = decltype(kern)::value;
    while (ctas > 1 && resident_clusters<k>(ctas, kThreads, 0) < a.n_seq) --ctas;
    const unsigned grid = (static_cast<unsigned>(a.n_seq) + (sole ? 1u : 0u)) * static_cast<unsigned>(ctas);
    return launch_pdl(k, dim3(grid), kThreads, 0, st, ctas, a, ctas, sole ? a.n_seq * n : 0, status);
  };
  return a.draft ? go(Kernel<verify_kernel<T, true>>{}) : go(Kernel<verify_kernel<T, false>>{});
}

}  // namespace

cudaError_t launch_verify(const Verify& a, bool f32, uint32_t* status, cudaStream_t st) {
  return f32 ? launch_t<float>(a, status, st) : launch_t<__nv_bfloat16>(a, status, st);
}

}  // namespace dsa
