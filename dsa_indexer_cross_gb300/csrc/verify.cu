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
// apart, so single precision would draw a neighbour now and then.  A thread keeps its sum as two floats
// (the error of each addition, and of p - q, is known exactly from a few more additions), some 48 bits;
// warps, CTAs and the region that is read again add in double precision, which this GPU is slow at but
// which is then a few hundred additions.
//
// What bounds it: see launch_verify.
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

// A thread's sum of weights: hi + lo, good to some 2^-46 of it.
struct Sum2 {
  float hi = 0.f, lo = 0.f;
  // adds p - q where it is positive (a NaN is not)
  __device__ __forceinline__ void add(float p, float q) {
    const float r = p - q;
    if (!(r > 0.f)) return;
    const float b = r - p;
    const float e1 = (p - (r - b)) - (q + b);            // p - q = r + e1
    const float s = hi + r, c = s - hi;
    const float e2 = (hi - (s - c)) + (r - c);           // hi + r = s + e2
    hi = s;
    lo += e1 + e2;
  }
};

struct Smem {
  double part[2][kMostCtas];      // by round: the CTAs' sums
  double warp[kWarps];
  double block[kWarps];
  int found, last;
};

__device__ __forceinline__ double warp_incl(double x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}
// Which of the `n` parts (lane c holds part c's sum x; `before`: what lies before part 0) holds the first
// point above `at`; the last part with any weight where rounding leaves none, -1 where no part has any.
// `start`: what lies before the part chosen.
__device__ __forceinline__ int pick(double x, double before, double at, double& start) {
  const double incl = before + warp_incl(x);
  double excl = __shfl_up_sync(0xffffffffu, incl, 1);
  if ((threadIdx.x & 31) == 0) excl = before;
  const uint32_t some = __ballot_sync(0xffffffffu, x > 0.0);
  const uint32_t over = __ballot_sync(0xffffffffu, x > 0.0 && incl > at);
  const int c = over ? __ffs(over) - 1 : 31 - __clz(some);
  start = __shfl_sync(0xffffffffu, excl, max(c, 0));
  return some ? c : -1;
}

__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void store_to_cta(double* p, uint32_t rank, double x) {
  asm volatile("{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %0, %1;\n st.shared::cluster.f64 [a], %2;\n}\n" ::"r"(smem_u32(p)),
               "r"(rank), "d"(x)
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
        ok = static_cast<double>(u) * static_cast<double>(q) < static_cast<double>(p);     // (exact)
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
  const auto weigh = [&](const uint4& pv, const uint4& qv, int k, auto&& each) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      float p = Prob<T>::get(pv, i);
      if (!DRAFT && k * PER - P.m + i == skip) p = 0.f;
      each(i, p, DRAFT ? Prob<T>::get(qv, i) : 0.f);
    }
  };

  // Twice where the draft's distribution covers the target's and no weight is left: then from the target's.
#pragma unroll 1
  for (int round = 0; round < 2; ++round) {
    const int lo = min(n_vec, (rank * kWarps + warp) * per), hi = min(n_vec, lo + per);
    Sum2 sum;
    constexpr int U = 4;                 // vectors in flight
#pragma unroll 1
    for (int k0 = lo + lane; k0 < hi; k0 += 32 * U) {
      uint4 pv[U], qv[U];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        pv[j] = qv[j] = make_uint4(0u, 0u, 0u, 0u);
        const int k = k0 + 32 * j;
        if (k < hi) {
          pv[j] = P.vec(k);
          if (DRAFT && use_q) qv[j] = Q.vec(k);
        }
      }
#pragma unroll
      for (int j = 0; j < U; ++j) weigh(pv[j], qv[j], k0 + 32 * j, [&](int, float p, float q) { sum.add(p, q); });
    }
    double x = static_cast<double>(sum.hi) + static_cast<double>(sum.lo);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if (lane == 0) sh.warp[warp] = x;
    __syncthreads();
    if (warp == 0) {
      x = lane < kWarps ? sh.warp[lane] : 0.0;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
      if (lane < n_cta) store_to_cta(&sh.part[round][rank], lane, x);
    }
    if (threadIdx.x == 0) {
      sh.found = INT_MAX;
      sh.last = -1;
    }
    cluster_sync_all();
    // the CTA, the warp's region
    x = lane < n_cta ? sh.part[round][lane] : 0.0;
    const double R = __shfl_sync(0xffffffffu, warp_incl(x), 31);
    const double at = u > 0.f ? static_cast<double>(u) * R : 0.0;
    double start;
    const int c = pick(x, 0.0, at, start);
    if (!(R < INFINITY)) {               // an infinite probability: no draw
      if (rank == 0 && threadIdx.x == 0) out[n_ok] = -1;
      return;
    }
    if (c < 0) {
      if (round == 0 && (use_q || skip >= 0)) {
        use_q = false;
        skip = -1;
        continue;
      }
      if (rank == 0 && threadIdx.x == 0) out[n_ok] = -1;
      return;
    }
    if (c != rank) return;
    double base;
    const int w = pick(lane < kWarps ? sh.warp[lane] : 0.0, start, at, base);
    const int from = min(n_vec, (rank * kWarps + w) * per), to = min(n_vec, from + per);
#pragma unroll 1
    for (int b = from; b < to; b += kThreads) {
      const int k = b + static_cast<int>(threadIdx.x);
      uint4 pv = make_uint4(0u, 0u, 0u, 0u), qv = pv;
      if (k < to) {
        pv = P.vec(k);
        if (DRAFT && use_q) qv = Q.vec(k);
      }
      double r[PER], mine = 0.0;
      weigh(pv, qv, k, [&](int i, float p, float q) {
        r[i] = p > q ? static_cast<double>(p) - static_cast<double>(q) : 0.0;
        mine += r[i];
      });
      const double incl = warp_incl(mine);
      if (lane == 31) sh.block[warp] = incl;
      __syncthreads();
      const double all = warp_incl(lane < kWarps ? sh.block[lane] : 0.0);
      double before = __shfl_sync(0xffffffffu, all, max(warp - 1, 0));
      if (warp == 0) before = 0.0;
      double run = base + before + (incl - mine);
      int found = INT_MAX, last = -1;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        run += r[i];
        if (r[i] > 0.0) {
          last = k * PER - P.m + i;
          if (found == INT_MAX && run > at) found = last;
        }
      }
      found = __reduce_min_sync(0xffffffffu, found);
      last = __reduce_max_sync(0xffffffffu, last);
      if (lane == 0) {
        if (found != INT_MAX) atomicMin(&sh.found, found);
        if (last >= 0) atomicMax(&sh.last, last);
      }
      base += __shfl_sync(0xffffffffu, all, 31);
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
  int sms = device_sm_count();
  if (sms <= 0) sms = 152;
  int ctas = kMostCtas;
  while (ctas > 1 && (static_cast<long long>(a.n_seq) * ctas > 4 * sms || a.vocab < 1024 * ctas)) ctas >>= 1;
  const unsigned grid = (static_cast<unsigned>(a.n_seq) + (sole ? 1u : 0u)) * static_cast<unsigned>(ctas);
  return launch_pdl(a.draft ? verify_kernel<T, true> : verify_kernel<T, false>, dim3(grid), kThreads, 0, st, ctas, a, ctas,
                    sole ? a.n_seq * n : 0, status);
}

}  // namespace

cudaError_t launch_verify(const Verify& a, bool f32, uint32_t* status, cudaStream_t st) {
  return f32 ? launch_t<float>(a, status, st) : launch_t<__nv_bfloat16>(a, status, st);
}

}  // namespace dsa
