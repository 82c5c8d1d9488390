// Rotary positions of strided heads, and the paged latent cache's writing and reading back.
// All three move data once and compute next to nothing: HBM bandwidth bounds them at size, a
// launch's latency when small (64 tokens written 1.7 us in a graph, 64 tokens of 128 heads turned 2.0).
#include <cuda_bf16.h>

#include <algorithm>

#include "fp8.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace dsa {
namespace {

constexpr int kLat = 512;      // latent dims of a row
constexpr int kRope = 64;      // rotary dims of a row
constexpr int kRow = kLat + kRope;

// ---------------------------------------------------------------------------- element access
template <typename T>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
  static __device__ __forceinline__ float load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
  static constexpr int VEC = 8;
  static __device__ __forceinline__ void unpack(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Elem<float> {
  static __device__ __forceinline__ float load(const float* p) { return *p; }
  static __device__ __forceinline__ void store(float* p, float v) { *p = v; }
  static constexpr int VEC = 4;
  static __device__ __forceinline__ void unpack(const uint4& v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x);
    f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z);
    f[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};

// One pair turned by (cos, sin): fp32, one rounding per product sum.
__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
  const float u = fmaf(a, c, -(b * s)), v = fmaf(a, s, b * c);
  a = u;
  b = v;
}

// ---------------------------------------------------------------------------- status
// Small calls have no clearing pass before the kernel, which costs as much as the kernel itself (and 2
// of 27 us at 8000 tokens of 64 heads): block 0 checks every item and writes the status words, and
// nothing else touches them.  Larger calls (block 0's checks would outlast the other blocks' copies:
// 41 us for 32768 tokens written, 16 with the clearing pass) are launched behind a kernel that clears
// them, about 2 us less than a memset.  (Always clearing costs small calls a launch: one head of 2048
// tokens 6.7 -> 8.6 us.)
constexpr int kSoleMostRope = 16384, kSoleMostWrite = 4096, kSoleMostPages = 4096;

__device__ __forceinline__ void report(uint32_t* status, bool sole, uint32_t bits) {
  if (sole) return;
  atomicOr(status, bits);
  atomicAdd(status + 1, 1u);
}
__global__ void clear_status_kernel(uint32_t* status) {
  grid_trigger();
  grid_wait();
  status[threadIdx.x] = 0u;
}
cudaError_t clear_status(uint32_t* status, cudaStream_t st) {
  return launch_pdl(clear_status_kernel, dim3(1), 2, 0, st, 1, status);
}
// Block 0 of a call that writes the status words itself: check(i) gives item i's error bits.
template <typename F>
__device__ __forceinline__ void sole_status(uint32_t* status, int n, F check) {
  __shared__ uint32_t s_bits, s_count;
  if (threadIdx.x == 0) s_bits = s_count = 0u;
  __syncthreads();
  uint32_t bits = 0, count = 0;
  int i = threadIdx.x;
  for (; i + 7 * static_cast<int>(blockDim.x) < n; i += 8 * blockDim.x) {
#pragma unroll
    for (int u = 0; u < 8; ++u) {        // (eight items' loads in flight)
      const uint32_t e = check(i + u * blockDim.x);
      bits |= e;
      count += e ? 1u : 0u;
    }
  }
  for (; i < n; i += blockDim.x) {
    const uint32_t e = check(i);
    bits |= e;
    count += e ? 1u : 0u;
  }
  if (bits) {
    atomicOr(&s_bits, bits);
    atomicAdd(&s_count, count);
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    status[0] = s_bits;
    status[1] = s_count;
  }
}

// ---------------------------------------------------------------------------- rotary positions
// A thread turns one 16-byte vector (interleaved: its own pairs) or one vector of each half
// (half layout) of up to U heads of one token, so the token's (cos, sin) are loaded once for U
// heads and U independent loads are in flight.  Neighbouring threads take neighbouring
// vectors, then neighbouring heads.  The input is read once (ld.cs: 2 of 26 us at 8000 tokens
// of 64 heads, 133 MB, which take 23.5 in a graph: 5.7 TB/s); U = 2 and 8 and smaller blocks measured the same.
template <typename T, bool INTER, int U>
__global__ void __launch_bounds__(256) rope_apply_vec(const T* x, T* out, const int32_t* pos, const float2* cs,
                                                      int n_pos, uint32_t n_items, int n_heads, int head_groups,
                                                      int rope, long long x_tok, long long x_head, long long o_tok,
                                                      long long o_head, float sgn, uint32_t* status, int sole) {
  using E = Elem<T>;
  constexpr int V = E::VEC;
  constexpr int NP = INTER ? V / 2 : V;          // pairs of one head in this thread
  grid_trigger();
  grid_wait();
  if (sole && blockIdx.x == 0)
    sole_status(status, sole, [&](int t) {
      const int p = gload(pos + t);
      return p < 0 || p >= n_pos ? DEV_ERR_BAD_INDEX : 0u;
    });
  const uint32_t item = blockIdx.x * blockDim.x + threadIdx.x;
  if (item >= n_items) return;
  const uint32_t nv = static_cast<uint32_t>(rope) / (INTER ? V : 2 * V);
  const uint32_t v = item % nv, hg = (item / nv) % head_groups, t = item / (nv * head_groups);
  const int p = gload(pos + t);
  if (p < 0 || p >= n_pos) {
    if (v == 0 && hg == 0) report(status, sole != 0, DEV_ERR_BAD_INDEX);
    return;
  }
  const T* xt = x + static_cast<long long>(t) * x_tok + v * V;
  T* ot = out + static_cast<long long>(t) * o_tok + v * V;
  const int half = rope / 2;
  uint4 a[U], b[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = static_cast<int>(hg) + u * head_groups;
    if (h < n_heads) {
      a[u] = __ldcs(reinterpret_cast<const uint4*>(xt + h * x_head));
      if constexpr (!INTER) b[u] = __ldcs(reinterpret_cast<const uint4*>(xt + h * x_head + half));
    }
  }
  float c[NP], s[NP];
  const float4* ct = reinterpret_cast<const float4*>(cs + static_cast<size_t>(p) * half + v * NP);
#pragma unroll
  for (int i = 0; i < NP / 2; ++i) {
    const float4 q = gload(ct + i);
    c[2 * i] = q.x;
    s[2 * i] = q.y * sgn;
    c[2 * i + 1] = q.z;
    s[2 * i + 1] = q.w * sgn;
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = static_cast<int>(hg) + u * head_groups;
    if (h < n_heads) {
      float f[V];
      E::unpack(a[u], f);
      if constexpr (INTER) {
#pragma unroll
        for (int i = 0; i < NP; ++i) turn(f[2 * i], f[2 * i + 1], c[i], s[i]);
        *reinterpret_cast<uint4*>(ot + h * o_head) = E::pack(f);
      } else {
        float g[V];
        E::unpack(b[u], g);
#pragma unroll
        for (int i = 0; i < NP; ++i) turn(f[i], g[i], c[i], s[i]);
        *reinterpret_cast<uint4*>(ot + h * o_head) = E::pack(f);
        *reinterpret_cast<uint4*>(ot + h * o_head + half) = E::pack(g);
      }
    }
  }
}

// Any width, stride and alignment: one pair per thread.
template <typename T, bool INTER>
__global__ void __launch_bounds__(256) rope_apply_pair(const T* x, T* out, const int32_t* pos, const float2* cs,
                                                       int n_pos, uint32_t n_items, int n_heads, int rope,
                                                       long long x_tok, long long x_head, long long o_tok,
                                                       long long o_head, float sgn, uint32_t* status, int sole) {
  using E = Elem<T>;
  grid_trigger();
  grid_wait();
  if (sole && blockIdx.x == 0)
    sole_status(status, sole, [&](int t) {
      const int p = gload(pos + t);
      return p < 0 || p >= n_pos ? DEV_ERR_BAD_INDEX : 0u;
    });
  const uint32_t item = blockIdx.x * blockDim.x + threadIdx.x;
  if (item >= n_items) return;
  const uint32_t half = static_cast<uint32_t>(rope) / 2;
  const uint32_t i = item % half, h = (item / half) % n_heads, t = item / (half * n_heads);
  const int p = gload(pos + t);
  if (p < 0 || p >= n_pos) {
    if (i == 0 && h == 0) report(status, sole != 0, DEV_ERR_BAD_INDEX);
    return;
  }
  const uint32_t ia = INTER ? 2 * i : i, ib = INTER ? 2 * i + 1 : i + half;
  const T* xr = x + static_cast<long long>(t) * x_tok + static_cast<long long>(h) * x_head;
  T* orow = out + static_cast<long long>(t) * o_tok + static_cast<long long>(h) * o_head;
  float a = E::load(xr + ia), b = E::load(xr + ib);
  const float2 q = gload(cs + static_cast<size_t>(p) * half + i);
  turn(a, b, q.x, q.y * sgn);
  E::store(orow + ia, a);
  E::store(orow + ib, b);
}

// ---------------------------------------------------------------------------- writing rows
// The last 64 dims of one row, turned when ROT: lanes 0-7 hold one 16-byte vector each.  In the
// half layout lane l's partner vector is lane l ^ 4's.
template <bool ROT>
__device__ __forceinline__ uint4 rope_vec(uint4 v, int lane, bool inter, const float2* cs_row) {
  if constexpr (!ROT) {
    return v;
  } else {
    using E = Elem<__nv_bfloat16>;
    uint4 o;
    o.x = __shfl_xor_sync(0xffffffffu, v.x, 4);
    o.y = __shfl_xor_sync(0xffffffffu, v.y, 4);
    o.z = __shfl_xor_sync(0xffffffffu, v.z, 4);
    o.w = __shfl_xor_sync(0xffffffffu, v.w, 4);
    float f[8];
    E::unpack(v, f);
    const int l = lane & 7;
    if (inter) {
      const float4* ct = reinterpret_cast<const float4*>(cs_row + l * 4);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 q = gload(ct + i);
        turn(f[4 * i], f[4 * i + 1], q.x, q.y);
        turn(f[4 * i + 2], f[4 * i + 3], q.z, q.w);
      }
    } else {
      float g[8];
      E::unpack(o, g);
      const float4* ct = reinterpret_cast<const float4*>(cs_row + (l & 3) * 8);
      const bool second = l >= 4;          // f is the second half's vector, g the first's
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 q = gload(ct + i);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float c = e ? q.z : q.x, s = e ? q.w : q.y;
          float a = second ? g[2 * i + e] : f[2 * i + e], b = second ? f[2 * i + e] : g[2 * i + e];
          turn(a, b, c, s);
          f[2 * i + e] = second ? b : a;
        }
      }
    }
    return E::pack(f);
  }
}

// The largest magnitude of a vector's even and of its odd bf16 values, as bits.
__device__ __forceinline__ uint32_t abs_max(const uint4& v) {
  return __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu), __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
}
// Eight tokens a block.  Warps 0-7 take one token's latent dims each: lane l holds the row's 16-byte
// vectors l and l + 32 (dims 8l.. and 256 + 8l..), 16 lanes make a scale group, and every load and store
// instruction covers whole consecutive lines.  Warps 8-9 take the rotary dims of four tokens each, so the
// turn's chain of loads (position, table row) holds up no latent dims, and is not done four times over: 60000
// tokens to fp8, 124 MB, 24 us, where one warp a token took 31, and two or four tokens a warp 37 and 46;
// 32768 tokens, 67 MB, 11.5 us in a graph (5.9 TB/s of a copy's 6.8).
template <bool FP8, bool ROT>
__global__ void __launch_bounds__(320) cache_write_kernel(const uint16_t* kv, long long kv_stride,
                                                          const int32_t* slot, const int32_t* pos, const float2* cs,
                                                          int n_pos, int n_tokens, int n_rows, bool inter,
                                                          uint8_t* latent, uint8_t* scale, uint16_t* rope,
                                                          uint32_t* status, int sole) {
  grid_trigger();
  grid_wait();
  if (sole && blockIdx.x == 0)
    sole_status(status, sole, [&](int i) {
      const int s = gload(slot + i), p = ROT ? gload(pos + i) : 0;
      return s >= 0 && (s >= n_rows || (ROT && (p < 0 || p >= n_pos))) ? DEV_ERR_BAD_INDEX : 0u;
    });
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool turns = warp >= 8;
  const int t = blockIdx.x * 8 + (turns ? 4 * (warp - 8) + (lane >> 3) : warp);
  const int tt = min(t, n_tokens - 1);
  const uint4* src = reinterpret_cast<const uint4*>(kv + static_cast<long long>(tt) * kv_stride);
  // (fp8: marked as read once, 32768 tokens 15.3 -> 14.4 us; to bf16 16.4 -> 17.0)
  const auto load = [](const uint4* q) { return FP8 ? __ldcs(q) : gload(q); };
  const uint4 a = load(src + (turns ? 64 + (lane & 7) : lane));
  uint4 b;
  if (!turns) b = load(src + 32 + lane);
  const int s = t < n_tokens ? gload(slot + tt) : -1;
  const int p = ROT ? gload(pos + tt) : 0;
  const bool bad = s >= n_rows || (ROT && (p < 0 || p >= n_pos)), stored = s >= 0 && !bad;
  if (turns) {
    const uint4 turned = rope_vec<ROT>(a, lane, inter, cs + static_cast<size_t>(stored ? p : 0) * (kRope / 2));
    if (!stored) return;
    uint16_t* row = FP8 ? rope + static_cast<size_t>(s) * kRope
                        : reinterpret_cast<uint16_t*>(latent) + static_cast<size_t>(s) * kRow + kLat;
    reinterpret_cast<uint4*>(row)[lane & 7] = turned;
    return;
  }
  if (!stored) {
    if (s >= 0 && lane == 0) report(status, sole != 0, DEV_ERR_BAD_INDEX);
    return;
  }
  if constexpr (!FP8) {
    uint4* dst = reinterpret_cast<uint4*>(latent) + static_cast<size_t>(s) * (kRow / 8);
    dst[lane] = a;
    dst[32 + lane] = b;
  } else {
    // the two groups' largest magnitudes, as bits, in the halves of one word
    const uint32_t m0 = abs_max(a), m1 = abs_max(b);
    uint32_t tops = __vmaxu2(__byte_perm(m0, m1, 0x5410), __byte_perm(m0, m1, 0x7632));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) tops = __vmaxu2(tops, __shfl_xor_sync(0xffffffffu, tops, o));
    uint32_t sb[2];
    uint2 codes[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint4 v = k ? b : a;
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      sb[k] = fp8_scale_byte(k ? tops >> 16 : tops & 0xFFFFu);
      if (sb[k] == kScaleNaN) {
        codes[k] = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
      } else {
        const float inv = __uint_as_float((254u - sb[k]) << 23);     // 2^-(b - 127)
        codes[k].x = bf16x2_to_fp8(w[0], inv) | (bf16x2_to_fp8(w[1], inv) << 16);
        codes[k].y = bf16x2_to_fp8(w[2], inv) | (bf16x2_to_fp8(w[3], inv) << 16);
      }
    }
    uint2* dst = reinterpret_cast<uint2*>(latent + static_cast<size_t>(s) * kLat);
    dst[lane] = codes[0];
    dst[32 + lane] = codes[1];
    // groups 0 and 2 end in lane 0, groups 1 and 3 in lane 16
    const uint32_t b1 = __shfl_sync(0xffffffffu, sb[0], 16), b3 = __shfl_sync(0xffffffffu, sb[1], 16);
    if (lane == 0)
      *reinterpret_cast<uint32_t*>(scale + static_cast<size_t>(s) * 4) = sb[0] | (b1 << 8) | (sb[1] << 16) | (b3 << 24);
  }
}

// ---------------------------------------------------------------------------- reading rows back
// One block per kReadRows rows of a (sequence, page): its valid rows go to out rows row_start[t] + j.
// A warp takes four rows, all their loads before the first store.  1.08 M rows of fp8, 1.9 GB moved:
// 286 us, 6.8 TB/s, what a copy reaches.
constexpr int kReadRows = 32;
constexpr int kReadSplit = kPageRows / kReadRows;
template <bool FP8>
__global__ void __launch_bounds__(256) cache_read_kernel(const uint8_t* latent, const uint8_t* scale,
                                                         const uint16_t* rope, const PagedRows pg,
                                                         const int32_t* row_start, int n_out, uint16_t* out,
                                                         uint32_t* status, int sole) {
  const int cap = pg.max_pages << kPageShift;
  // valid rows of a page, its physical page and its first output row; the error bits, if any
  auto place = [&](int blk, int& n, int& page, long long& o0) -> uint32_t {
    const int t = blk / pg.max_pages, pl = blk % pg.max_pages;
    const int want = gload(pg.seq_len + t);
    const uint32_t range = pl == 0 && (want < 0 || want > cap) ? DEV_ERR_RANGE : 0u;
    n = min(min(want, cap) - (pl << kPageShift), kPageRows);
    if (n <= 0) return range;
    page = gload(pg.block_table + static_cast<size_t>(t) * pg.max_pages + pl);
    o0 = static_cast<long long>(gload(row_start + t)) + (pl << kPageShift);
    return range | (page < 0 || page >= pg.n_pages || o0 < 0 || o0 + n > n_out ? DEV_ERR_BAD_INDEX : 0u);
  };
  int n = 0, page = 0;
  long long o0 = 0;
  grid_trigger();
  grid_wait();
  if (sole && blockIdx.x == 0) sole_status(status, sole, [&](int b) { return place(b, n, page, o0); });
  const uint32_t err = place(blockIdx.x / kReadSplit, n, page, o0);
  const int part = blockIdx.x % kReadSplit * kReadRows;
  if (err && part == 0 && threadIdx.x == 0) report(status, sole != 0, err);
  n = min(n - part, kReadRows);
  if (n <= 0 || (err & DEV_ERR_BAD_INDEX)) return;
  o0 += part;
  const size_t row0 = (static_cast<size_t>(page) << kPageShift) + part;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint4* dst = reinterpret_cast<uint4*>(out + static_cast<size_t>(o0) * kRow);
  if constexpr (!FP8) {
    // rows are contiguous on both sides
    const uint4* src = reinterpret_cast<const uint4*>(latent) + row0 * (kRow / 8);
    const int total = n * (kRow / 8);
    for (int e = threadIdx.x; e < total; e += 4 * 256) {
      uint4 v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (e + 256 * k < total) v[k] = gload(src + e + 256 * k);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (e + 256 * k < total) dst[e + 256 * k] = v[k];
    }
  } else {
    const int r0 = warp * 4;
    static_assert(kReadRows == 32, "eight warps of four rows");
    if (r0 < n) {
      uint2 c[4][2];
      uint32_t sc[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const size_t row = row0 + min(r0 + k, n - 1);
        const uint2* src = reinterpret_cast<const uint2*>(latent + row * kLat);
        c[k][0] = gload(src + lane);
        c[k][1] = gload(src + 32 + lane);
        sc[k] = gload(reinterpret_cast<const uint32_t*>(scale) + row);
      }
      const int rr = r0 + (lane >> 3);        // the four rows' rotary dims, eight lanes each
      const uint4 rv = gload(reinterpret_cast<const uint4*>(rope + (row0 + min(rr, n - 1)) * kRope) + (lane & 7));
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (r0 + k >= n) continue;
        uint4* d = dst + static_cast<size_t>(r0 + k) * (kRow / 8);
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const uint32_t m = fp8_mult((sc[k] >> (16 * g + (lane >= 16 ? 8 : 0))) & 0xFFu);
          uint4 o;
          fp8x4_to_bf16(c[k][g].x, m, o.x, o.y);
          fp8x4_to_bf16(c[k][g].y, m, o.z, o.w);
          d[32 * g + lane] = o;
        }
      }
      if (rr < n) dst[static_cast<size_t>(rr) * (kRow / 8) + 64 + (lane & 7)] = rv;
    }
  }
}

template <typename T, bool INTER>
cudaError_t launch_rope_t(const RopeApply& a, const int32_t* pos, const float* cs, int n_pos, uint32_t* status,
                          cudaStream_t st) {
  constexpr int V = Elem<T>::VEC;
  constexpr int U = 4;
  const auto mult = [](long long s) { return s % V == 0; };
  const bool vec = a.rope % (INTER ? V : 2 * V) == 0 && mult(a.x_tok) && mult(a.x_head) && mult(a.o_tok) &&
                   mult(a.o_head) && (reinterpret_cast<uintptr_t>(a.x) & 15) == 0 &&
                   (reinterpret_cast<uintptr_t>(a.out) & 15) == 0;
  const int groups = vec ? (a.n_heads + U - 1) / U : a.n_heads;
  const long long per = static_cast<long long>(groups) * (vec ? a.rope / (INTER ? V : 2 * V) : a.rope / 2);
  // thread indices are 32-bit: larger problems go in several launches
  const int most = static_cast<int>(std::max(1LL, std::min<long long>(a.n_tokens, kRopeMostPairs / per)));
  const float sgn = a.inverse ? -1.f : 1.f;
  const int sole = a.n_tokens <= std::min(kSoleMostRope, most) ? a.n_tokens : 0;      // (one launch)
  cudaError_t e = sole ? cudaSuccess : clear_status(status, st);
  if (e != cudaSuccess) return e;
  for (long long t0 = 0; t0 < a.n_tokens; t0 += most) {      // (t0 + most may pass 32 bits)
    const int n = static_cast<int>(std::min<long long>(most, a.n_tokens - t0));
    const uint32_t items = static_cast<uint32_t>(per * n);
    const unsigned grid = (items + 255) / 256;
    const T* x = static_cast<const T*>(a.x) + t0 * a.x_tok;
    T* out = static_cast<T*>(a.out) + t0 * a.o_tok;
    const float2* c2 = reinterpret_cast<const float2*>(cs);
    e = vec ? launch_pdl(rope_apply_vec<T, INTER, U>, dim3(grid), 256, 0, st, 1, x, out, pos + t0, c2, n_pos, items,
                         a.n_heads, groups, a.rope, a.x_tok, a.x_head, a.o_tok, a.o_head, sgn, status, sole)
            : launch_pdl(rope_apply_pair<T, INTER>, dim3(grid), 256, 0, st, 1, x, out, pos + t0, c2, n_pos, items,
                         a.n_heads, a.rope, a.x_tok, a.x_head, a.o_tok, a.o_head, sgn, status, sole);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_rope_apply(const RopeApply& a, const int32_t* pos, const float* cs, int n_pos, uint32_t* status,
                              cudaStream_t st) {
  if (a.f32)
    return a.interleaved ? launch_rope_t<float, true>(a, pos, cs, n_pos, status, st)
                         : launch_rope_t<float, false>(a, pos, cs, n_pos, status, st);
  return a.interleaved ? launch_rope_t<__nv_bfloat16, true>(a, pos, cs, n_pos, status, st)
                       : launch_rope_t<__nv_bfloat16, false>(a, pos, cs, n_pos, status, st);
}

cudaError_t launch_cache_write(const LatentCache& c, const void* kv, long long kv_stride, const int32_t* slot,
                               const int32_t* pos, const float* cs, int n_pos, int n_tokens, bool interleaved,
                               uint32_t* status, cudaStream_t st) {
  const unsigned grid = (static_cast<unsigned>(n_tokens) + 7) / 8;
  const int sole = n_tokens <= kSoleMostWrite ? n_tokens : 0;
  const cudaError_t e = sole ? cudaSuccess : clear_status(status, st);
  if (e != cudaSuccess) return e;
  const auto go = [&](auto kern) {
    return launch_pdl(kern, dim3(grid), 320, 0, st, 1, static_cast<const uint16_t*>(kv), kv_stride, slot, pos,
                      reinterpret_cast<const float2*>(cs), n_pos, n_tokens, c.n_rows, interleaved, c.latent, c.scale,
                      c.rope, status, sole);
  };
  if (c.fp8) return cs ? go(cache_write_kernel<true, true>) : go(cache_write_kernel<true, false>);
  return cs ? go(cache_write_kernel<false, true>) : go(cache_write_kernel<false, false>);
}

cudaError_t launch_cache_read(const LatentCache& c, const PagedRows& pg, int n_seq, const int32_t* row_start, int n_out,
                              void* out, uint32_t* status, cudaStream_t st) {
  const unsigned n_pg = static_cast<unsigned>(n_seq) * static_cast<unsigned>(pg.max_pages);   // < 2^29: the ABI's check
  const unsigned grid = n_pg * kReadSplit;
  const int sole = n_pg <= kSoleMostPages ? static_cast<int>(n_pg) : 0;
  const cudaError_t e = sole ? cudaSuccess : clear_status(status, st);
  if (e != cudaSuccess) return e;
  return launch_pdl(c.fp8 ? cache_read_kernel<true> : cache_read_kernel<false>, dim3(grid), 256, 0, st, 1, c.latent,
                    c.scale, c.rope, pg, row_start, n_out, static_cast<uint16_t*>(out), status, sole);
}

}  // namespace dsa
