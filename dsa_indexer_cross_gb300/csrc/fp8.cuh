// The fp8 latent cache's number format.  A row's 512 latent dims are e4m3 codes with one scale
// byte b per 128 dims: code c stands for c * 2^(b - 127).  Power-of-two scales make every stored
// value exact in bf16 (4 significant bits), so reading the cache back, or multiplying its rows
// on the bf16 tensor cores, adds nothing to e4m3's own rounding (at most 2^-4 of the value).
//
// Encoding: b - 127 is the smallest integer e with amax <= 448 * 2^e, kept within [-100, 7]:
// the upper end keeps b + 120 a bf16 exponent, so decoding is one multiply (values past
// 448 * 2^7 saturate); the lower end only concerns groups whose largest value is under 2^-91.
// A group holding a NaN or an infinity is stored as b = 255, which reads back as NaN, as does
// any byte above 134.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp8.h>

namespace dsa {

constexpr int kScaleGroup = 128;          // latent dims per scale byte
constexpr uint32_t kScaleNaN = 255u;      // scale byte of a group with a NaN or an infinity
constexpr int kScaleMinExp = -100, kScaleMaxExp = 7;

// The multiplier of a scale byte, as a bf16 pair: 2^(b - 7), the 2^120 between an e4m3 code's
// bits read as bf16 (below) and its value included.
__device__ __forceinline__ uint32_t fp8_mult(uint32_t b) {
  const uint32_t h = b <= 134u ? (b + 120u) << 7 : 0x7FC0u;
  return h | (h << 16);
}

__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Four codes (one word) -> four bf16 values (two words), times the group's multiplier.  A byte
// permute sign-extends two codes to 16 bits; shifted left by four and masked, a code's exponent and
// mantissa bits lie at the low end of bf16's exponent field and the high end of its mantissa, its
// sign at the top: the code's value times 2^-120 (an e4m3 subnormal becomes a bf16 subnormal).  The
// multiply is exact.  Two integer-pipe instructions a pair (the shift is a multiply-add): the
// integer pipe runs at half rate and bounds a conversion that masks sign and magnitude apart.
__device__ __forceinline__ void fp8x4_to_bf16(uint32_t w, uint32_t mult, uint32_t& lo, uint32_t& hi) {
  uint32_t a, b;
  asm("prmt.b32 %0, %1, 0, 0x9180;" : "=r"(a) : "r"(w));
  asm("prmt.b32 %0, %1, 0, 0xB3A2;" : "=r"(b) : "r"(w));
  lo = bf16x2_mul((a * 16u) & 0x87F087F0u, mult);
  hi = bf16x2_mul((b * 16u) & 0x87F087F0u, mult);
}

// Scale byte of a group whose largest |value| has the bf16 bits `top` (sign cleared; NaN and
// infinity are 0x7F80 and above).
__device__ __forceinline__ uint32_t fp8_scale_byte(uint32_t top) {
  if (top >= 0x7F80u) return kScaleNaN;
  // top = 1.m * 2^(E - 127): 448 = 1.75 * 2^8, so e = E - 135, one more when 1.m > 1.75
  int e = static_cast<int>(top >> 7) - 135 + ((top & 0x7Fu) > 0x60u ? 1 : 0);
  e = max(kScaleMinExp, min(kScaleMaxExp, e));
  return static_cast<uint32_t>(e + 127);
}

// Two bf16 values (one word) -> two codes, values times inv = 2^-(b - 127), rounded to nearest
// even, saturating.
__device__ __forceinline__ uint32_t bf16x2_to_fp8(uint32_t v, float inv) {
  const float2 f = make_float2(__uint_as_float(v << 16) * inv, __uint_as_float(v & 0xFFFF0000u) * inv);
  return __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
}

}  // namespace dsa
