// quant8.cuh -- the 8-bit cache's codes and scales.
//
// A code is an e4m3 value or an int8 from -127 to 127; its block's scale is the
// power of two 2^(s - 127) of one byte s.  Being a power of two it costs the
// codes nothing but range: code * scale is exact in the cache's 16-bit type for
// every scale that the store writes, and an e4m3 code moves to a larger scale
// without a rounding unless it becomes subnormal.
#pragma once
#include <cuda_fp8.h>

#include "internal.h"
#include "maskattn.h"

namespace mab {

constexpr int SCALE_NAN = 255;  // a block into which a value that is not finite was written

// Scale byte of a block in units of the codes' type: the least that a block gets
// (below it a code's value may have no 16-bit form: 2^-24 is f16's least number,
// 2^-9 e4m3's; bf16's exponents go on far below any block that matters), and
// those from which on the largest codes' values would round past the type's
// largest finite number, with the magnitude that codes stop at there.
template <bool BF16, bool I8>
struct CodeRange {
  static constexpr int least = 127 + (BF16 ? -110 : I8 ? -24 : -15);
  static constexpr int big = 127 + (BF16 ? (I8 ? 122 : 120) : (I8 ? 10 : 8));
  static constexpr float big_top = I8 ? 63.f : 240.f;
};

// Least scale byte for which `amax` (finite) fits the codes: amax <= 448 * 2^e
// (448 = 1.75 * 2^8) or 127 * 2^e (127 = 1.984375 * 2^6).
template <bool BF16, bool I8>
__device__ __forceinline__ int scale_for(float amax) {
  const int bits = __float_as_int(amax);
  const int up = (bits & 0x7fffff) > (I8 ? 0x7e0000 : 0x600000) ? 1 : 0;
  return max((bits >> 23) - (I8 ? 6 : 8) + up, CodeRange<BF16, I8>::least);
}

__device__ __forceinline__ float exp2_int(int e) {  // 2^e, -127 <= e <= 127
  return __int_as_float(e == -127 ? 0x400000 : (e + 127) << 23);
}

// Four values in units of the scale to four codes (round to nearest even).
template <bool I8>
__device__ __forceinline__ uint32_t codes_of(float a, float b, float c, float d) {
  if (I8) {
    return (uint32_t)(__float2int_rn(a) & 0xff) | (uint32_t)(__float2int_rn(b) & 0xff) << 8 |
           (uint32_t)(__float2int_rn(c) & 0xff) << 16 | (uint32_t)__float2int_rn(d) << 24;
  }
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3) |
         (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3) << 16;
}

// A scale byte as a pair of the 16-bit type.  f16: exponents outside [-24, 15]
// count as the nearest of them; bf16: byte 0 counts as 1.
template <bool BF16>
__device__ __forceinline__ uint32_t scale_pair(int s) {
  uint32_t h;
  if (BF16) {
    h = (uint32_t)max(s, 1) << 7;
  } else {
    const int e = min(max(s - 127, -24), 15);
    h = e >= -14 ? (uint32_t)(e + 15) << 10 : 1u << (e + 24);
  }
  if (s == SCALE_NAN) h = 0x7fffu;
  return h | h << 16;
}

template <bool BF16>
__device__ __forceinline__ uint32_t mul16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  if (BF16)
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  else
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

template <bool BF16>
__device__ __forceinline__ uint32_t add16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  if (BF16)
    asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  else
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// e4m3 codes `lo` and `hi` (bytes of a, b) as a pair of bf16 values times 2^-120:
// sign, exponent and mantissa in their places.
__device__ __forceinline__ uint32_t code_bits(uint32_t a, uint32_t b, int lo, int hi) {
  // a byte at the head of each half, anything below it
  const uint32_t h = __byte_perm(a, b, (uint32_t)(lo << 4 | hi << 12));
  return ((h >> 4) & 0x07f007f0u) | (h & 0x80008000u);
}

// Codes `lo` and `hi` (bytes of the register pair a, b as __byte_perm counts
// them) as a pair of 16-bit values, exactly.
//   int8: the byte becomes the low bits of a number whose exponent makes its
//     unit 1 (f16: 1024 + (c + 128); bf16, which has seven bits below the first:
//     128 + the low seven), and what was added is taken off;
//   e4m3 to f16: the conversion; to bf16: code_bits, times 2^120.
template <bool BF16, bool I8>
__device__ __forceinline__ uint32_t code_pair(uint32_t a, uint32_t b, int lo, int hi) {
  if (I8) {
    // a byte at the foot of each half, anything above it
    const uint32_t u = __byte_perm(a, b, (uint32_t)(lo | hi << 8));
    if (!BF16) return add16x2<false>((u & 0x00ff00ffu) ^ 0x64806480u, 0xe480e480u);  // - 1152
    // 128 + low bits, less 128, or 256 for a set sign
    return add16x2<true>((u & 0x007f007fu) | 0x43004300u, (u & 0x00800080u) | 0xc300c300u);
  }
  if (!BF16) {
    uint32_t d;
    const uint16_t two = (uint16_t)__byte_perm(a, b, (uint32_t)(lo | hi << 4));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(two));
    return d;
  }
  return mul16x2<true>(code_bits(a, b, lo, hi), 0x7b807b80u);  // 2^120
}

// Four codes times their block's scale (a pair, scale_pair): exact for scales
// that the store writes.
template <bool BF16, bool I8>
__device__ __forceinline__ uint2 values_of(uint32_t codes, uint32_t scale2) {
  return make_uint2(mul16x2<BF16>(code_pair<BF16, I8>(codes, codes, 0, 1), scale2),
                    mul16x2<BF16>(code_pair<BF16, I8>(codes, codes, 2, 3), scale2));
}

// A scale byte as fp32 (the same numbers as scale_pair's).
template <bool BF16>
__device__ __forceinline__ float scale_float(int s) {
  const int e = BF16 ? max(s, 1) : min(max(s, 127 - 24), 127 + 15);
  return __int_as_float(s == SCALE_NAN ? 0x7fffffff : e << 23);
}

}  // namespace mab
