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
    // 1.5 * 2^23 has a unit of 1 in its last place: the sum's rounding is the code's,
    // and its low byte the code (conversions go at a quarter of the adds' rate)
    constexpr float UNIT = 12582912.f;
    const uint32_t lo = __byte_perm(__float_as_uint(a + UNIT), __float_as_uint(b + UNIT), 0x0040);
    const uint32_t hi = __byte_perm(__float_as_uint(c + UNIT), __float_as_uint(d + UNIT), 0x0040);
    return __byte_perm(lo, hi, 0x5410);
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

// (w & mask) | set in one instruction (the compiler takes two for two constants).
__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t mask, uint32_t set) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(d) : "r"(w), "r"(mask), "r"(set));
  return d;
}
// int8 codes at the foot of w's halves as bf16: 128 + the low bits, less 128, or 256
// for a set sign.
__device__ __forceinline__ uint32_t bf16_of_i8(uint32_t w) {
  return add16x2<true>(and_or(w, 0x007f007fu, 0x43004300u), and_or(w, 0x00800080u, 0xc300c300u));
}

// Codes to 16-bit values, exactly.
//   int8: the byte becomes the low bits of a number whose exponent makes its
//     unit 1 (f16: 1024 + (c + 128); bf16, which has seven bits below the first:
//     128 + the low seven), and what was added is taken off;
//   e4m3 to f16: the conversion; to bf16: sign, exponent and mantissa moved to
//     their places, which leaves the exponent 120 too small (BITS: left so).

// The four codes of a word as pairs (0, 1) and (2, 3).
template <bool BF16, bool I8>
__device__ __forceinline__ uint2 word_pairs(uint32_t w) {
  if (I8 && !BF16) {
    const uint32_t u = w ^ 0x80808080u;
    return make_uint2(add16x2<false>(__byte_perm(u, 0x64646464u, 0x4140), 0xe480e480u),
                      add16x2<false>(__byte_perm(u, 0x64646464u, 0x4342), 0xe480e480u));
  }
  if (I8) {
    return make_uint2(bf16_of_i8(__byte_perm(w, 0, 0x4140)),
                      bf16_of_i8(__byte_perm(w, 0, 0x4342)));
  }
  if (!BF16) {
    uint2 d;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(d.x), "=r"(d.y)
        : "r"(w));
    return d;
  }
  const uint32_t a = __byte_perm(w, 0, 0x1404), b = __byte_perm(w, 0, 0x3424);
  return make_uint2(
      mul16x2<true>(and_or(a, 0x80008000u, (a >> 4) & 0x07f007f0u), 0x7b807b80u),  // 2^120
      mul16x2<true>(and_or(b, 0x80008000u, (b >> 4) & 0x07f007f0u), 0x7b807b80u));
}

// The codes of words a and b as pairs (a's byte i, b's byte i).
template <bool BF16, bool I8, bool BITS>
__device__ __forceinline__ void cross_pairs(uint32_t a, uint32_t b, uint32_t (&d)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (!I8 && !BF16) {
      const uint2 v = word_pairs<false, false>(__byte_perm(a, b, i == 0 ? 0x5140 : 0x7362));
      d[2 * i] = v.x;
      d[2 * i + 1] = v.y;
      continue;
    }
    // a's two bytes, b's two bytes: the first of each at the foot of its half
    const uint32_t y = i == 0 ? __byte_perm(a, b, 0x5410) : __byte_perm(a, b, 0x7632);
    if (I8 && !BF16) {
      const uint32_t u = y ^ 0x80808080u;
      d[2 * i] = add16x2<false>(__byte_perm(u, 0x64646464u, 0x4240), 0xe480e480u);
      d[2 * i + 1] = add16x2<false>(__byte_perm(u, 0x64646464u, 0x4341), 0xe480e480u);
    } else if (I8) {
      d[2 * i] = bf16_of_i8(y);
      d[2 * i + 1] = bf16_of_i8(y >> 8);
    } else {
      // byte << 4, its sign on from bit 11 to 15 (products, off the busier pipe)
      const uint32_t z = __byte_perm(y, 0, 0x4341);
      uint32_t e = (y & 0x00ff00ffu) * 16u + (y & 0x00800080u) * 240u;
      uint32_t o = z * 16u + (z & 0x00800080u) * 240u;
      if (!BITS) {
        e = mul16x2<true>(e, 0x7b807b80u);  // 2^120
        o = mul16x2<true>(o, 0x7b807b80u);
      }
      d[2 * i] = e;
      d[2 * i + 1] = o;
    }
  }
}

// The four codes of a word times a scale pair, for the matrix unit's tiles: as pairs
// (0, 1), (2, 3) for f16, and (0, 2), (1, 3) for bf16, which spares putting bytes
// together that lie apart.  SMALL: the scale pair is 2^120 times the scale (whose
// exponent is at most 7), so that e4m3's moved bits need one product.
template <bool BF16, bool I8, bool SMALL>
__device__ __forceinline__ uint2 tile_words(uint32_t w, uint32_t scale2) {
  uint2 v;
  if (!BF16) {
    v = word_pairs<false, I8>(w);
  } else if (I8) {
    v.x = bf16_of_i8(w);
    v.y = bf16_of_i8(w >> 8);
  } else {
    v.x = (w & 0x00ff00ffu) * 16u + (w & 0x00800080u) * 240u;
    v.y = and_or(w, 0x80008000u, (w >> 4) & 0x07f007f0u);
    if (!SMALL) {
      v.x = mul16x2<true>(v.x, 0x7b807b80u);  // 2^120
      v.y = mul16x2<true>(v.y, 0x7b807b80u);
    }
  }
  return make_uint2(mul16x2<BF16>(v.x, scale2), mul16x2<BF16>(v.y, scale2));
}

// Four codes times their block's scale (a pair, scale_pair): exact for scales
// that the store writes.
template <bool BF16, bool I8>
__device__ __forceinline__ uint2 values_of(uint32_t codes, uint32_t scale2) {
  const uint2 v = word_pairs<BF16, I8>(codes);
  return make_uint2(mul16x2<BF16>(v.x, scale2), mul16x2<BF16>(v.y, scale2));
}

// A scale byte as fp32 (the same numbers as scale_pair's).
template <bool BF16>
__device__ __forceinline__ float scale_float(int s) {
  const int e = BF16 ? max(s, 1) : min(max(s, 127 - 24), 127 + 15);
  return __int_as_float(s == SCALE_NAN ? 0x7fffffff : e << 23);
}

}  // namespace mab
