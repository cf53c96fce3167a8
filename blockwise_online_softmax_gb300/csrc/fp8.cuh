// Rows held in 8 bits: e4m3 codes with one scale per row, a power of two.
//
// For a row x of d columns (one KV head of one token):
//   e = the least integer in [-117, 120] with max |x| <= 448 2^e,
//   code = x 2^-e to the nearest e4m3 (halves to even),  byte = e + 127.
// A code has four bits whatever the scale is, so a power of two costs nothing
// in precision against max |x| / 448 (a last bit where the row's small entries
// run into e4m3's subnormals), and x 2^-e and code 2^e are exact: what is
// read back is a bf16 value, and every implementation gets the same codes.
// (With scales max |x| / 448, bf16 rows divide to within an ulp of the middle
// between two codes in one of some 400 entries, where the division's rounding
// would decide.)  The scale is one byte (e8m0) of 238.  The range of e keeps every
// value that a code and a scale stand for a normal fp32 (and bf16) number, but for
// the codes from 256 on with e = 120: entries from 248 2^120 = 1.9375 2^127 on, of a
// largest fp32 below 256 2^120, round to 2^128 and are read as infinities.  Entries
// that are not finite become NaN and do not count in max |x|.
#pragma once
#include <cstdint>

namespace ra {

// |x| as an ordered integer, 0 where x is not finite.
__device__ __forceinline__ unsigned finite_bits(float x) {
  const unsigned b = __float_as_uint(x) & 0x7fffffffu;
  return b < 0x7f800000u ? b : 0u;
}
// The scale's byte for a row whose largest entry has these bits: its exponent
// less 8, one more above 1.75 (448 = 1.75 2^8).
__device__ __forceinline__ int scale_byte(unsigned top) {
  const int b = static_cast<int>((top + 0x1fffffu) >> 23) - 8;
  return b < 10 ? 10 : b;  // (at most 247)
}
__device__ __forceinline__ float inverse_scale(int byte) { return __uint_as_float(static_cast<unsigned>(254 - byte) << 23); }
__device__ __forceinline__ float scale_of(unsigned byte) { return __uint_as_float(byte << 23); }

// Two codes, x's in the low byte.  (An infinity would become 448.)
__device__ __forceinline__ uint32_t codes2(float x, float y) {
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(y), "f"(x));
  return c;
}
// The values of two codes as fp16 (exact), the low byte's in the low half.
__device__ __forceinline__ uint32_t halves2(uint16_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(codes));
  return h;
}

}  // namespace ra
