// What the two tcgen05 decode kernels share (paged_tc_kernel.cu and
// paged_prefix_kernel.cu): their tiles, TMEM accesses and the cutting of weights into
// bf16 terms.  Device code only.
#pragma once
#include "paged_walk.cuh"

namespace ra {
namespace paged {
namespace umma {

constexpr int BT = 128;          // keys per tile
constexpr int RT = 128;          // query rows of an item
constexpr int kThreads = 512;
constexpr uint32_t CHB = BT * 128;  // one 64-column chunk of a tile, 128-byte swizzle

// 32 lanes x 8 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// 32 lanes x 16 consecutive 32-bit columns (valid after tmem_wait_ld).
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
// The two values cut to bf16, the first in the low half.
__device__ __forceinline__ uint32_t high_halves(float a, float b) {
  return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}
// What that leaves of them, exactly.
__device__ __forceinline__ void drop_high(float& a, float& b) {
  const float na = __uint_as_float((__float_as_uint(a) & 0xffff0000u) ^ 0x80000000u);
  const float nb = __uint_as_float((__float_as_uint(b) & 0xffff0000u) ^ 0x80000000u);
  f2unpack(fadd2(f2pack(a, b), f2pack(na, nb)), a, b);
}

}  // namespace umma
}  // namespace paged
}  // namespace ra
