// The rows of a quantised cache: one position of one kv head.
//
//   8 bits  D e4m3 codes c; the value is g c
//   4 bits  D / 2 bytes of e2m1 codes c (element 2 j in the low half of byte j), then D / 16
//           e4m3 scales s, one for each block of 16 elements; the value is g s c
//
// g is the tensor's scale, a float of the call's.  Every s c (2 + 4 significant bits between 2^-10 and
// 2688) and every e4m3 code is exact in 16-bit floats, so a product with the unscaled values loses nothing.
#pragma once

#include <stdint.h>

namespace rdquant {

__host__ __device__ constexpr int row_bytes(int D, int bits) { return bits == 8 ? D : D / 2 + D / 16; }

// the four bytes of w, two e2m1 codes each, as pairs of 16-bit floats (low half first)
__device__ __forceinline__ void e2m1x8(uint32_t w, uint32_t (&v)[4])
{
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
        : "r"(w));
}

// the four e4m3 codes of w as two pairs of 16-bit floats
__device__ __forceinline__ void e4m3x4(uint32_t w, uint32_t& lo, uint32_t& hi)
{
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

}  // namespace rdquant
