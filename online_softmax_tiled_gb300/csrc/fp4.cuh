// The 4-bit rows of a cache (kernels that write them: cache_append.cu; that
// read them: cache_append.cu, decode_window.cu).
//
// A row of D elements is D/32 groups of 32 adjacent ones; a group holds e2m1
// codes (a sign bit and 0, 0.5, 1, 1.5, 2, 3, 4 or 6) and one bf16 scale. Byte
// (D/16)·g + 2c + b of a row's D/2 code bytes holds elements 32c + 4g + 2b (low
// half) and the next one (high half), g < 8, b < 2: the D/16 bytes of one g hold
// four adjacent elements of every group, those of 2t and 2t + 1 eight. These are
// the elements of a row that one lane contracts in a matrix product of 16-bit
// fragments: lane (g, t) reads bytes (D/8)·t of keys g as its part of K, bytes
// (D/16)·g of keys 2t, 2t + 1 as its part of Vᵀ, and all products of one
// instruction belong to one group, whose scale then multiplies their sum.
#pragma once

#include "common.cuh"

namespace attn {

// Byte `i` of `w` as two float16 values, the low half's first (every e2m1
// value is exact in float16).
template <int i> ATTN_DEVINL uint32_t e2m1x2_to_f16x2(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b%2;\n\t}" : "=r"(r) : "r"(w), "n"(i));
  return r;
}

// The codes nearest to eight values, two a byte, the first in the low half; ties to
// the even code, beyond 6 the code of 6.
ATTN_DEVINL uint32_t f32_to_e2m1x8(const f2 (&x)[4]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tcvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\tcvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\tmov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(x[0].x), "f"(x[0].y), "f"(x[1].x), "f"(x[1].y), "f"(x[2].x), "f"(x[2].y), "f"(x[3].x),
        "f"(x[3].y));
  return r;
}

}  // namespace attn
