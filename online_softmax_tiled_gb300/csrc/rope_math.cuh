// Angles of the rotary positions, for the kernels that turn queries and keys
// (rope.cu, cache_append.cu).
//
// p·w loses all of its meaning in float32 at far positions (at p = 10^6 and
// w = 1 an ulp is 1/16 rad), and float64 multiplies are scarce on this chip.
// The angle is kept as a 64-bit fraction of a full turn instead: t = 2^64 ·
// frac(w / 2π) once per pair from w's bits and 128 bits of 2/π, then p·t modulo
// 2^64, where whole turns fall off by themselves. For |w| < 2^64 the error is
// at most |p|·1.5·2^-64 turns (below 2^-32 for every 32-bit p); larger
// frequencies, of which 128 bits do not tell the fraction, give NaN like those
// that are not finite. The remainder is rounded to 32 bits, then to float32, and
// goes to sincospi.
#pragma once

#include "common.cuh"

namespace attn {

// 2^64 · frac(w / 2π) for |w| < 2^64: w = M · 2^(e - 63) with M in
// [2^63, 2^64), and C = floor(2^128 · 2/π), so w / 2π · 2^64 =
// P · 2^(e - 65) with P = M·C / 2^64, below 2^128. P is off by less than two
// units, one for the bits of 2/π past C and one for those cut off, and they
// count 2^(e - 65) <= 1/4 each here.
ATTN_DEVINL uint64_t turns_of(double w) {
  constexpr uint64_t kHi = 0xA2F9836E4E441529ull, kLo = 0xFC2757D1F534DDC0ull;
  const uint64_t bits = uint64_t(__double_as_longlong(w));
  const int ef = int((bits >> 52) & 0x7ff);            // e + 1023
  const uint64_t M = (bits << 11) | (1ull << 63);
  const uint64_t mid = M * kHi, low = mid + __umul64hi(M, kLo);
  const uint64_t high = __umul64hi(M, kHi) + (low < mid);
  const int sh = max(2, 1088 - ef);                    // 65 - e
  // (ef = 0: zero, and below 2^-1022)
  const uint64_t t = ef == 0 || sh >= 128 ? 0
                     : sh >= 64           ? high >> (sh - 64)
                                          : high << (64 - sh) | low >> sh;
  return (bits >> 63) ? 0 - t : t;
}

// cos and sin of p·w times `magnitude`
ATTN_DEVINL void turn_cos_sin(long long p, double w, float magnitude, float& c, float& s) {
  // the angle as a fraction of a turn: its top 32 bits, rounded, are off
  // by 2^-33 turns at most, and rounded to float32 once more
  const uint64_t t = uint64_t(p) * turns_of(w) + 0x80000000ull;
  float sine, cosine;
  sincospif(float(int(uint32_t(t >> 32))) * 0x1p-31f, &sine, &cosine);
  // a frequency that is not finite, or of 2^64 and more, gives NaN, not a
  // wrong angle (its exponent tells; comparing float64 values is slow here)
  const bool good = ((uint64_t(__double_as_longlong(w)) >> 52) & 0x7ff) < 1023 + 64;
  const float m = good ? magnitude : __int_as_float(0x7fffffff);
  c = cosine * m;
  s = sine * m;
}

}  // namespace attn
