// Int4 codes as matrix-core operands.
//
// A 4-bit code q in [-8, 7] is used as the 16-bit number 16 + u, u = q + 8 in 0..15:
// in fp16 and in bf16 those 16 numbers are one exponent with u in the top mantissa
// bits, so two codes become a register of two numbers with a shift and an and-or.  The
// offset 24 = 16 + 8 is taken back inside the matrix cores: the accumulator starts at
// -24 sum(x) (a product of x with a constant -24 operand), so
//     sum (16 + u) x - 24 sum x = sum q x
// with exact products and fp32 sums of one group of 32 at a time; the group's scale
// multiplies that fp32 sum.  The offset makes the summed terms at most 31 |x| instead of
// 8 |x|: about 2 bits of the 24 of an fp32 sum of 32 terms.
#pragma once
#include "sfx_mfma.hpp"

namespace sfx {

template <class T>
struct Q4;
template <>
struct Q4<TF16> {
  static constexpr uint32_t mask = 0x03C003C0u, one16 = 0x4C004C00u, minus24 = 0xCE00CE00u;
  static constexpr int up = 6;     // bit where the lowest of the four mantissa bits sits
};
template <>
struct Q4<TBF16> {
  static constexpr uint32_t mask = 0x00780078u, one16 = 0x41804180u, minus24 = 0xC1C0C1C0u;
  static constexpr int up = 3;
};

// Nibbles P and P + 4 of v (u codes) as a register of two 16-bit numbers 16 + u.
template <class T, int P>
__device__ __forceinline__ uint32_t q4_pair(uint32_t v) {
  constexpr int sh = Q4<T>::up - 4 * P;
  if constexpr (sh >= 0) return ((v << sh) & Q4<T>::mask) | Q4<T>::one16;
  else return ((v >> -sh) & Q4<T>::mask) | Q4<T>::one16;
}
// The eight codes of a word: registers (0, 4) (1, 5) (2, 6) (3, 7).
template <class T>
__device__ __forceinline__ Raw<16> q4_word(uint32_t v) {
  Raw<16> r;
  r.w[0] = q4_pair<T, 0>(v);
  r.w[1] = q4_pair<T, 1>(v);
  r.w[2] = q4_pair<T, 2>(v);
  r.w[3] = q4_pair<T, 3>(v);
  return r;
}
template <class T>
__device__ __forceinline__ Raw<16> q4_minus24() {
  Raw<16> r;
  r.w[0] = r.w[1] = r.w[2] = r.w[3] = Q4<T>::minus24;
  return r;
}
__device__ __forceinline__ float half_at(uint32_t pair, int hi) {
  const half2_t h = __builtin_bit_cast(half2_t, pair);
  return hi ? (float)h.y : (float)h.x;
}

// 4 x 4 transposition between the four quarters (16 lanes) of a wave and four registers:
// on return w[j] of quarter c is what quarter j held in w[c].
__device__ __forceinline__ void quarter_transpose(uint32_t (&w)[4]) {
  const auto a = __builtin_amdgcn_permlane16_swap(w[0], w[1], false, false);
  const auto b = __builtin_amdgcn_permlane16_swap(w[2], w[3], false, false);
  const auto c = __builtin_amdgcn_permlane32_swap(a[0], b[0], false, false);
  const auto d = __builtin_amdgcn_permlane32_swap(a[1], b[1], false, false);
  w[0] = c[0];
  w[1] = d[0];
  w[2] = c[1];
  w[3] = d[1];
}

__device__ __forceinline__ uint16_t to_16(TF16, float v) { return __builtin_bit_cast(uint16_t, (_Float16)v); }
__device__ __forceinline__ uint16_t to_16(TBF16, float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }

}  // namespace sfx
