// Int4 codes as matrix-core operands.
//
// A 4-bit code is held as u = q + 8 in 0..15.  An and-or that puts u into the mantissa of a
// 16-bit number of known exponent makes it base + u, two codes per register:
//   fp16  nibbles at bits 0..3 take base 1024, those at bits 4..7 base 64 (no shift; the
//         upper byte's nibbles after one shift by 8).  A packed addition of -(base + 8),
//         exact, leaves q: 9 operations per 8 codes.
//   bf16  has no packed addition.  All four nibble positions are shifted to base 16 and the
//         24 = 16 + 8 is taken back by the matrix cores: the accumulator starts at
//         -24 sum(x), a product of x with a constant operand.  sum (16 + u) x - 24 sum x =
//         sum q x, with exact products and fp32 sums of one scale group at a time; the
//         summed terms are at most 31 |x| instead of 8 |x|, about 2 of an fp32 sum's 24 bits.
//         Both operands are 2^-12 of these numbers (the exponent of the base is free): 24
//         sum |x| over 128 columns is then below the largest |x|, so no finite x makes the
//         sums of a group overflow.  What is summed from them is multiplied by 2^12 (unit)
//         in the end; powers of two change no bit of it.
// The scale of a group multiplies its fp32 sum.
//
// The masks and bases are kept in registers behind empty asm statements: as literals, two of
// them do not fit one instruction and the and-or becomes an and and an or.
#pragma once
#include "sfx_mfma.hpp"

namespace sfx {

__device__ __forceinline__ uint32_t scalar_const(uint32_t v) {
  asm("" : "+s"(v));
  return v;
}
__device__ __forceinline__ uint32_t vector_const(uint32_t v) {
  asm("" : "+v"(v));
  return v;
}
__device__ __forceinline__ uint32_t pk_add(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2_t, a) + __builtin_bit_cast(half2_t, b));
}
__device__ __forceinline__ uint32_t pk_mul(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2_t, a) * __builtin_bit_cast(half2_t, b));
}

template <class T>
struct Q4;
template <>
struct Q4<TF16> {
  static constexpr bool offset = false;
  static constexpr float unit = 1.f;
  uint32_t m0, m1, o0, o1, d0, d1;
  __device__ __forceinline__ Q4()
      : m0(scalar_const(0x000F000Fu)), m1(scalar_const(0x00F000F0u)), o0(vector_const(0x64006400u)),
        o1(vector_const(0x54005400u)), d0(scalar_const(0xE408E408u)), d1(scalar_const(0xD480D480u)) {}
  // The codes of nibbles (0, 4) (1, 5) (2, 6) (3, 7) of v.
  __device__ __forceinline__ Raw<16> word(uint32_t v) const {
    const uint32_t h = v >> 8;
    Raw<16> r;
    r.w[0] = pk_add((v & m0) | o0, d0);
    r.w[1] = pk_add((v & m1) | o1, d1);
    r.w[2] = pk_add((h & m0) | o0, d0);
    r.w[3] = pk_add((h & m1) | o1, d1);
    return r;
  }
};
template <>
struct Q4<TBF16> {
  static constexpr bool offset = true;       // word() gives (24 + q) / unit
  static constexpr float unit = 4096.f;
  uint32_t m, o;
  __device__ __forceinline__ Q4() : m(scalar_const(0x00780078u)), o(vector_const(0x3B803B80u)) {}
  __device__ __forceinline__ Raw<16> word(uint32_t v) const {
    Raw<16> r;
    r.w[0] = ((v << 3) & m) | o;
    r.w[1] = ((v >> 1) & m) | o;
    r.w[2] = ((v >> 5) & m) | o;
    r.w[3] = ((v >> 9) & m) | o;
    return r;
  }
  // Written anew at each call: a product of it with something fixed is not kept in
  // registers across a loop.
  __device__ __forceinline__ static Raw<16> minus24() {
    uint32_t k = 0xBBC0BBC0u;
    asm volatile("" : "+v"(k));
    Raw<16> r;
    r.w[0] = r.w[1] = r.w[2] = r.w[3] = k;
    return r;
  }
};

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

// Keeps the memory operations before it before those after it in program order: a wait that
// counts the younger operations is only right if groups of them are issued in their order.
__device__ __forceinline__ void memory_order() { asm volatile("" ::: "memory"); }
// Waits of a wave for its own copies into LDS (all but the N youngest memory operations) and
// for its own LDS reads; the compiler moves no memory access across them.
template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N < 64, "vmcnt holds 6 bits");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

__device__ __forceinline__ uint16_t to_16(TF16, float v) { return __builtin_bit_cast(uint16_t, (_Float16)v); }
__device__ __forceinline__ uint16_t to_16(TBF16, float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }

}  // namespace sfx
