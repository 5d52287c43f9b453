// Rows of keys and queries on their way into a cache: eight elements to a thread, turned by
// the angles of their position.
//
// R(pos) turns pairs of the first `rot` dims by the angles whose cosines and sines the caller's
// fp32 table holds for the position.  The two products and their sum are taken in 64 bits
// (the products are exact there) and rounded once to fp32: a quotient next to a rounding
// border then falls the same way wherever it is computed.
#pragma once
#include <type_traits>

#include "sfx_q4.hpp"

namespace sfx {

struct Rotation {
  const float* cs;          // [max_pos][rot]: cosines, then sines; null: none
  int rot, max_pos, pairs;
};

template <int DT>
__device__ __forceinline__ float load_elem(const void* p, size_t i) {
  if constexpr (DT == DT_F32) return ((const float*)p)[i];
  else if constexpr (DT == DT_F16) return (float)((const _Float16*)p)[i];
  else return __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16);
}
template <int DT>
__device__ __forceinline__ void store_elem(void* p, size_t i, float v) {
  if constexpr (DT == DT_F32) ((float*)p)[i] = v;
  else if constexpr (DT == DT_F16) ((_Float16*)p)[i] = (_Float16)v;
  else ((__bf16*)p)[i] = (__bf16)v;
}

// Eight consecutive elements as they lie; VEC: at 16-byte aligned places.
template <int DT>
struct Eight {
  Raw<16> r[DT == DT_F32 ? 2 : 1];
};
template <int DT, bool VEC>
__device__ __forceinline__ Eight<DT> load8(const void* p, size_t i) {
  Eight<DT> e;
  if constexpr (VEC) {
    const uint8_t* q = (const uint8_t*)p + i * (DT == DT_F32 ? 4 : 2);
    e.r[0] = load_raw<16>(q);
    if constexpr (DT == DT_F32) e.r[1] = load_raw<16>(q + 16);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if constexpr (DT == DT_F32) {
        e.r[j >> 2].w[j & 3] = ((const uint32_t*)p)[i + j];
      } else {
        const uint32_t v = ((const uint16_t*)p)[i + j];
        e.r[0].w[j >> 1] = (j & 1) ? e.r[0].w[j >> 1] | (v << 16) : v;
      }
    }
  }
  return e;
}
template <int DT>
__device__ __forceinline__ void widen(const Eight<DT>& e, float (&x)[8]) {
  if constexpr (DT == DT_F32) {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = __uint_as_float(e.r[j >> 2].w[j & 3]);
  } else if constexpr (DT == DT_F16) {
    unpack<TF16, 4>(e.r[0].w, x);
  } else {
    unpack<TBF16, 4>(e.r[0].w, x);
  }
}

// x co + turn in 64 bits, where the product and the sum's operands are exact, rounded once.
// The fp32 value is what is rounded on to 16 bits or quantised: the copy keeps the compiler
// from converting the 64-bit sum to 16 bits directly.
__device__ __forceinline__ float turned(float x, float o, float co, float si, bool first) {
  const double turn = (double)o * (double)si;
  float y = (float)((double)x * (double)co + (first ? -turn : turn));
  asm volatile("" : "+v"(y));
  return y;
}

template <int DT>
__device__ __forceinline__ void store8(void* p, size_t i, const float (&x)[8]) {
  Raw<16> r;
  if constexpr (DT == DT_F32) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
      for (int j = 0; j < 4; ++j) r.w[j] = __float_as_uint(x[4 * k + j]);
      *(Raw<16>*)((float*)p + i + 4 * k) = r;
    }
  } else {
    using T = std::conditional_t<DT == DT_F16, TF16, TBF16>;
#pragma unroll
    for (int j = 0; j < 4; ++j) r.w[j] = (uint32_t)to_16(T{}, x[2 * j]) | ((uint32_t)to_16(T{}, x[2 * j + 1]) << 16);
    *(Raw<16>*)((uint16_t*)p + i) = r;
  }
}

// The same at any element: one wide access each, which takes any address.
template <int N>
__device__ __forceinline__ Raw<N> load_raw_at(const uint8_t* p) {
  Raw<N> r;
  __builtin_memcpy(&r, p, N);
  return r;
}
template <int DT>
__device__ __forceinline__ Eight<DT> load8_at(const void* p, size_t i) {
  Eight<DT> e;
  __builtin_memcpy(&e, (const uint8_t*)p + i * (DT == DT_F32 ? 4 : 2), sizeof e);
  return e;
}
template <int DT>
__device__ __forceinline__ void store8_at(void* p, size_t i, const float (&x)[8]) {
  Eight<DT> e;
  store8<DT>(&e, 0, x);
  __builtin_memcpy((uint8_t*)p + i * (DT == DT_F32 ? 4 : 2), &e, sizeof e);
}

// What turns a thread's dims d0 .. d0 + 7 at one position: cosine and sine per dim, whether it
// is the first of its pair, and where the other one is.
struct Turn {
  float co[8], si[8];
};
__device__ __forceinline__ int turn_pair(const Rotation& a, int d) { return a.pairs ? d >> 1 : d < (a.rot >> 1) ? d : d - (a.rot >> 1); }
__device__ __forceinline__ bool turn_first(const Rotation& a, int d) { return a.pairs ? (d & 1) == 0 : d < (a.rot >> 1); }
__device__ __forceinline__ int turn_other(const Rotation& a, int d) {
  return a.pairs ? d ^ 1 : d < (a.rot >> 1) ? d + (a.rot >> 1) : d - (a.rot >> 1);
}
// A slice's cosines and its sines are eight (pairs: four) neighbours each, except where a half ends
// inside it.
struct alignas(4) Four {
  float v[4];
};
__device__ __forceinline__ void load_turn(const Rotation& a, const float* cs, int d0, Turn& t) {
  const int half = a.rot >> 1, i0 = turn_pair(a, d0), n = a.pairs ? 4 : 8;
  if (i0 + n <= half && (a.pairs || d0 + 8 <= half || d0 >= half)) {
    const Four c = *(const Four*)(cs + i0), s = *(const Four*)(cs + half + i0);
    Four c2 = c, s2 = s;
    if (!a.pairs) {
      c2 = *(const Four*)(cs + i0 + 4);
      s2 = *(const Four*)(cs + half + i0 + 4);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      t.co[j] = a.pairs ? c.v[j >> 1] : j < 4 ? c.v[j & 3] : c2.v[j & 3];
      t.si[j] = a.pairs ? s.v[j >> 1] : j < 4 ? s.v[j & 3] : s2.v[j & 3];
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int i = min(turn_pair(a, d0 + j), half - 1);         // dims past rot are not turned
    t.co[j] = cs[i];
    t.si[j] = cs[half + i];
  }
}
// Where the slice's partners lie, for a whole slice of them in another place.
__device__ __forceinline__ bool turn_apart(const Rotation& a, int d0) { return a.cs && !a.pairs && d0 < a.rot; }

// VEC: the first `rot` dims and their halves are whole slices of 8.
template <int DT, bool VEC>
__device__ __forceinline__ void turn8(const Rotation& a, const void* p, size_t head, int d0, const Eight<DT>& own,
                                      const Eight<DT>& apart, const Turn& t, float (&y)[8]) {
  float x[8];
  widen<DT>(own, x);
#pragma unroll
  for (int j = 0; j < 8; ++j) y[j] = x[j];
  if (!a.cs || d0 >= a.rot) return;
  if constexpr (VEC) {
    if (a.pairs) {
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = turned(x[j], x[j ^ 1], t.co[j], t.si[j], (j & 1) == 0);
    } else {
      float o[8];
      widen<DT>(apart, o);
      const bool first = d0 < (a.rot >> 1);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = turned(x[j], o[j], t.co[j], t.si[j], first);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (d0 + j < a.rot)
        y[j] = turned(x[j], load_elem<DT>(p, head + turn_other(a, d0 + j)), t.co[j], t.si[j], turn_first(a, d0 + j));
  }
}

}  // namespace sfx
