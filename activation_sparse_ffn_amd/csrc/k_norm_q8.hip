// Residual addition, root-mean-square norm and int8 rows.
//
//   h = x + r;  n = h w / sqrt(mean h^2 + eps)  (or n = h);  s = fp32(max |n| / 127),
//   q = clamp(rne(n / s), -127, 127);  y = n rounded to its type;  r' = h rounded to r's type
//
// Sums, products and quotients are taken in 64 bits: a code next to a rounding border then
// falls the same way wherever it is computed, and 64-bit operations run at the rate of 32-bit
// ones here.  Codes are those of the exact quotient: fp32 decides them unless it comes to rest next to
// a border.
//
// A row is read twice, the second time out of a cache, in pieces of 8 at any place.  Where the rows
// together are more than the last-level cache (256 MB) holds, they stay in registers between the two
// passes instead, and workgroups take several, with the weight kept and the next one on its way.
// Measured with fp32 weights (rows x length, types of x, residual, y; us by the first and the second):
// 1 x 4096 f32 f32 f16 4.9 and 5.6; 512 x 8192 f32 16.7 and 20.9; 4099 x 8192 bf16 bf16 - (235 MB) 54 and
// 57; 16384 x 4096 bf16 bf16 - 110 and 96; 4099 x 8192 f32 135 and 116.  Since, with fewer 64-bit
// operations in both: 4.6, 17.0, 50 (4.7 TB/s; 65 with nothing in the cache) by the first, 90 by the second.
#include <type_traits>

#include "sfx_launch.hpp"
#include "sfx_turn.hpp"

namespace sfx {
namespace {

struct NormArgs {
  const void* x;
  const void* r;
  void* r_out;
  const float* w;
  int8_t* q;
  float* s;
  void* y;
  size_t ldx, ldr, ldro, ldy;   // elements between rows
  double eps, per_d;            // per_d: 1 / d
  int T, d, norm, xdt, rdt, ydt;
};

// f(type) for a storage type known at run time.
template <class F>
__device__ __forceinline__ void by_type(int dt, F f) {
  if (dt == DT_F32) f(std::integral_constant<int, DT_F32>{});
  else if (dt == DT_F16) f(std::integral_constant<int, DT_F16>{});
  else f(std::integral_constant<int, DT_BF16>{});
}

__device__ __forceinline__ double lane_xor_f64(double v, int o) {
  const int lo = __shfl_xor(__double2loint(v), o), hi = __shfl_xor(__double2hiint(v), o);
  return __hiloint2double(hi, lo);
}

struct RowScale {
  double f, sd, inv;        // n = h f (w); scale and 1 / scale
  float s;
};
__device__ __forceinline__ RowScale row_scale(const NormArgs& a, double sum, double top, bool bad) {
  RowScale c;
  c.f = a.norm ? 1.0 / sqrt(sum * a.per_d + a.eps) : 1.0;
  c.s = bad ? __uint_as_float(0x7FC00000u) : (float)(top * c.f * (1.0 / 127.0));
  c.sd = (double)c.s;
  c.inv = 1.0 / c.sd;
  return c;
}

// The scale of a row from its threads' sums, largest values and whether any holds `bad`.  The first wave
// makes it for all (the divisions and the root are as much work as a few hundred elements); it is
// stored by its first thread.
template <int NT>
__device__ __forceinline__ RowScale row_total(const NormArgs& a, double sum, double top, bool bad, size_t t, double (*sh)[NT / kWave],
                                              RowScale& out) {
#pragma unroll
  for (int o = 32; o; o >>= 1) {
    sum += lane_xor_f64(sum, o);
    top = fmax(top, lane_xor_f64(top, o));
  }
  if (__any(bad)) top = INFINITY;
  RowScale c;
  if constexpr (NT > kWave) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
      sh[0][wave] = sum;
      sh[1][wave] = top;
    }
    __syncthreads();
    if (wave == 0) {
      sum = top = 0.;
#pragma unroll
      for (int k = 0; k < NT / kWave; ++k) {
        sum += sh[0][k];
        top = fmax(top, sh[1][k]);
      }
      c = row_scale(a, sum, top, !(top < INFINITY));
      if (threadIdx.x == 0) {
        out = c;
        if (a.s) a.s[t] = c.s;
      }
    }
    __syncthreads();                                           // the next row's totals come behind all reads of sh
    c = out;
  } else {
    c = row_scale(a, sum, top, !(top < INFINITY));
    if (a.s && threadIdx.x == 0) a.s[t] = c.s;
  }
  return c;
}
// The nearest code (ties to even): the rest n - k s of a candidate decides, exactly, as k s is.
__device__ __forceinline__ int row_code(const RowScale& c, double n) {
  const double k = rint(n * c.inv), rest = fma(-k, c.sd, n), half = 0.5 * c.sd, over = fabs(rest) - half;
  const int i = (int)fmin(fmax(k, -127.), 127.);
  const int step = over > 0. || (over == 0. && (i & 1)) ? (rest > 0. ? 1 : -1) : 0;
  return c.s > 0.f ? min(max(i + step, -127), 127) : 0;
}

// f / s in fp32, what m below is made of.  It is 127 / max |h w|: where that or s is below fp32's normal numbers
// it has fewer bits than m needs, and quotients by such an s pass 127.5.  NaN then, so that every code of
// the row is taken in 64 bits.  (A product g w below them is off by 2^-150, times h by less than 2^-22.)
__device__ __forceinline__ float row_factor(const RowScale& c) {
  const float g = (float)(c.f * c.inv);
  return g >= 0x1p-126f && c.s >= 0x1p-126f ? g : __uint_as_float(0x7FC00000u);
}

// Codes of eight n, from fp32 values m of n / s: four roundings of 2^-24 of at most 127, 2^-15, unless a
// code comes to rest nearer to a border than 2^-14, or s is no positive number (m is none then either): then
// from n64(j), in 64 bits, one element at a time (all eight of a piece at once: 4099 x 8192 bf16 out of memory 74 us
// instead of 65).  Adding
// 1.5 2^23 rounds to a whole number and leaves its low byte in place.
template <class F>
__device__ __forceinline__ Raw<8> codes8(const RowScale& c, const float (&m)[8], F n64) {
  uint32_t u[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float k = m[j] + 12582912.f;
    u[j] = __float_as_uint(k);
    if (!(fabsf(m[j] - (k - 12582912.f)) <= 0.5f - 0x1p-14f)) u[j] = (uint32_t)row_code(c, n64(j));
  }
  Raw<8> q;
#pragma unroll
  for (int k = 0; k < 2; ++k)
    q.w[k] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(u[4 * k + 3], u[4 * k + 2], 0x0c0c0400u),
                                   __builtin_amdgcn_perm(u[4 * k + 1], u[4 * k], 0x0c0c0400u), 0x05040100u);
  return q;
}

// Eight elements of a type known at run time as they lie; fp32 (WIDE) takes both registers' worth.
template <bool WIDE>
struct Any8 {
  Raw<16> r[WIDE ? 2 : 1];
};
template <bool WIDE>
__device__ __forceinline__ void load_any(int dt, const void* p, size_t i, Any8<WIDE>& e) {
  const uint8_t* b = (const uint8_t*)p + i * (WIDE && dt == DT_F32 ? 4 : 2);
  e.r[0] = load_raw_at<16>(b);
  if constexpr (WIDE)
    if (dt == DT_F32) e.r[1] = load_raw_at<16>(b + 16);
}
template <bool WIDE>
__device__ __forceinline__ void widen_any(int dt, const Any8<WIDE>& e, float (&x)[8]) {
  if constexpr (WIDE)
    if (dt == DT_F32) {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = __uint_as_float(e.r[j >> 2].w[j & 3]);
      return;
    }
  if (dt == DT_F16) unpack<TF16, 4>(e.r[0].w, x);
  else unpack<TBF16, 4>(e.r[0].w, x);
}

__device__ __forceinline__ void load_weights(const NormArgs& a, int i, float (&w)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j] = 1.f;
  if (a.w) __builtin_memcpy(w, a.w + i, 32);
}

// NT threads to a row, V pieces of 8 to a thread; the next row is on its way while one is worked on.
// WIDE: x or the residual is fp32.  The last piece of a row whose length is no multiple of 8
// starts inside the one before: what both have counts once in the sum and is stored twice alike.
template <int NT, int V, bool WIDE>
__global__ __launch_bounds__(NT) void k_norm_q8_held(NormArgs a) {
  __shared__ double sh[2][NT / kWave];
  __shared__ RowScale scale;
  float w[V][8];
  bool bad_w = false;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int i = (v * NT + threadIdx.x) * 8;
    load_weights(a, min(i, a.d - 8), w[v]);
    if (i < a.d)
#pragma unroll
      for (int j = 0; j < 8; ++j) bad_w |= !(fabsf(w[v][j]) < INFINITY);
  }
  Any8<WIDE> xn[V], rn[V];
  const auto fetch = [&](int t) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int i = min((v * NT + (int)threadIdx.x) * 8, a.d - 8);
      load_any(a.xdt, a.x, (size_t)t * a.ldx + i, xn[v]);
      if (a.r) load_any(a.rdt, a.r, (size_t)t * a.ldr + i, rn[v]);
    }
  };
  fetch(blockIdx.x);
  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
    // behind empty asm: as 64-bit numbers, made once for all rows, the weights would take twice their registers
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) asm volatile("" : "+v"(w[v][j]));
    Any8<WIDE> x[V], r[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      x[v] = xn[v];
      r[v] = rn[v];
    }
    if (t + (int)gridDim.x < a.T) fetch(t + gridDim.x);
    double sum = 0., top = 0.;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float xf[8], rf[8];
      widen_any(a.xdt, x[v], xf);
      if (a.r) widen_any(a.rdt, r[v], rf);
      const int i = (v * NT + (int)threadIdx.x) * 8, twice = i - (a.d - 8);
      if (twice > 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < twice) xf[j] = rf[j] = 0.f;
      }
      if (i < a.d)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const double h = a.r ? (double)xf[j] + (double)rf[j] : (double)xf[j];
          sum = fma(h, h, sum);
          top = fmax(top, fabs(h * (double)w[v][j]));
        }
      __builtin_amdgcn_sched_barrier(0);
    }
    // h is finite where its square is, and h w where w is too
    bool bad = bad_w || !(sum < INFINITY);
    const RowScale c = row_total<NT>(a, sum, top, bad, t, sh, scale);
    const float g = row_factor(c);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if ((v * NT + (int)threadIdx.x) * 8 >= a.d) continue;
      const int i = min((v * NT + (int)threadIdx.x) * 8, a.d - 8);
      float xf[8], rf[8], hf[8];
      widen_any(a.xdt, x[v], xf);
      if (a.r) widen_any(a.rdt, r[v], rf);
      const auto n64 = [&](int j) {
        const double h = a.r ? (double)xf[j] + (double)rf[j] : (double)xf[j];
        return a.w ? h * c.f * (double)w[v][j] : h * c.f;
      };
#pragma unroll
      for (int j = 0; j < 8; ++j) hf[j] = a.r ? xf[j] + rf[j] : xf[j];
      if (a.q) {
        float mf[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) mf[j] = hf[j] * (g * w[v][j]);
        const Raw<8> q = codes8(c, mf, n64);
        __builtin_memcpy(a.q + (size_t)t * a.d + i, &q, 8);
      }
      if (a.r_out) by_type(a.rdt, [&](auto dt) { store8_at<decltype(dt)::value>(a.r_out, (size_t)t * a.ldro + i, hf); });
      if (a.y) {
        float nf[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) nf[j] = (float)n64(j);
        by_type(a.ydt, [&](auto dt) { store8_at<decltype(dt)::value>(a.y, (size_t)t * a.ldy + i, nf); });
      }
      __builtin_amdgcn_sched_barrier(0);                       // one piece's temporaries at a time
    }
  }
}

__device__ __forceinline__ float load_one(int dt, const void* p, size_t i) {
  float v = 0.f;
  by_type(dt, [&](auto t) { v = load_elem<decltype(t)::value>(p, i); });
  return v;
}

// A row to a workgroup of NT threads, read twice, with U pieces of 8 on their way to a thread; the
// elements behind the last whole piece go one to a thread.
template <int NT, bool WIDE>
__global__ __launch_bounds__(NT) void k_norm_q8_twice(NormArgs a) {
  constexpr int U = 2;
  __shared__ double sh[2][NT / kWave];
  __shared__ RowScale scale;
  const size_t t = blockIdx.x;
  const int whole = a.d & ~7;
  struct Piece {
    Any8<WIDE> x, r;
    float w[8];
  };
  const auto fetch = [&](int i, Piece& p) {
    load_any(a.xdt, a.x, t * a.ldx + i, p.x);
    if (a.r) load_any(a.rdt, a.r, t * a.ldr + i, p.r);
    load_weights(a, i, p.w);
  };
  const auto widen_both = [&](const Piece& p, float (&x)[8], float (&r)[8]) {
    widen_any(a.xdt, p.x, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = 0.f;
    if (a.r) widen_any(a.rdt, p.r, r);
  };
  const auto sum_of = [&](int i) {
    double h = (double)load_one(a.xdt, a.x, t * a.ldx + i);
    if (a.r) h += (double)load_one(a.rdt, a.r, t * a.ldr + i);
    return h;
  };
  double sum = 0., top = 0.;
  float w_not = 0.f;                                           // NaN behind a weight that is not finite
  const auto count = [&](double h, float w) {
    sum = fma(h, h, sum);
    top = fmax(top, fabs(h * (double)w));
    w_not = fmaf(w, 0.f, w_not);
  };
  const int tail = whole + (int)threadIdx.x;
  if (tail < a.d) count(sum_of(tail), a.w ? a.w[tail] : 1.f);
  for (int i0 = (int)threadIdx.x * 8; i0 < whole; i0 += U * NT * 8) {
    Piece p[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + u * NT * 8 < whole) fetch(i0 + u * NT * 8, p[u]);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i0 + u * NT * 8 >= whole) continue;
      float x[8], r[8];
      widen_both(p[u], x, r);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const double h = a.r ? (double)x[j] + (double)r[j] : (double)x[j];
        if (a.w) {
          count(h, p[u].w[j]);
        } else {
          sum = fma(h, h, sum);
          top = fmax(top, fabs(h));
        }
      }
    }
  }
  // h is finite where its square is, and h w where w is too
  const RowScale c = row_total<NT>(a, sum, top, !(sum < INFINITY) || w_not != 0.f, t, sh, scale);
  const float g = row_factor(c);
  for (int i = (int)threadIdx.x * 8; i < whole; i += NT * 8) {
    Piece p;
    fetch(i, p);                                               // before r_out, which may be r, is written
    float x[8], r[8], hf[8], mf[8];
    widen_both(p, x, r);
    const auto n64 = [&](int j) { return ((double)x[j] + (double)r[j]) * c.f * (double)p.w[j]; };
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      hf[j] = x[j] + r[j];
      mf[j] = hf[j] * (g * p.w[j]);
    }
    if (a.q) {
      const Raw<8> q = codes8(c, mf, n64);
      __builtin_memcpy(a.q + t * a.d + i, &q, 8);
    }
    if (a.r_out) by_type(a.rdt, [&](auto dt) { store8_at<decltype(dt)::value>(a.r_out, t * a.ldro + i, hf); });
    if (a.y) {
      float nf[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) nf[j] = (float)n64(j);
      by_type(a.ydt, [&](auto dt) { store8_at<decltype(dt)::value>(a.y, t * a.ldy + i, nf); });
    }
  }
  if (tail < a.d) {
    const double h = sum_of(tail), n = a.w ? h * c.f * (double)a.w[tail] : h * c.f;
    if (a.q) a.q[t * a.d + tail] = (int8_t)row_code(c, n);
    if (a.r_out) by_type(a.rdt, [&](auto dt) { store_elem<decltype(dt)::value>(a.r_out, t * a.ldro + tail, (float)h); });
    if (a.y) by_type(a.ydt, [&](auto dt) { store_elem<decltype(dt)::value>(a.y, t * a.ldy + tail, (float)n); });
  }
}

template <int NT>
void norm_twice(hipStream_t st, const NormArgs& a, bool wide) {
  if (wide) k_norm_q8_twice<NT, true><<<dim3(a.T), dim3(NT), 0, st>>>(a);
  else k_norm_q8_twice<NT, false><<<dim3(a.T), dim3(NT), 0, st>>>(a);
}

// As many workgroups as the device holds at once, each with as many rows as any other or one less.
template <int NT, int V>
void norm_held(hipStream_t st, const NormArgs& a, bool wide) {
  const int most = 256 * (V >= 4 ? 1 : 1024 / NT), each = (a.T + most - 1) / most;
  const dim3 g((a.T + each - 1) / each);
  if (wide) k_norm_q8_held<NT, V, true><<<g, dim3(NT), 0, st>>>(a);
  else k_norm_q8_held<NT, V, false><<<g, dim3(NT), 0, st>>>(a);
}

}  // namespace

hipError_t launch_norm_q8(hipStream_t st, int xdt, int rdt, int ydt, int T, int d, int norm, float eps, const void* x,
                          size_t ldx, const void* r, size_t ldr, void* r_out, size_t ldro, const float* w, int8_t* q,
                          float* s, void* y, size_t ldy) {
  const NormArgs a{x, r, r_out, w, q, s, y, ldx, ldr, ldro, ldy, (double)eps, 1.0 / d, T, d, norm, xdt, rdt, ydt};
  const auto size = [](int dt) { return dt == DT_F32 ? 4 : 2; };
  const bool wide = xdt == DT_F32 || (r && rdt == DT_F32);
  if (d >= 8 && d <= 16384 && (long long)T * d * (size(xdt) + (r ? size(rdt) : 0)) > 192ll << 20) {
    if (d <= 512) norm_held<64, 1>(st, a, wide);
    else if (d <= 1024) norm_held<64, 2>(st, a, wide);
    else if (d <= 2048) norm_held<256, 1>(st, a, wide);
    else if (d <= 4096) norm_held<256, 2>(st, a, wide);
    else if (d <= 8192) norm_held<512, 2>(st, a, wide);
    else norm_held<512, 4>(st, a, wide);
  } else if (d <= 512) norm_twice<64>(st, a, wide);             // a piece or two to a thread
  else if (d <= 1024) norm_twice<128>(st, a, wide);             // (2048 x 1024: 7.9 us; by 64 or 256 threads 8.1, 10.2)
  else if (d <= 2048 || (d <= 4096 && T > 512)) norm_twice<256>(st, a, wide);   // 4096 x 4096: 32 us, by 512 40
  else if (d <= 16384 || T > 256) norm_twice<512>(st, a, wide);                 // 1 x 4096: 4.9 us, by 256 5.5
  else norm_twice<1024>(st, a, wide);                           // 1 x 32768: 14.1 us, by 512 15.7
  return hipGetLastError();
}

}  // namespace sfx
