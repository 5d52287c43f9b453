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
// Rows of up to 32768 elements whose pieces of 8 are aligned stay in registers between the two
// passes; workgroups take several rows and keep the weight.  Other rows are read twice.
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
  double eps;
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

// Sum and largest of a workgroup's threads, and whether any holds `bad`.  (The barrier in front of
// the writes keeps the last row's reads apart from them.)
template <int NT>
__device__ __forceinline__ void row_totals(double& sum, double& top, bool& bad, double (*sh)[NT / kWave]) {
#pragma unroll
  for (int o = 32; o; o >>= 1) {
    sum += lane_xor_f64(sum, o);
    top = fmax(top, lane_xor_f64(top, o));
  }
  if (__any(bad)) top = INFINITY;
  if constexpr (NT > kWave) {
    const int wave = threadIdx.x >> 6;
    __syncthreads();
    if ((threadIdx.x & 63) == 0) {
      sh[0][wave] = sum;
      sh[1][wave] = top;
    }
    __syncthreads();
    sum = top = 0.;
#pragma unroll
    for (int k = 0; k < NT / kWave; ++k) {
      sum += sh[0][k];
      top = fmax(top, sh[1][k]);
    }
  }
  bad = !(top < INFINITY);
}

struct RowScale {
  double f, sd, inv;        // n = h f (w); scale and 1 / scale
  float s;
};
__device__ __forceinline__ RowScale row_scale(const NormArgs& a, double sum, double top, bool bad) {
  RowScale c;
  c.f = a.norm ? 1.0 / sqrt(sum / a.d + a.eps) : 1.0;
  c.s = bad ? __uint_as_float(0x7FC00000u) : (float)(top * c.f / 127.0);
  c.sd = (double)c.s;
  c.inv = 1.0 / c.sd;
  return c;
}
// The nearest code (ties to even): the rest n - k s of a candidate decides, exactly, as k s is.
__device__ __forceinline__ int row_code(const RowScale& c, double n) {
  const double k = rint(n * c.inv), rest = fma(-k, c.sd, n), half = 0.5 * c.sd, over = fabs(rest) - half;
  const int i = (int)fmin(fmax(k, -127.), 127.);
  const int step = over > 0. || (over == 0. && (i & 1)) ? (rest > 0. ? 1 : -1) : 0;
  return c.s > 0.f ? min(max(i + step, -127), 127) : 0;
}

// Eight elements of a type known at run time as they lie; fp32 (WIDE) takes both registers' worth.
template <bool WIDE>
struct Any8 {
  Raw<16> r[WIDE ? 2 : 1];
};
template <bool WIDE>
__device__ __forceinline__ void load_any(int dt, const void* p, size_t i, Any8<WIDE>& e) {
  const uint8_t* b = (const uint8_t*)p + i * (WIDE && dt == DT_F32 ? 4 : 2);
  e.r[0] = load_raw<16>(b);
  if constexpr (WIDE)
    if (dt == DT_F32) e.r[1] = load_raw<16>(b + 16);
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

// NT threads to a row, V pieces of 8 to a thread; the next row is on its way while one is worked on.
// WIDE: x or the residual is fp32.
template <int NT, int V, bool WIDE>
__global__ __launch_bounds__(NT) void k_norm_q8(NormArgs a) {
  __shared__ double sh[2][NT / kWave];
  float w[V][8];
  bool bad_w = false;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int i = (v * NT + threadIdx.x) * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) w[v][j] = a.w ? a.w[min(i, a.d - 8) + j] : 1.f;
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
      if ((v * NT + (int)threadIdx.x) * 8 < a.d)
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
    row_totals<NT>(sum, top, bad, sh);
    const RowScale c = row_scale(a, sum, top, bad);
    if (a.s && threadIdx.x == 0) a.s[t] = c.s;
    const float g = (float)(c.f * c.inv);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int i = (v * NT + threadIdx.x) * 8;
      if (i >= a.d) continue;
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
        // in fp32: four roundings of 2^-24 of at most 127, 2^-15, unless a code comes to rest nearer
        // to a border than 2^-14: then in 64 bits.  Adding 1.5 2^23 rounds to a whole number and
        // leaves its low byte in place.
        uint32_t u[8];
        bool near = false;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float m = hf[j] * (g * w[v][j]), k = m + 12582912.f;
          near |= !(fabsf(m - (k - 12582912.f)) <= 0.5f - 0x1p-14f);
          u[j] = __float_as_uint(k);
        }
        uint32_t q[2];
#pragma unroll
        for (int k = 0; k < 2; ++k)
          q[k] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(u[4 * k + 3], u[4 * k + 2], 0x0c0c0400u),
                                       __builtin_amdgcn_perm(u[4 * k + 1], u[4 * k], 0x0c0c0400u), 0x05040100u);
        if (near || !(c.s > 0.f)) {
          q[0] = q[1] = 0;
#pragma unroll
          for (int j = 0; j < 8; ++j) q[j >> 2] |= ((uint32_t)row_code(c, n64(j)) & 255u) << (8 * (j & 3));
        }
        *(Raw<8>*)(a.q + (size_t)t * a.d + i) = Raw<8>{{q[0], q[1]}};
      }
      if (a.r_out) by_type(a.rdt, [&](auto dt) { store8<decltype(dt)::value>(a.r_out, (size_t)t * a.ldro + i, hf); });
      if (a.y) {
        float nf[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) nf[j] = (float)n64(j);
        by_type(a.ydt, [&](auto dt) { store8<decltype(dt)::value>(a.y, (size_t)t * a.ldy + i, nf); });
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

// Any row, read twice.
__global__ __launch_bounds__(kBlock) void k_norm_q8_any(NormArgs a) {
  __shared__ double sh[2][kWavesPerBlock];
  const int t = blockIdx.x;
  const auto sum_of = [&](int i) {
    double h = (double)load_one(a.xdt, a.x, (size_t)t * a.ldx + i);
    if (a.r) h += (double)load_one(a.rdt, a.r, (size_t)t * a.ldr + i);
    return h;
  };
  double sum = 0., top = 0.;
  bool bad = false;
  for (int i = threadIdx.x; i < a.d; i += kBlock) {
    const double h = sum_of(i), m = fabs(a.w ? h * (double)a.w[i] : h);
    sum = fma(h, h, sum);
    bad |= !(m < INFINITY);
    top = fmax(top, m);
  }
  row_totals<kBlock>(sum, top, bad, sh);
  const RowScale c = row_scale(a, sum, top, bad);
  if (a.s && threadIdx.x == 0) a.s[t] = c.s;
  for (int i = threadIdx.x; i < a.d; i += kBlock) {
    const double h = sum_of(i);                                // before res_out, which may be res, is written
    double n = h * c.f;
    if (a.w) n *= (double)a.w[i];
    if (a.r_out) by_type(a.rdt, [&](auto dt) { store_elem<decltype(dt)::value>(a.r_out, (size_t)t * a.ldro + i, (float)h); });
    if (a.y) by_type(a.ydt, [&](auto dt) { store_elem<decltype(dt)::value>(a.y, (size_t)t * a.ldy + i, (float)n); });
    if (a.q) a.q[(size_t)t * a.d + i] = (int8_t)row_code(c, n);
  }
}

// As many workgroups as the device holds at once, each with as many rows as any other or one less
// (4099 x 8192, bf16 with residual: 59 us; one row to a workgroup, 87).
template <int NT, int V>
void norm_run(hipStream_t st, const NormArgs& a) {
  const int most = 256 * (V >= 4 ? 1 : 1024 / NT), each = (a.T + most - 1) / most;
  const dim3 g((a.T + each - 1) / each), b(NT);
  if (a.xdt == DT_F32 || (a.r && a.rdt == DT_F32)) k_norm_q8<NT, V, true><<<g, b, 0, st>>>(a);
  else k_norm_q8<NT, V, false><<<g, b, 0, st>>>(a);
}

}  // namespace

hipError_t launch_norm_q8(hipStream_t st, int xdt, int rdt, int ydt, int T, int d, int norm, float eps, const void* x,
                          size_t ldx, const void* r, size_t ldr, void* r_out, size_t ldro, const float* w, int8_t* q,
                          float* s, void* y, size_t ldy) {
  const NormArgs a{x, r, r_out, w, q, s, y, ldx, ldr, ldro, ldy, (double)eps, T, d, norm, xdt, rdt, ydt};
  const auto apart = [](const void* p, size_t ld, int dt) {     // pieces of 8 at 16-byte places
    return p && (((uintptr_t)p & 15u) || ld * (dt == DT_F32 ? 4 : 2) % 16 != 0);
  };
  if (d % 8 != 0 || d > 32768 || ((uintptr_t)w & 15u) || apart(x, ldx, xdt) || apart(r, ldr, rdt) || apart(r_out, ldro, rdt) ||
      apart(y, ldy, ydt)) {
    k_norm_q8_any<<<dim3(T), dim3(kBlock), 0, st>>>(a);
    return hipGetLastError();
  }
  const int pieces = d / 8;
  if (pieces <= 64) norm_run<64, 1>(st, a);
  else if (pieces <= 128 && T > 512) norm_run<64, 2>(st, a);
  else if (pieces <= 256) norm_run<256, 1>(st, a);
  else if (pieces <= 512 && T > 512) norm_run<256, 2>(st, a);
  else if (pieces <= 512) norm_run<512, 1>(st, a);              // few rows: all the threads they take
  else if (pieces <= 1024) norm_run<512, 2>(st, a);
  else if (pieces <= 2048) norm_run<512, 4>(st, a);
  else norm_run<1024, 4>(st, a);
  return hipGetLastError();
}

}  // namespace sfx
