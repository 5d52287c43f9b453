// Residual addition, root-mean-square norm and int8 rows.
//
//   h = x + r;  n = h w / sqrt(mean h^2 + eps)  (or n = h);  s = fp32(max |n| / 127),
//   q = clamp(rne(n / s), -127, 127);  y = n rounded to its type;  r' = h rounded to r's type
//
// Sums, products and quotients are taken in 64 bits: a code next to a rounding border then
// falls the same way wherever it is computed, and 64-bit operations run at the rate of 32-bit
// ones here, so a row's bytes stay what bounds it.  n * (1 / s) decides a code unless it comes
// to rest within 2^-30 of a border, where the quotient itself is taken.
//
// A workgroup takes a row.
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
  int T, d, norm;
};

__device__ __forceinline__ double lane_xor_f64(double v, int o) {
  const int lo = __shfl_xor(__double2loint(v), o), hi = __shfl_xor(__double2hiint(v), o);
  return __hiloint2double(hi, lo);
}

template <int XT, int RT, int YT>
__global__ __launch_bounds__(kBlock) void k_norm_q8_simple(NormArgs a) {
  __shared__ double sh[2][kWavesPerBlock];
  const int t = blockIdx.x, wave = threadIdx.x >> 6;
  const size_t ox = (size_t)t * a.ldx, orr = (size_t)t * a.ldr;
  double sum = 0., top = 0.;
  bool bad = false;
  for (int i = threadIdx.x; i < a.d; i += kBlock) {
    double h = (double)load_elem<XT>(a.x, ox + i);
    if (a.r) h += (double)load_elem<RT>(a.r, orr + i);
    sum = fma(h, h, sum);
    const double v = fabs(a.w ? h * (double)a.w[i] : h);
    bad |= !(v < INFINITY);
    top = fmax(top, v);
  }
#pragma unroll
  for (int o = 32; o; o >>= 1) {
    sum += lane_xor_f64(sum, o);
    top = fmax(top, lane_xor_f64(top, o));
  }
  if ((threadIdx.x & 63) == 0) {
    sh[0][wave] = sum;
    sh[1][wave] = top;
  }
  bad = __syncthreads_or(bad);
  sum = top = 0.;
  for (int k = 0; k < kWavesPerBlock; ++k) {
    sum += sh[0][k];
    top = fmax(top, sh[1][k]);
  }
  const double f = a.norm ? 1.0 / sqrt(sum / a.d + a.eps) : 1.0;
  const float s = bad ? __uint_as_float(0x7FC00000u) : (float)(top * f / 127.0);
  const double sd = (double)s, inv = 1.0 / sd;
  if (a.s && threadIdx.x == 0) a.s[t] = s;
  for (int i = threadIdx.x; i < a.d; i += kBlock) {
    double h = (double)load_elem<XT>(a.x, ox + i);
    if (a.r) h += (double)load_elem<RT>(a.r, orr + i);
    if (a.r_out) store_elem<RT>(a.r_out, (size_t)t * a.ldro + i, (float)h);
    double n = h * f;
    if (a.w) n *= (double)a.w[i];
    if (a.y) store_elem<YT>(a.y, (size_t)t * a.ldy + i, (float)n);
    if (a.q) {
      const double v = n * inv;
      double c = rint(v);
      if (fabs(fabs(v - c) - 0.5) < 0x1p-30) c = rint(n / sd);
      a.q[(size_t)t * a.d + i] = s > 0.f ? (int8_t)(int)fmin(fmax(c, -127.), 127.) : (int8_t)0;
    }
  }
}

template <int XT, int RT>
void norm_run(hipStream_t st, const NormArgs& a, int ydt) {
  const dim3 g(a.T), b(kBlock);
  if (ydt == DT_F32) k_norm_q8_simple<XT, RT, DT_F32><<<g, b, 0, st>>>(a);
  else if (ydt == DT_F16) k_norm_q8_simple<XT, RT, DT_F16><<<g, b, 0, st>>>(a);
  else k_norm_q8_simple<XT, RT, DT_BF16><<<g, b, 0, st>>>(a);
}
template <int XT>
void norm_run(hipStream_t st, const NormArgs& a, int rdt, int ydt) {
  if (rdt == DT_F32) norm_run<XT, DT_F32>(st, a, ydt);
  else if (rdt == DT_F16) norm_run<XT, DT_F16>(st, a, ydt);
  else norm_run<XT, DT_BF16>(st, a, ydt);
}

}  // namespace

hipError_t launch_norm_q8(hipStream_t st, int xdt, int rdt, int ydt, int T, int d, int norm, float eps, const void* x,
                          size_t ldx, const void* r, size_t ldr, void* r_out, size_t ldro, const float* w, int8_t* q,
                          float* s, void* y, size_t ldy) {
  const NormArgs a{x, r, r_out, w, q, s, y, ldx, ldr, ldro, ldy, (double)eps, T, d, norm};
  if (!r) rdt = xdt;
  if (!y) ydt = DT_F16;
  if (xdt == DT_F32) norm_run<DT_F32>(st, a, rdt, ydt);
  else if (xdt == DT_F16) norm_run<DT_F16>(st, a, rdt, ydt);
  else norm_run<DT_BF16>(st, a, rdt, ydt);
  return hipGetLastError();
}

}  // namespace sfx
