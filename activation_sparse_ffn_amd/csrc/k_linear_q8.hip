// y[t][i] (+)= sx[t] sw[i] sum_c X[t][c] W[i][c] + bias[i] for int8 rows X (a scale per token)
// and int8 weights W (a scale per row), any number of tokens.
//
// The sum of products is taken by 16x16x64 int8 products in 32-bit integers and is exact
// (d <= 131056: at most 2^31 - 2^18); what follows is fp32.
//
// Lane layout of v_mfma_i32_16x16x64_i8: lane l holds A[l % 16][16 (l / 16) + 0..15],
// B[16 (l / 16) + 0..15][l % 16], and D[4 (l / 16) + i][l % 16] for i = 0..3.
#include "sfx_launch.hpp"
#include "sfx_turn.hpp"

namespace sfx {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

struct Linear8Args {
  const int8_t* x;
  size_t ldx;
  const float* sx;
  const int8_t* W;
  const float* sw;
  const float* bias;
  void* y;
  size_t ldy;
  int T, n, d, accumulate;
};

__device__ __forceinline__ i32x4 mma8(const Raw<16>& a, const Raw<16>& b, i32x4 c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
}

template <int YT>
__device__ __forceinline__ void lin8_store(const Linear8Args& a, int t, int i, int sum) {
  float v = (float)sum * (a.sx[t] * a.sw[i]);
  if (a.bias) v += a.bias[i];
  const size_t at = (size_t)t * a.ldy + i;
  if (a.accumulate) v += load_elem<YT>(a.y, at);
  store_elem<YT>(a.y, at, v);
}

// 16 weight rows and 64 tokens per workgroup; the waves deal the columns among themselves.
template <int YT>
__global__ __launch_bounds__(kBlock) void k_linear_q8_simple(Linear8Args a) {
  constexpr int NT = 4;
  __shared__ int sum[kWavesPerBlock][NT * 16][17];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, m = lane & 15, c = lane >> 4;
  const int row0 = blockIdx.x * 16, tok0 = blockIdx.y * (16 * NT);
  const int8_t* w = a.W + (size_t)min(row0 + m, a.n - 1) * a.d;
  const int8_t* x[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) x[t] = a.x + (size_t)min(tok0 + 16 * t + m, a.T - 1) * a.ldx;
  i32x4 acc[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) acc[t] = i32x4{0, 0, 0, 0};
  for (int k = wave * 64 + 16 * c; k - 16 * c < a.d; k += kWavesPerBlock * 64) {
    const bool in = k < a.d;
    const int at = in ? k : 0;
    const Raw<16> wf = load_raw<16>(w + at);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      Raw<16> xf = load_raw<16>(x[t] + at);
      if (!in) xf = zero16();
      acc[t] = mma8(xf, wf, acc[t]);
    }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) sum[wave][16 * t + 4 * c + i][m] = acc[t][i];
  __syncthreads();
  for (int e = threadIdx.x; e < NT * 16 * 16; e += kBlock) {
    const int tok = e / 16, row = e % 16;
    if (tok0 + tok >= a.T || row0 + row >= a.n) continue;
    int v = 0;
    for (int k = 0; k < kWavesPerBlock; ++k) v += sum[k][tok][row];
    lin8_store<YT>(a, tok0 + tok, row0 + row, v);
  }
}

}  // namespace

hipError_t launch_linear_q8(hipStream_t st, int ydt, int T, int n, int d, const int8_t* x, size_t ldx, const float* sx,
                            const int8_t* W, const float* sw, const float* bias, int accumulate, void* y, size_t ldy) {
  const Linear8Args a{x, ldx, sx, W, sw, bias, y, ldy, T, n, d, accumulate};
  const dim3 g((n + 15) / 16, (T + 63) / 64), b(kBlock);
  if (ydt == DT_F32) k_linear_q8_simple<DT_F32><<<g, b, 0, st>>>(a);
  else if (ydt == DT_F16) k_linear_q8_simple<DT_F16><<<g, b, 0, st>>>(a);
  else k_linear_q8_simple<DT_BF16><<<g, b, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace sfx
