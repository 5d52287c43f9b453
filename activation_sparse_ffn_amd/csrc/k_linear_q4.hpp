// y[b][i] (+)= sum_c W[i][c] x[b][c] + bias[i] for int4 weights with one fp16 scale per
// group of 32, 64 or 128 columns, 1..64 tokens (the projections around the FFN step, in
// the storage of its int4 rows).
//
// Tokens are the rows and 16 weight rows the columns of 16x16x32 products, so a lane
// meets one weight row only and needs one scale per group.  A lane's 16-byte load is one
// group of 32 codes of its row (four lanes cover 128 columns of 16 rows); a 4 x 4
// transposition over the wave's quarters turns the four loaded words into the operands of
// four products, one per group.  The waves of a workgroup share 16 R rows and deal the
// 128-column chunks among themselves; their sums are added in wave order through LDS, so
// y is bitwise reproducible.
#pragma once
#include "sfx_launch.hpp"
#include "sfx_q4.hpp"

namespace sfx {
namespace {

struct LinearArgs {
  const uint8_t* x;
  size_t ldx;               // bytes between token rows of x
  const uint8_t* W;
  const uint16_t* s;
  const float* bias;
  float* y;
  size_t ldy;               // elements between token rows of y
  int B, n, d, accumulate;
};

constexpr int kLinWaves = 8;

// Token that row m of token tile nt stands for.  NI accumulator rows per lane are used:
// below 16 tokens the tokens are spread over the quarters (row 4 c + i is token NI c + i),
// so only NI of a lane's four sums are scaled.
template <int NI>
__device__ __forceinline__ int lin_token(int nt, int m) {
  return NI == 4 ? 16 * nt + m : NI * (m >> 2) + (m & (NI - 1));
}

template <class T, int NT, int NI, int R, int GSH>
__global__ __launch_bounds__(kLinWaves * kWave) void k_linear_q4(LinearArgs a) {
  __shared__ float red[kLinWaves][16 * R][4 * NI * NT + 1];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x >> 6;
  const int m = lane & 15, c = lane >> 4;
  const int row0 = blockIdx.x * 16 * R;
  const int ng = a.d >> 5, nsc = ng >> GSH;
  const int nchunk = (ng + 3) >> 2;
  const uint8_t* wrow[R];
  const uint16_t* srow[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int row = min(row0 + 16 * r + m, a.n - 1);
    wrow[r] = a.W + (size_t)row * (a.d >> 1);
    srow[r] = a.s + (size_t)row * nsc;
  }
  const uint8_t* xrow[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) xrow[t] = a.x + (size_t)min(lin_token<NI>(t, m), a.B - 1) * a.ldx;

  float acc[R][NT][NI];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < NI; ++i) acc[r][t][i] = 0.f;
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  const Q4<T> dec;

  for (int ck = wave; ck < nchunk; ck += kLinWaves) {
    uint32_t w[R][4];
    float sc[R][4];
    const int gl = min(4 * ck + c, ng - 1);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const Raw<16> q = load_raw<16>(wrow[r] + (size_t)gl * 16);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[r][j] = q.w[j] ^ 0x88888888u;
        sc[r][j] = (float)__builtin_bit_cast(_Float16, srow[r][min(4 * ck + j, ng - 1) >> GSH]);
      }
      quarter_transpose(w[r]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (4 * ck + j < ng) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const Raw<16> xv = load_raw<16>(xrow[t] + (size_t)(4 * ck + j) * 64 + c * 16);
          Raw<16> xp;                              // columns in the order of q4_word's registers
          xp.w[0] = __builtin_amdgcn_perm(xv.w[2], xv.w[0], 0x05040100u);
          xp.w[1] = __builtin_amdgcn_perm(xv.w[2], xv.w[0], 0x07060302u);
          xp.w[2] = __builtin_amdgcn_perm(xv.w[3], xv.w[1], 0x05040100u);
          xp.w[3] = __builtin_amdgcn_perm(xv.w[3], xv.w[1], 0x07060302u);
          f32x4 c24 = zero;
          if constexpr (Q4<T>::offset) c24 = Mma<T>::run(xp, Q4<T>::minus24(), zero);
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const f32x4 p = Mma<T>::run(xp, dec.word(w[r][j]), c24);
#pragma unroll
            for (int i = 0; i < NI; ++i) acc[r][t][i] = fmaf(sc[r][j], p[i], acc[r][t][i]);
          }
        }
      }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < NI; ++i) red[wave][16 * r + m][(4 * t + c) * NI + i] = acc[r][t][i];
  __syncthreads();
  constexpr int TT = 4 * NI * NT;
  for (int e = threadIdx.x; e < 16 * R * TT; e += kLinWaves * kWave) {
    const int row = e % (16 * R), tok = e / (16 * R);
    if (row0 + row < a.n && tok < a.B) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kLinWaves; ++w) v += red[w][row][tok];
      if (a.bias) v += a.bias[row0 + row];
      float* y = a.y + (size_t)tok * a.ldy + row0 + row;
      *y = a.accumulate ? *y + v : v;
    }
  }
}

template <class T, int NT, int NI, int R>
hipError_t lin_run(hipStream_t s, const LinearArgs& a, int gsh) {
  const dim3 grid((a.n + 16 * R - 1) / (16 * R)), blk(kLinWaves * kWave);
  if (gsh == 0) k_linear_q4<T, NT, NI, R, 0><<<grid, blk, 0, s>>>(a);
  else if (gsh == 1) k_linear_q4<T, NT, NI, R, 1><<<grid, blk, 0, s>>>(a);
  else k_linear_q4<T, NT, NI, R, 2><<<grid, blk, 0, s>>>(a);
  return hipGetLastError();
}

template <class T>
hipError_t lin_launch(hipStream_t s, const LinearArgs& a, int gsh) {
  if (a.B <= 4) return lin_run<T, 1, 1, 1>(s, a, gsh);
  if (a.B <= 8) return lin_run<T, 1, 2, 1>(s, a, gsh);
  if (a.B <= 16) return lin_run<T, 1, 4, 1>(s, a, gsh);
  if (a.B <= 32) return lin_run<T, 2, 4, 1>(s, a, gsh);
  return lin_run<T, 4, 4, 1>(s, a, gsh);
}

}  // namespace
}  // namespace sfx
