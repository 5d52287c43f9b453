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

// Columns of an 8-column slice in the order of the decoder's registers: (0 4) (1 5) (2 6) (3 7).
__device__ __forceinline__ Raw<16> lin_order(const Raw<16>& x) {
  Raw<16> p;
  p.w[0] = __builtin_amdgcn_perm(x.w[2], x.w[0], 0x05040100u);
  p.w[1] = __builtin_amdgcn_perm(x.w[2], x.w[0], 0x07060302u);
  p.w[2] = __builtin_amdgcn_perm(x.w[3], x.w[1], 0x05040100u);
  p.w[3] = __builtin_amdgcn_perm(x.w[3], x.w[1], 0x07060302u);
  return p;
}

// A chunk of 128 columns of 16 weight rows: 32 codes of group c of row m, and the row's four
// scales (packed as they lie: 4 >> GSH of them).
template <int GSH>
struct LinChunk {
  Raw<16> q;
  uint32_t s[2];
};
template <int GSH>
__device__ __forceinline__ void lin_load(const uint8_t* wrow, const uint16_t* srow, int ck, int c, int ng,
                                         LinChunk<GSH>& x) {
  x.q = load_raw<16>(wrow + (size_t)min(4 * ck + c, ng - 1) * 16);
  if constexpr (GSH == 2) {
    x.s[0] = srow[ck];
  } else {
    // the last chunk may end inside: its scales are loaded one by one
    if (4 * ck + 4 <= ng) {
      typedef uint32_t __attribute__((aligned(2))) u32a2;
      const u32a2* p = (const u32a2*)(srow + ((4 * ck) >> GSH));
      x.s[0] = p[0];
      if constexpr (GSH == 0) x.s[1] = p[1];
    } else {
      const int last = ((ng - 1) >> GSH), s0 = (4 * ck) >> GSH;
      x.s[0] = srow[s0] | (uint32_t)srow[min(s0 + 1, last)] << 16;
      if constexpr (GSH == 0) x.s[1] = srow[min(s0 + 2, last)] | (uint32_t)srow[min(s0 + 3, last)] << 16;
    }
  }
}
template <int GSH>
__device__ __forceinline__ float lin_scale(const LinChunk<GSH>& x, int j) {
  if constexpr (GSH == 0) return half_at(x.s[j >> 1], j & 1);
  else if constexpr (GSH == 1) return half_at(x.s[0], j >> 1);
  else return half_at(x.s[0], 0);
}

// XLDS: x lies in LDS, ordered, token rows d * 2 + 16 bytes apart (the 16 put eight tokens on
// different banks).  AHEAD chunks of a wave's weights are on the way at a time.
template <class T, int NT, int NI, int R, int GSH, bool XLDS, int AHEAD>
__global__ __launch_bounds__(kLinWaves * kWave) void k_linear_q4(LinearArgs a) {
  constexpr int TT = 4 * NI * NT, kThreads = kLinWaves * kWave;
  extern __shared__ __attribute__((aligned(16))) uint8_t sh[];
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = lane & 15, c = lane >> 4;
  const int row0 = blockIdx.x * 16 * R;
  const int ng = a.d >> 5, nsc = ng >> GSH;
  const int nchunk = (ng + 3) >> 2;
  // the wave's chunks: a run of its own, so its rows are read in whole lines
  const int per = (nchunk + kLinWaves - 1) / kLinWaves;
  const int ck0 = wave * per, ck1 = min(nchunk, ck0 + per);
  const uint8_t* wrow[R];
  const uint16_t* srow[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int row = min(row0 + 16 * r + m, a.n - 1);
    wrow[r] = a.W + (size_t)row * (a.d >> 1);
    srow[r] = a.s + (size_t)row * nsc;
  }
  LinChunk<GSH> w[AHEAD][R];
#pragma unroll
  for (int u = 0; u < AHEAD; ++u)
    if (ck0 + u < ck1) {
#pragma unroll
      for (int r = 0; r < R; ++r) lin_load<GSH>(wrow[r], srow[r], ck0 + u, c, ng, w[u][r]);
    }
  const int xstride = a.d * 2 + 16;
  const uint8_t* xrow[NT];
  if constexpr (XLDS) {
    const int pieces = a.d >> 3;
    for (int b = 0; b < a.B; ++b)
      for (int i = threadIdx.x; i < pieces; i += kThreads)
        *reinterpret_cast<Raw<16>*>(sh + b * xstride + i * 16) = lin_order(load_raw<16>(a.x + (size_t)b * a.ldx + i * 16));
    __syncthreads();
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int tok = min(lin_token<NI>(t, m), a.B - 1);
    xrow[t] = (XLDS ? sh + tok * xstride : a.x + (size_t)tok * a.ldx) + c * 16;
  }

  float acc[R][NT][NI];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < NI; ++i) acc[r][t][i] = 0.f;
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  const Q4<T> dec;

  for (int ckb = ck0; ckb < ck1; ckb += AHEAD) {
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      const int ck = ckb + u;
      if (ck < ck1) {
        uint32_t k[R][4];
        float sc[R][4];
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            k[r][j] = w[u][r].q.w[j] ^ 0x88888888u;
            sc[r][j] = lin_scale<GSH>(w[u][r], j);
          }
          quarter_transpose(k[r]);
        }
        if (ck + AHEAD < ck1) {
#pragma unroll
          for (int r = 0; r < R; ++r) lin_load<GSH>(wrow[r], srow[r], ck + AHEAD, c, ng, w[u][r]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (4 * ck + j < ng) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              Raw<16> xp = load_raw<16>(xrow[t] + (size_t)(4 * ck + j) * 64);
              if constexpr (!XLDS) xp = lin_order(xp);
              f32x4 from = zero;
              if constexpr (Q4<T>::offset) from = Mma<T>::run(xp, Q4<T>::minus24(), zero);
#pragma unroll
              for (int r = 0; r < R; ++r) {
                const f32x4 p = Mma<T>::run(xp, dec.word(k[r][j]), from);
#pragma unroll
                for (int i = 0; i < NI; ++i) acc[r][t][i] = fmaf(sc[r][j], p[i], acc[r][t][i]);
              }
            }
          }
        }
      }
    }
  }
  // the waves' sums in wave order: red[wave][row][token]
  float* red = (float*)sh;
  if constexpr (XLDS) __syncthreads();
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < NI; ++i) red[(wave * 16 * R + 16 * r + m) * (TT + 1) + (4 * t + c) * NI + i] = acc[r][t][i];
  __syncthreads();
  for (int e = threadIdx.x; e < 16 * R * TT; e += kThreads) {
    const int row = e % (16 * R), tok = e / (16 * R);
    if (row0 + row < a.n && tok < a.B) {
      float v = 0.f;
#pragma unroll
      for (int k = 0; k < kLinWaves; ++k) v += red[(k * 16 * R + row) * (TT + 1) + tok];
      if (a.bias) v += a.bias[row0 + row];
      float* y = a.y + (size_t)tok * a.ldy + row0 + row;
      *y = a.accumulate ? *y + v : v;
    }
  }
}

constexpr int kLinXLds = 64 << 10;       // x is kept in LDS up to here: two workgroups per compute unit

template <class T, int NT, int NI, int R, bool XLDS, int AHEAD>
hipError_t lin_run(hipStream_t s, const LinearArgs& a, int gsh) {
  const dim3 grid((a.n + 16 * R - 1) / (16 * R)), blk(kLinWaves * kWave);
  const size_t red = (size_t)kLinWaves * 16 * R * (4 * NI * NT + 1) * 4, xl = XLDS ? (size_t)a.B * (a.d * 2 + 16) : 0;
  const size_t lds = red > xl ? red : xl;
  if (gsh == 0) k_linear_q4<T, NT, NI, R, 0, XLDS, AHEAD><<<grid, blk, lds, s>>>(a);
  else if (gsh == 1) k_linear_q4<T, NT, NI, R, 1, XLDS, AHEAD><<<grid, blk, lds, s>>>(a);
  else k_linear_q4<T, NT, NI, R, 2, XLDS, AHEAD><<<grid, blk, lds, s>>>(a);
  return hipGetLastError();
}

template <class T>
hipError_t lin_launch(hipStream_t s, const LinearArgs& a, int gsh) {
  const bool x_lds = (size_t)a.B * (a.d * 2 + 16) <= (size_t)kLinXLds;
  if (a.B <= 4) return x_lds ? lin_run<T, 1, 1, 1, true, 4>(s, a, gsh) : lin_run<T, 1, 1, 1, false, 4>(s, a, gsh);
  if (a.B <= 8) return x_lds ? lin_run<T, 1, 2, 1, true, 4>(s, a, gsh) : lin_run<T, 1, 2, 1, false, 4>(s, a, gsh);
  if (a.B <= 16) return x_lds ? lin_run<T, 1, 4, 1, true, 4>(s, a, gsh) : lin_run<T, 1, 4, 1, false, 4>(s, a, gsh);
  if (a.B <= 32) return lin_run<T, 2, 4, 2, false, 1>(s, a, gsh);
  if (a.B <= 48) return lin_run<T, 3, 4, 2, false, 1>(s, a, gsh);
  return lin_run<T, 4, 4, 2, false, 1>(s, a, gsh);
}

}  // namespace
}  // namespace sfx
