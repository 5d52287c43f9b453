// y[t][i] (+)= sx[t] sw[i] sum_c X[t][c] W[i][c] + bias[i] for int8 rows X (a scale per token)
// and int8 weights W (a scale per row), any number of tokens.
//
// The sum of products is taken by int8 products in 32-bit integers and is exact (d <= 131056: at
// most 2^31 - 2^18), so how it is cut changes no bit; what follows is fp32.  Two kernels:
//   few    16 NT tokens x 16 RT rows per workgroup, whose waves deal the columns among themselves,
//          operands straight from memory, sums joined in LDS;
//   tiles  256 x 256 or 128 x 128, operands through LDS by direct copies.
//
// Lane layouts (checked against CPU products): v_mfma_i32_16x16x64_i8 lane l holds
// A[l % 16][16 (l / 16) + 0..15], B[16 (l / 16) + 0..15][l % 16], and D[4 (l / 16) + i][l % 16], i < 4;
// v_mfma_i32_32x32x32_i8 A[l % 32][16 (l / 32) + 0..15], B alike, D[8 (i / 4) + 4 (l / 32) + i % 4][l % 32],
// i < 16.
#include <algorithm>

#include "sfx_launch.hpp"
#include "sfx_turn.hpp"

namespace sfx {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

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

// x, or 0 in lanes whose mask is 0.  (A zero assigned under a condition of the lane came out for some of
// the registers only.)
__device__ __forceinline__ void keep(Raw<16>& x, uint32_t mask) {
#pragma unroll
  for (int i = 0; i < 4; ++i) x.w[i] &= mask;
}

template <int YT>
__device__ __forceinline__ void lin8_store(const Linear8Args& a, int t, int i, int sum) {
  float v = (float)sum * (a.sx[t] * a.sw[i]);
  if (a.bias) v += a.bias[i];
  const size_t at = (size_t)t * a.ldy + i;
  if (a.accumulate) v += load_elem<YT>(a.y, at);
  store_elem<YT>(a.y, at, v);
}

// ---- few tokens

// A wave takes pairs of 64-column units, every W-th pair, P units on the way.
template <int YT, int NT, int RT, int W, int P>
__global__ __launch_bounds__(W * kWave) void k_linear_q8_few(Linear8Args a) {
  constexpr int TT = 16 * NT, RR = 16 * RT, LS = RR + 1;
  __shared__ int sum[W * TT * LS];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), m = lane & 15, c = lane >> 4;
  const int row0 = blockIdx.x * RR, tok0 = blockIdx.y * TT;
  const int8_t *w[RT], *x[NT];
#pragma unroll
  for (int i = 0; i < RT; ++i) w[i] = a.W + (size_t)min(row0 + 16 * i + m, a.n - 1) * a.d;
#pragma unroll
  for (int i = 0; i < NT; ++i) x[i] = a.x + (size_t)min(tok0 + 16 * i + m, a.T - 1) * a.ldx;
  const int pairs = (a.d + 127) / 128, mine = 2 * ((pairs - wave + W - 1) / W);   // units of this wave
  Raw<16> wf[P][RT], xf[P][NT];
  const auto column = [&](int q) { return (((q >> 1) * W + wave) * 2 + (q & 1)) * 64 + 16 * c; };
  const auto fetch = [&](int q, Raw<16>(&wq)[RT], Raw<16>(&xq)[NT]) {
    const int at = min(column(q), a.d - 16);
#pragma unroll
    for (int i = 0; i < RT; ++i) wq[i] = load_raw<16>(w[i] + at);
#pragma unroll
    for (int i = 0; i < NT; ++i) xq[i] = load_raw<16>(x[i] + at);
  };
  i32x4 acc[NT][RT];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < RT; ++i) acc[t][i] = i32x4{0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < P; ++j) fetch(j, wf[j], xf[j]);
  for (int q = 0; q < mine; q += P) {
#pragma unroll
    for (int j = 0; j < P; ++j) {
      if (column(q + j) - 16 * c + 64 > a.d) {                 // the last columns: products with 0 past the end
        const uint32_t mask = column(q + j) < a.d ? ~0u : 0u;
#pragma unroll
        for (int t = 0; t < NT; ++t) keep(xf[j][t], mask);
      }
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < RT; ++i) acc[t][i] = mma8(xf[j][t], wf[j][i], acc[t][i]);
      if (q + P < mine) fetch(q + P + j, wf[j], xf[j]);
    }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[(wave * TT + 16 * t + 4 * c + e) * LS + 16 * i + m] = acc[t][i][e];
  __syncthreads();
  const int tokens = min(TT, a.T - tok0);
  for (int e = threadIdx.x; e < tokens * RR; e += W * kWave) {
    const int tok = e / RR, row = e % RR;
    if (row0 + row >= a.n) continue;
    int v = 0;
#pragma unroll
    for (int k = 0; k < W; ++k) v += sum[(k * TT + tok) * LS + row];
    lin8_store<YT>(a, tok0 + tok, row0 + row, v);
  }
}

// ---- many tokens

constexpr int kBK = 128;               // columns of a stage

// BN rows x BT tokens by WN x WT waves, rows as the first operand (a lane ends with four
// neighbouring outputs of one token).  Two stages of LDS: the barrier that ends a stage stands in front of its last
// quarter's products, which are in registers by then, so that the next stage's first operands
// are read while they run, and the stage after it is copied into what the barrier has freed.  A row's
// 16-byte chunks are swizzled by (row / 2) % 8: 16 lanes that read one chunk of 16 rows meet all
// banks once.
template <int YT, int BN, int BT, int WN, int WT>
__global__ __launch_bounds__(WN * WT * kWave) void k_linear_q8_tiles(Linear8Args a, int tn, int tt) {
  constexpr int NTH = WN * WT * kWave, MI = BN / WN / 32, NI = BT / WT / 32, LA = BN * 8 / NTH, LB = BT * 8 / NTH;
  static_assert(MI % 2 == 0 && BN % (NTH / 8) == 0 && BT % (NTH / 8) == 0 && NTH % 128 == 0, "tile");
  // two objects: copies into one are then no reason to wait before reads of the other
  __shared__ __attribute__((aligned(16))) uint8_t buf0[(BN + BT) * kBK];
  __shared__ __attribute__((aligned(16))) uint8_t buf1[(BN + BT) * kBK];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wn = wave / WT, wt = wave % WT, r = lane & 31, c = lane >> 5;
  // workgroups 8 apart are on one XCD: it takes a run of tiles, eight token tiles under each row tile
  const int total = tn * tt, per = (total + 7) / 8, id = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
  if ((int)(blockIdx.x >> 3) >= per || id >= total) return;
  const int group = id / (8 * tn), in_group = id % (8 * tn), deep = min(8, tt - group * 8);
  const int t0 = (group * 8 + in_group % deep) * BT, n0 = in_group / deep * BN;
  const int8_t* wb = a.W + (size_t)n0 * a.d;
  const int8_t* xb = a.x + (size_t)t0 * a.ldx;
  const int lrow = threadIdx.x >> 3, chunk = ((threadIdx.x & 7) ^ ((lrow >> 1) & 7)) * 16;
  size_t off[LA + LB];
#pragma unroll
  for (int j = 0; j < LA + LB; ++j) {
    const int row = j * (NTH / 8) + lrow;
    off[j] = j < LA ? (size_t)min(row, a.n - 1 - n0) * a.d : (size_t)min(row - BN, a.T - 1 - t0) * a.ldx;
  }
  const auto fetch = [&](int s, uint8_t* buf) {
    const int k = min(s * kBK + chunk, a.d - 16);
#pragma unroll
    for (int j = 0; j < LA + LB; ++j)
      __builtin_amdgcn_global_load_lds((const void*)((j < LA ? wb : xb) + off[j] + k),
                                       (__attribute__((address_space(3))) void*)(buf + (j * NTH + wave * kWave) * 16), 16, 0, 0);
  };
  i32x16 acc[MI][NI];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j) acc[i][j] = i32x16{0};
  struct Frag {
    Raw<16> a[MI], b[NI];
  };
  const int ra = wn * MI * 32 + r, rb = BN + wt * NI * 32 + r, swizzle = (r >> 1) & 7;
  const auto load = [&](const uint8_t* buf, int ks, Frag& f) {
    const int p = ((ks * 2 + c) ^ swizzle) * 16;
#pragma unroll
    for (int i = 0; i < MI; ++i) f.a[i] = load_raw<16>(buf + (ra + 32 * i) * kBK + p);
#pragma unroll
    for (int j = 0; j < NI; ++j) f.b[j] = load_raw<16>(buf + (rb + 32 * j) * kBK + p);
  };
  const auto mma = [&](const Frag& f) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4, f.a[i]), __builtin_bit_cast(i32x4, f.b[j]),
                                                          acc[i][j], 0, 0, 0);
  };
  // the next operands' reads dealt out among the products
  const auto mix = [&]() {
#pragma unroll
    for (int q = 0; q < MI + NI; ++q) {
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);                       // a read of LDS
      __builtin_amdgcn_sched_group_barrier(0x008, MI * NI / (MI + NI), 0);     // matrix products
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  const int S = (a.d + kBK - 1) / kBK;
  Frag f0, f1;
  const auto body = [&](uint8_t* cur, const uint8_t* next, int s) {
    load(cur, 1, f1);
    mma(f0);
    mix();
    load(cur, 2, f0);
    mma(f1);
    mix();
    load(cur, 3, f1);
    mma(f0);
    mix();
    __syncthreads();                                           // `next` has landed, `cur` has been read
    if (s + 2 < S) fetch(s + 2, cur);
    load(next, 0, f0);
    mma(f1);
    mix();
  };
  const auto last = [&](const uint8_t* cur, int s) {
    const int left = (a.d - s * kBK) >> 4;                     // chunks of the last stage
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      Frag f;
      load(cur, ks, f);
      const uint32_t mask = 2 * ks + c < left ? ~0u : 0u;
#pragma unroll
      for (int j = 0; j < NI; ++j) keep(f.b[j], mask);
      mma(f);
    }
  };
  fetch(0, buf0);
  __syncthreads();
  if (S > 1) fetch(1, buf1);
  load(buf0, 0, f0);
  int s = 0;
  for (; s + 2 < S; s += 2) {
    body(buf0, buf1, s);
    body(buf1, buf0, s + 1);
  }
  if (s + 1 < S) {
    body(buf0, buf1, s);
    last(buf1, s + 1);
  } else {
    last(buf0, s);
  }

  // out by way of LDS, 32 tokens x 64 rows of a wave at a time: straight from the registers a
  // store instruction would write 64 pieces of 8 bytes (240 us of 780 at 8192 x 16384 x 4096)
  constexpr int LS = 68, esz = YT == DT_F32 ? 4 : 2;
  static_assert(NTH / 128 * 32 * LS * 4 <= (BN + BT) * kBK, "staging");
  __syncthreads();
  float* st = (float*)((wave & 1) ? buf1 : buf0) + (wave >> 1) * (32 * LS);
  const bool vec = ((uintptr_t)a.y & 15u) == 0 && a.ldy * esz % 16 == 0;
  const int col = (lane & 7) * 8;
#pragma unroll
  for (int i2 = 0; i2 < MI; i2 += 2) {
    const int nb = n0 + wn * MI * 32 + i2 * 32 + col;
    float sw[8], bias[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int n = min(nb + e, a.n - 1);
      sw[e] = a.sw[n];
      bias[e] = a.bias ? a.bias[n] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const int tb = t0 + wt * NI * 32 + j * 32;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          f32x4 v;
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = (float)acc[i2 + i][j][4 * q + e];
          *(f32x4*)(st + r * LS + i * 32 + 8 * q + 4 * c) = v;
        }
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        const int tr = it * 8 + (lane >> 3), t = tb + tr;
        const f32x4 v0 = *(const f32x4*)(st + tr * LS + col), v1 = *(const f32x4*)(st + tr * LS + col + 4);
        if (t >= a.T) continue;
        const float sx = a.sx[t];
        float o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = (e < 4 ? v0[e & 3] : v1[e & 3]) * (sx * sw[e]) + bias[e];
        const size_t at = (size_t)t * a.ldy + nb;
        if (vec && nb + 8 <= a.n) {
          if (a.accumulate) {
            float was[8];
            widen<YT>(load8<YT, true>(a.y, at), was);
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] += was[e];
          }
          store8<YT>(a.y, at, o);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (nb + e < a.n) store_elem<YT>(a.y, at + e, a.accumulate ? o[e] + load_elem<YT>(a.y, at + e) : o[e]);
        }
      }
    }
  }
}

template <int YT, int NT, int RT, int W, int P>
void few_run(hipStream_t st, const Linear8Args& a) {
  const dim3 g((a.n + 16 * RT - 1) / (16 * RT), (a.T + 16 * NT - 1) / (16 * NT));
  k_linear_q8_few<YT, NT, RT, W, P><<<g, dim3(W * kWave), 0, st>>>(a);
}
template <int YT, int BN, int BT, int WN, int WT>
void tiles_run(hipStream_t st, const Linear8Args& a) {
  const int tn = (a.n + BN - 1) / BN, tt = (a.T + BT - 1) / BT;
  k_linear_q8_tiles<YT, BN, BT, WN, WT><<<dim3((tn * tt + 7) / 8 * 8), dim3(WN * WT * kWave), 0, st>>>(a, tn, tt);
}

template <int YT>
void lin8_run(hipStream_t st, const Linear8Args& a) {
  const auto tiles = [&](int b) { return (long long)((a.n + b - 1) / b) * ((a.T + b - 1) / b); };
  if (a.T <= 16) return few_run<YT, 1, 1, 8, 4>(st, a);
  if (a.T <= 32) return few_run<YT, 2, 2, 8, 2>(st, a);
  if (a.T <= 48) return few_run<YT, 3, 3, 8, 2>(st, a);
  if (a.T <= 64) return few_run<YT, 4, 3, 8, 2>(st, a);
  if (tiles(256) >= 256) return tiles_run<YT, 256, 256, 2, 4>(st, a);
  if (tiles(128) >= 128) return tiles_run<YT, 128, 128, 2, 2>(st, a);
  few_run<YT, 4, 4, 8, 2>(st, a);
}

}  // namespace

hipError_t launch_linear_q8(hipStream_t st, int ydt, int T, int n, int d, const int8_t* x, size_t ldx, const float* sx,
                            const int8_t* W, const float* sw, const float* bias, int accumulate, void* y, size_t ldy) {
  const Linear8Args a{x, ldx, sx, W, sw, bias, y, ldy, T, n, d, accumulate};
  if (ydt == DT_F32) lin8_run<DT_F32>(st, a);
  else if (ydt == DT_F16) lin8_run<DT_F16>(st, a);
  else lin8_run<DT_BF16>(st, a);
  return hipGetLastError();
}

}  // namespace sfx
