// y[t][i] (+)= sx[t] sw[i] sum_c X[t][c] W[i][c] + bias[i] for int8 rows X (a scale per token)
// and int8 weights W (a scale per row), any number of tokens.
//
// The sum of products is taken by int8 products in 32-bit integers and is exact (d <= 131056: at
// most 2^31 - 2^18), so how it is cut changes no bit; what follows is fp32.  Three kernels:
//   one    a few tokens and rows: operands straight from memory;
//   few    16 NT tokens x 16 RT rows per workgroup, whose waves deal the columns among themselves,
//          lines copied into LDS, sums joined there;
//   tiles  256 x 256, 128 x 128 or 128 x 64, waves share what is copied into LDS.
// Few tokens are bound by the weights' bytes (1 x 4096 x 4096: 5.2 us, 3.2 TB/s; 64 x 11008 x 4096: 15, 3.1 TB/s),
// many by the matrix units and the operands' way through LDS (8192 x 16384 x 4096: 549 us, 2.0 POP/s).
//
// Lane layouts (checked against CPU products): v_mfma_i32_16x16x64_i8 lane l holds
// A[l % 16][16 (l / 16) + 0..15], B[16 (l / 16) + 0..15][l % 16], and D[4 (l / 16) + i][l % 16], i < 4;
// v_mfma_i32_32x32x32_i8 A[l % 32][16 (l / 32) + 0..15], B alike, D[8 (i / 4) + 4 (l / 32) + i % 4][l % 32],
// i < 16.
#include <algorithm>
#include <type_traits>

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
  int T, n, d, accumulate, ydt;
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

// One rounding of scales' product and one with the bias, written out so that every kernel takes the same.
__device__ __forceinline__ float lin8_value(float sum, float sx, float sw, float bias) { return __builtin_fmaf(sum, sx * sw, bias); }

__device__ __forceinline__ void lin8_store(const Linear8Args& a, int t, int i, int sum) {
  float v = lin8_value((float)sum, a.sx[t], a.sw[i], a.bias ? a.bias[i] : 0.f);
  const size_t at = (size_t)t * a.ldy + i;
  const auto put = [&](auto dt) {
    constexpr int YT = decltype(dt)::value;
    if (a.accumulate) v += load_elem<YT>(a.y, at);
    store_elem<YT>(a.y, at, v);
  };
  if (a.ydt == DT_F32) put(std::integral_constant<int, DT_F32>{});
  else if (a.ydt == DT_F16) put(std::integral_constant<int, DT_F16>{});
  else put(std::integral_constant<int, DT_BF16>{});
}

// ---- few tokens

// One workgroup per 16 rows, at most 16 tokens; a wave takes pairs of 64-column units, every W-th
// pair, P units on the way, operands straight from memory.
template <int W, int P>
__global__ __launch_bounds__(W * kWave) void k_linear_q8_one(Linear8Args a) {
  __shared__ int sum[W * 16 * 17];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), m = lane & 15, c = lane >> 4;
  const int row0 = blockIdx.x * 16;
  const int8_t* w = a.W + (size_t)min(row0 + m, a.n - 1) * a.d;
  const int8_t* x = a.x + (size_t)min(m, a.T - 1) * a.ldx;
  const int pairs = (a.d + 127) / 128, mine = 2 * ((pairs - wave + W - 1) / W);   // units of this wave
  Raw<16> wf[P], xf[P];
  const auto column = [&](int q) { return (((q >> 1) * W + wave) * 2 + (q & 1)) * 64; };
  const auto fetch = [&](int q, int j) {
    const int at = min(column(q) + 16 * c, a.d - 16);
    wf[j] = load_raw<16>(w + at);
    xf[j] = load_raw<16>(x + at);
  };
  i32x4 acc = {0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < P; ++j) fetch(j, j);
  for (int q = 0; q < mine; q += P) {
#pragma unroll
    for (int j = 0; j < P; ++j) {
      if (column(q + j) + 64 > a.d) keep(xf[j], column(q + j) + 16 * c < a.d ? ~0u : 0u);   // products with 0 past the end
      acc = mma8(xf[j], wf[j], acc);
      if (q + P < mine) fetch(q + P + j, j);
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) sum[(wave * 16 + 4 * c + e) * 17 + m] = acc[e];
  __syncthreads();
  for (int e = threadIdx.x; e < min(16, a.T) * 16; e += W * kWave) {
    const int tok = e / 16, row = e % 16;
    if (row0 + row >= a.n) continue;
    int v = 0;
#pragma unroll
    for (int k = 0; k < W; ++k) v += sum[(k * 16 + tok) * 17 + row];
    lin8_store(a, tok, row0 + row, v);
  }
}

// 16 NT tokens x 16 RT rows; a wave takes 128 columns of all of them at a time, copied into its own
// part of LDS in whole 128-byte lines (operands read straight from memory ask for half lines
// of 16 rows at a time: 20.0 us instead of 15.0 at 64 x 11008 x 4096).  The waves' copies overlap each
// other, not their own products.  A row's 16-byte chunks are swizzled by row % 8.
constexpr int few_waves(int NT, int RT) { return NT + RT <= 4 ? 16 : NT + RT <= 10 ? 8 : 6; }
template <int NT, int RT>
__global__ __launch_bounds__(few_waves(NT, RT) * kWave) void k_linear_q8_few(Linear8Args a) {
  constexpr int W = few_waves(NT, RT), TT = 16 * NT, RR = 16 * RT, LS = RR + 1, kSlot = (TT + RR) * 128;
  static_assert(W * kSlot <= 160 * 1024 && TT * LS * 4 <= W * kSlot, "LDS");
  __shared__ __attribute__((aligned(16))) uint8_t mem[W * kSlot];
  int* sum = (int*)mem;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), m = lane & 15, c = lane >> 4;
  const int row0 = blockIdx.x * RR, tok0 = blockIdx.y * TT, tokens = min(TT, a.T - tok0);
  uint8_t* slot = mem + wave * kSlot;
  const int lrow = lane >> 3, chunk = ((lane & 7) ^ lrow) * 16;
  const int8_t* src[2 * RT + 2 * NT];                          // rows 8 j + lrow: weights, then tokens
#pragma unroll
  for (int j = 0; j < 2 * RT + 2 * NT; ++j)
    src[j] = j < 2 * RT ? a.W + (size_t)min(row0 + 8 * j + lrow, a.n - 1) * a.d
                        : a.x + (size_t)min(tok0 + 8 * (j - 2 * RT) + lrow, a.T - 1) * a.ldx;
  i32x4 acc[NT][RT];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < RT; ++i) acc[t][i] = i32x4{0, 0, 0, 0};
  const int pairs = (a.d + 127) / 128;
  for (int p = wave; p < pairs; p += W) {
    const int at = min(p * 128 + chunk, a.d - 16);
    wait_lds();                                                // the reads of the last round
#pragma unroll
    for (int j = 0; j < 2 * RT + 2 * NT; ++j)                  // rows of tokens that are not there: left as they are
      if (j < 2 * RT || 8 * (j - 2 * RT) < tokens)
        __builtin_amdgcn_global_load_lds((const void*)(src[j] + at), (__attribute__((address_space(3))) void*)(slot + j * 1024),
                                         16, 0, 0);
    wait_vm<0>();
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      Raw<16> wf[RT], xf[NT];
      const int pos = ((4 * u + c) ^ (m & 7)) * 16, col = p * 128 + 64 * u;
#pragma unroll
      for (int i = 0; i < RT; ++i) wf[i] = load_raw<16>(slot + (16 * i + m) * 128 + pos);
#pragma unroll
      for (int t = 0; t < NT; ++t) xf[t] = load_raw<16>(slot + (RR + 16 * t + m) * 128 + pos);
      if (col + 64 > a.d) {                                    // products with 0 past the end
        const uint32_t mask = col + 16 * c < a.d ? ~0u : 0u;
#pragma unroll
        for (int t = 0; t < NT; ++t) keep(xf[t], mask);
      }
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < RT; ++i) acc[t][i] = mma8(xf[t], wf[i], acc[t][i]);
    }
  }
  // integer sums: their order changes nothing
  __syncthreads();
  for (int e = threadIdx.x; e < TT * LS; e += W * kWave) sum[e] = 0;
  __syncthreads();
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) atomicAdd(&sum[(16 * t + 4 * c + e) * LS + 16 * i + m], acc[t][i][e]);
  __syncthreads();
  for (int e = threadIdx.x; e < tokens * RR; e += W * kWave) {
    const int tok = e / RR, row = e % RR;
    if (row0 + row < a.n) lin8_store(a, tok0 + tok, row0 + row, sum[tok * LS + row]);
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
template <int YT, int BN, int BT, int WN, int WT, int NS>
__global__ __launch_bounds__(WN * WT * kWave) void k_linear_q8_tiles(Linear8Args a, int tn, int tt) {
  constexpr int NTH = WN * WT * kWave, MI = BN / WN / 32, NI = BT / WT / 32, LA = BN * 8 / NTH, LB = BT * 8 / NTH;
  static_assert(MI % 2 == 0 && BN % (NTH / 8) == 0 && BT % (NTH / 8) == 0 && NTH % 128 == 0, "tile");
  // two objects: copies into one are then no reason to wait before reads of the other
  constexpr int kStage = (BN + BT) * kBK;
  __shared__ __attribute__((aligned(16))) uint8_t buf0[kStage];
  __shared__ __attribute__((aligned(16))) uint8_t buf1[kStage];
  __shared__ __attribute__((aligned(16))) uint8_t buf2[NS > 2 ? kStage : 16];
  __shared__ __attribute__((aligned(16))) uint8_t buf3[NS > 2 ? kStage : 16];
  const auto stage = [&](auto i) -> uint8_t* {
    constexpr int I = decltype(i)::value % NS;
    if constexpr (I == 0) return buf0;
    else if constexpr (I == 1) return buf1;
    else if constexpr (I == 2) return buf2;
    else return buf3;
  };
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
  const auto body = [&](auto i, int s) {
    uint8_t* cur = stage(i);
    load(cur, 1, f1);
    mma(f0);
    mix();
    load(cur, 2, f0);
    mma(f1);
    mix();
    load(cur, 3, f1);
    mma(f0);
    mix();
    // the next stage has landed (those behind it are on their way), and `cur` has been read
    if (s + NS - 1 < S) wait_vm<(NS - 2) * (LA + LB)>();
    else wait_vm<0>();
    wait_lds();
    __builtin_amdgcn_s_barrier();
    memory_order();
    if (s + NS < S) fetch(s + NS, cur);
    load(stage(std::integral_constant<int, decltype(i)::value + 1>{}), 0, f0);
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
  constexpr std::integral_constant<int, 0> c0{};
  constexpr std::integral_constant<int, 1> c1{};
  constexpr std::integral_constant<int, 2> c2{};
  constexpr std::integral_constant<int, 3> c3{};
  fetch(0, buf0);
  if (S > 1) fetch(1, buf1);
  if (NS > 2 && S > 2) fetch(2, buf2);
  if (NS > 2 && S > 3) fetch(3, buf3);
  if (S >= NS) wait_vm<(NS - 1) * (LA + LB)>();
  else wait_vm<0>();
  __builtin_amdgcn_s_barrier();
  memory_order();
  load(buf0, 0, f0);
  int s = 0;
  for (; s + NS < S; s += NS) {
    body(c0, s);
    body(c1, s + 1);
    if constexpr (NS > 2) {
      body(c2, s + 2);
      body(c3, s + 3);
    }
  }
  // 1 .. NS stages are left
  const int bodies = S - 1 - s;
  if (bodies > 0) body(c0, s);
  if constexpr (NS > 2) {
    if (bodies > 1) body(c1, s + 1);
    if (bodies > 2) body(c2, s + 2);
  }
  last(bodies == 0 ? buf0 : NS == 2 || bodies == 1 ? buf1 : bodies == 2 ? buf2 : buf3, S - 1);

  // out by way of LDS, 32 tokens x 64 rows of a wave at a time: straight from the registers a
  // store instruction would write 64 pieces of 8 bytes (240 us of 780 at 8192 x 16384 x 4096)
  constexpr int LS = 68;
  static_assert(NTH / 128 * 32 * LS * 4 <= (BN + BT) * kBK, "staging");
  __syncthreads();
  float* st = (float*)((wave & 1) ? buf1 : buf0) + (wave >> 1) * (32 * LS);
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
        for (int e = 0; e < 8; ++e) o[e] = lin8_value(e < 4 ? v0[e & 3] : v1[e & 3], sx, sw[e], bias[e]);
        const size_t at = (size_t)t * a.ldy + nb;
        if (nb + 8 <= a.n) {
          if (a.accumulate) {
            float was[8];
            widen<YT>(load8_at<YT>(a.y, at), was);
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] += was[e];
          }
          store8_at<YT>(a.y, at, o);                           // rows may lie at any element
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (nb + e < a.n) store_elem<YT>(a.y, at + e, a.accumulate ? o[e] + load_elem<YT>(a.y, at + e) : o[e]);
        }
      }
    }
  }
}

template <int YT, int BN, int BT, int WN, int WT, int NS>
void tiles_run(hipStream_t st, const Linear8Args& a) {
  const int tn = (a.n + BN - 1) / BN, tt = (a.T + BT - 1) / BT;
  k_linear_q8_tiles<YT, BN, BT, WN, WT, NS><<<dim3((tn * tt + 7) / 8 * 8), dim3(WN * WT * kWave), 0, st>>>(a, tn, tt);
}
template <int BN, int BT, int WN, int WT, int NS>
void tiles_run(hipStream_t st, const Linear8Args& a) {
  if (a.ydt == DT_F32) tiles_run<DT_F32, BN, BT, WN, WT, NS>(st, a);
  else if (a.ydt == DT_F16) tiles_run<DT_F16, BN, BT, WN, WT, NS>(st, a);
  else tiles_run<DT_BF16, BN, BT, WN, WT, NS>(st, a);
}

template <int NT, int RT>
void few_run(hipStream_t st, const Linear8Args& a) {
  const dim3 g((a.n + 16 * RT - 1) / (16 * RT), (a.T + 16 * NT - 1) / (16 * NT));
  k_linear_q8_few<NT, RT><<<g, dim3(few_waves(NT, RT) * kWave), 0, st>>>(a);
}
template <int NT>
void few_run(hipStream_t st, const Linear8Args& a, int rt) {
  switch (rt) {
    case 1: return few_run<NT, 1>(st, a);
    case 2: return few_run<NT, 2>(st, a);
    case 3: return few_run<NT, 3>(st, a);
    case 4: return few_run<NT, 4>(st, a);
    case 6: return few_run<NT, 6>(st, a);
    default: return few_run<NT, 8>(st, a);
  }
}
// The cheapest of the kernels by what each took per round over 256 compute units, in us (d 512 and
// 4096, n 1024..28672, 32..8192 tokens): a part for its start and end, one per column.
//   few           (lines of a workgroup + 16) x (0.035 + 2.3e-5 d): 64 x 11008 x 4096 15.4 (256 x 64
//                 tiles 58), 512 x 4096 x 4096 22.3
//   128 x 64      4.5 + 4.2e-3 d    512 x 4096 x 4096 20.1
//   128 x 128     4.8 + 5.4e-3 d with four stages, 1024 x 4096 x 4096 27.9 (few 39.6, 256 x 256 59)
//                 5.5 + 8.2e-3 d with two, two workgroups per unit: 512 x 11008 x 4096 44 (256 x 256 64)
//   256 x 256     13 + 11.5e-3 d    4096 x 4096 x 4096 60 (128 x 128 78)
// Not in the costs: pieces of 128 columns that do not divide by a workgroup's waves (1056 columns are nine for
// the eight waves of `few`: the ninth is a round of its own).
enum { kFew, kTile64, kTile128x4, kTile128x2, kTile256 };
struct Choice8 {
  int kind, nt, rt;
  double us;
};
Choice8 choose8(const Linear8Args& a) {
  const auto rounds = [&](int bn, int bt, int units) {
    const long long tiles = (long long)((a.n + bn - 1) / bn) * ((a.T + bt - 1) / bt);
    return (double)((tiles + units - 1) / units);
  };
  Choice8 best{kFew, 1, 1, 1e30};
  const auto offer = [&](int kind, int nt, int rt, double us) {
    if (us < best.us) best = Choice8{kind, nt, rt, us};
  };
  for (int nt : {1, 2, 4})
    for (int rt : {1, 2, 3, 4, 6, 8})
      offer(kFew, nt, rt, rounds(16 * rt, 16 * nt, 256) * (std::min((a.T + 7) / 8 * 8, 16 * nt) + 16 * rt + 16) *
                              (0.035 + 2.3e-5 * a.d));
  if (a.T <= 16) return best;                                  // bound by the weights' bytes
  offer(kTile64, 0, 0, rounds(128, 64, 256) * (4.5 + 4.2e-3 * a.d));
  offer(kTile128x4, 0, 0, rounds(128, 128, 256) * (4.8 + 5.4e-3 * a.d));
  offer(kTile128x2, 0, 0, rounds(128, 128, 512) * (5.5 + 8.2e-3 * a.d));
  offer(kTile256, 0, 0, rounds(256, 256, 256) * (13 + 11.5e-3 * a.d));
  return best;
}

}  // namespace

hipError_t launch_linear_q8(hipStream_t st, int ydt, int T, int n, int d, const int8_t* x, size_t ldx, const float* sx,
                            const int8_t* W, const float* sw, const float* bias, int accumulate, void* y, size_t ldy) {
  const Linear8Args a{x, ldx, sx, W, sw, bias, y, ldy, T, n, d, accumulate, ydt};
  if (T <= 4 && n <= 8192) {
    // here and with lines through LDS, us: 1 x 4096 x 4096 5.5 and 5.9, 1 x 8192 x 4096 7.8 and 9.1, 4 x 8192 x 4096 8.4
    // and 9.2.  With more rows it goes by the columns: 1 x 11008 x 4096 10.7 and 11.1, 4 x 11008 x 4096 11.6 and 11.0,
    // 9000 x 1024 6.9 and 4.8, 28672 x 7168 41.4 and 40.0, 32768 x 8192 46.9 and 56.8
    k_linear_q8_one<16, 4><<<dim3((n + 15) / 16), dim3(16 * kWave), 0, st>>>(a);
    return hipGetLastError();
  }
  const Choice8 c = choose8(a);
  if (c.kind == kTile64) tiles_run<128, 64, 2, 2, 4>(st, a);
  else if (c.kind == kTile128x4) tiles_run<128, 128, 2, 2, 4>(st, a);
  else if (c.kind == kTile128x2) tiles_run<128, 128, 2, 2, 2>(st, a);
  else if (c.kind == kTile256) tiles_run<256, 256, 2, 4, 2>(st, a);
  else if (c.nt == 1) few_run<1>(st, a, c.rt);
  else if (c.nt == 2) few_run<2>(st, a, c.rt);
  else few_run<4>(st, a, c.rt);
  return hipGetLastError();
}

}  // namespace sfx
