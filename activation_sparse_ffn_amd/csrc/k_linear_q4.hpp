// y[b][i] (+)= sum_c W[i][c] x[b][c] + bias[i] for int4 weights with one fp16 scale per
// group of 32, 64 or 128 columns, 1..64 tokens (the projections around the FFN step, in
// the storage of its int4 rows).
//
// Tokens are the rows and 16 weight rows the columns of 16x16x32 products, so a lane
// meets one weight row only and needs one scale per group.  The waves of a workgroup share
// their rows and deal the columns among themselves; their sums are added in wave order
// through LDS, so y is bitwise reproducible.  Three kernels, by how much of x there is:
//   few tokens   up to 8, all of x in LDS; bound by reading the codes.
//   wide, rows   x in blocks, 16 or 32 rows per workgroup: each workgroup reads all of x, from
//                L2, and writes it to LDS; from about 16 tokens on that and the decoding
//                weigh more than the codes.
// Measured (one MI355X): 1 x 28672 x 7168, scales per 128: 25.6 us = 4.1 TB/s of 106 MB; 1 x 4096
// x 4096: 5.3 us; 37 x 8192 x 8192, scales per 64: 24.1 us against 7.1 for its 38.7 MB (VALU 28%
// of the time busy, MFMA 16%).
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

// Token that row m stands for where NI < 4 accumulator rows per lane are used: up to 8 tokens
// are spread over the quarters (row 4 c + i is token NI c + i), so only NI of a lane's four
// sums are scaled.
template <int NI>
__device__ __forceinline__ int lin_token(int m) {
  return NI * (m >> 2) + (m & (NI - 1));
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

// The operand that takes the codes' offset back, where there is one.
template <class T>
__device__ __forceinline__ Raw<16> lin_offset() {
  if constexpr (Q4<T>::offset) return Q4<T>::minus24();
  else return zero16();
}

// Sums of a chunk: `groups` of its 32 columns exist (4 but in the last chunk); k: the codes
// as loaded; xrow: this lane's slice of the chunk's ordered x per token tile, in LDS.
template <class T, int NT, int GSH>
__device__ __forceinline__ void lin_chunk(const LinChunk<GSH>& w, const uint8_t* const (&xrow)[NT], int groups,
                                          const Q4<T>& dec, const Raw<16>& m24, float (&acc)[NT][4]) {
  uint32_t k[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) k[j] = w.q.w[j] ^ 0x88888888u;
  quarter_transpose(k);
  // groups that share a scale (1 << GSH of them) are summed in the matrix cores before it
  constexpr int kPer = 1 << GSH;
#pragma unroll
  for (int j = 0; j < 4; j += kPer) {
    if (j < groups) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        Raw<16> xp[kPer];
        f32x4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
          xp[u] = load_raw<16>(xrow[t] + (j + u) * 64);
          if constexpr (Q4<T>::offset) p = Mma<T>::run(xp[u], m24, p);
        }
#pragma unroll
        for (int u = 0; u < kPer; ++u) p = Mma<T>::run(xp[u], dec.word(k[j + u]), p);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[t][i] = fmaf(lin_scale<GSH>(w, j), p[i], acc[t][i]);
      }
    }
  }
}

// The waves' sums in wave order, bias, y.  RG groups of W waves, 16 rows from row0 on each.
template <class T, int NT, int NI, int W, int RG>
__device__ __forceinline__ void lin_finish(const LinearArgs& a, float* red, int row0, int wave, int rg, int m, int c,
                                           const float (&acc)[NT][NI]) {
  constexpr int TT = 4 * NI * NT;
  red += rg * (W * 16 * (TT + 1));
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < NI; ++i) red[(wave * 16 + m) * (TT + 1) + (4 * t + c) * NI + i] = acc[t][i];
  __syncthreads();
  for (int e = threadIdx.x - rg * W * kWave; e < 16 * TT; e += W * kWave) {
    const int row = e % 16, tok = e / 16;
    if (row0 + row < a.n && tok < a.B) {
      float v = 0.f;
#pragma unroll
      for (int k = 0; k < W; ++k) v += red[(k * 16 + row) * (TT + 1) + tok];
      v *= Q4<T>::unit;
      if (a.bias) v += a.bias[row0 + row];
      float* y = a.y + (size_t)tok * a.ldy + row0 + row;
      *y = a.accumulate ? *y + v : v;
    }
  }
}

constexpr int kLinWaves = 8;

// ---- few tokens.  A unit is 256 columns of 16 weight rows: 128 bytes of codes per row, so rows
// are read in whole lines (with 64 bytes per row and load, the loads alone of 28672 x 7168
// codes took 25 us instead of 21).  It is copied into LDS by the wave that uses it: row r's
// eight 16-byte pieces (a group each) lie rotated by r / 2, so the 64 lanes of a read hit 64
// banks.
constexpr int kLinUnit = 16 * 128;       // bytes
// Units of a wave in LDS or on the way.  Two, not more: 32 KB leave room for three or four
// workgroups per compute unit (four units: 8192 x 8192 at one token 16.7 us against 12.2, 16384 x
// 4096 at four 20.5 against 13.9).  A longer queue could not help as compiled: the counted wait
// is what a unit needs, but the compiler adds a wait for all copies into LDS before the unit's
// first LDS reads, so a wave's copies overlap with other waves' work only.
constexpr int kLinSlots = 2;

// A row's scales of one unit, as they lie: 8 >> GSH of them.
template <int GSH>
struct LinScales {
  uint32_t w[GSH == 0 ? 4 : GSH == 1 ? 2 : 1];
};
template <int GSH>
__device__ __forceinline__ LinScales<GSH> lin_scales(const uint16_t* srow, int unit, int ng) {
  constexpr int N = 8 >> GSH;
  LinScales<GSH> s;
  const int s0 = unit * N, last = ((ng - 1) >> GSH);
  if (s0 + N - 1 <= last) {
    struct __attribute__((packed, aligned(2))) Words {
      uint32_t w[N / 2];
    };
    const Words v = *reinterpret_cast<const Words*>(srow + s0);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) s.w[i] = v.w[i];
  } else {                               // the row ends in this unit
#pragma unroll
    for (int i = 0; i < N / 2; ++i)
      s.w[i] = srow[min(s0 + 2 * i, last)] | (uint32_t)srow[min(s0 + 2 * i + 1, last)] << 16;
  }
  return s;
}

// All of x lies in LDS, ordered, token rows 2 d + 16 bytes apart (the 16 put eight tokens on
// different banks).  16 weight rows per workgroup; unit u is wave u % 8's.
template <class T, int NI, int GSH>
__global__ __launch_bounds__(kLinWaves * kWave) void k_linear_q4(LinearArgs a) {
  constexpr int kThreads = kLinWaves * kWave, kPer = 1 << GSH;
  __shared__ __attribute__((aligned(16))) uint8_t ring[kLinWaves][kLinSlots][kLinUnit];
  extern __shared__ __attribute__((aligned(16))) uint8_t sh[];
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = lane & 15, c = lane >> 4;
  const int row0 = blockIdx.x * 16;
  const int ng = a.d >> 5, nunit = (ng + 7) >> 3;
  // x first: the wait for it then leaves the weights on their way
  const int xstride = a.d * 2 + 16, pieces = a.d >> 3;
  constexpr int NB = 4 * NI;                                   // tokens whose loads go out together
  Raw<16> xv[NB];
  const int p0 = min((int)threadIdx.x, pieces - 1);
#pragma unroll
  for (int b = 0; b < NB; ++b) xv[b] = load_raw<16>(a.x + (size_t)min(b, a.B - 1) * a.ldx + (size_t)p0 * 16);
  // copy: lane l brings the piece of row 8 i + l / 8 that its slot of LDS holds
  const uint8_t* from[2];
  int piece[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = 8 * i + (lane >> 3);
    from[i] = a.W + (size_t)min(row0 + r, a.n - 1) * (a.d >> 1);
    piece[i] = ((lane & 7) - (r >> 1)) & 7;
  }
  const uint16_t* srow = a.s + (size_t)min(row0 + m, a.n - 1) * (ng >> GSH);
  const int todo = nunit > wave ? (nunit - wave + kLinWaves - 1) / kLinWaves : 0;
  LinScales<GSH> sc[kLinSlots];
  auto fetch = [&](int i, int slot, LinScales<GSH>& s) {
    const int unit = wave + i * kLinWaves;
    memory_order();                                            // units are waited for in this order
#pragma unroll
    for (int k = 0; k < 2; ++k)
      __builtin_amdgcn_global_load_lds((const void*)(from[k] + (size_t)min(8 * unit + piece[k], ng - 1) * 16),
                                       (__attribute__((address_space(3))) void*)(ring[wave][slot] + k * 1024), 16, 0, 0);
    s = lin_scales<GSH>(srow, unit, ng);
    memory_order();
  };
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < kLinSlots; ++i)
    if (i < todo) fetch(i, i, sc[i]);
  __builtin_amdgcn_sched_barrier(0);
  for (int i = threadIdx.x; i < pieces; i += kThreads) {
    if (i >= kThreads) {
#pragma unroll
      for (int b = 0; b < NB; ++b) xv[b] = load_raw<16>(a.x + (size_t)min(b, a.B - 1) * a.ldx + (size_t)i * 16);
    }
#pragma unroll
    for (int b = 0; b < NB; ++b)
      if (b < a.B) *reinterpret_cast<Raw<16>*>(sh + b * xstride + i * 16) = lin_order(xv[b]);
  }
  __syncthreads();
  const uint8_t* xlane = sh + min(lin_token<NI>(m), a.B - 1) * xstride + c * 16;

  float acc[1][NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) acc[0][i] = 0.f;
  const Q4<T> dec;
  const Raw<16> m24 = lin_offset<T>();
  for (int i0 = 0; i0 < todo; i0 += kLinSlots) {
#pragma unroll
    for (int s = 0; s < kLinSlots; ++s) {
      const int i = i0 + s;
      if (i < todo) {
        // a unit is two copies and at least one load; the younger ones may still be on the way
        const int younger = min(todo - 1 - i, kLinSlots - 1);
        static_assert(kLinSlots == 2, "the waits count one younger unit");
        if (younger > 0) wait_vm<3>();
        else wait_vm<0>();
        const int unit = wave + i * kLinWaves, groups = ng - 8 * unit;
        const uint8_t* w = ring[wave][s] + m * 128 + c * 4;
        const uint8_t* xr = xlane + unit * 512;
#pragma unroll
        for (int j = 0; j < 8; j += kPer) {
          if (j < groups) {
            f32x4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int u = 0; u < kPer; ++u) {
              const Raw<16> xp = load_raw<16>(xr + (j + u) * 64);
              const uint32_t k = *reinterpret_cast<const uint32_t*>(w + ((j + u + (m >> 1)) & 7) * 16) ^ 0x88888888u;
              if constexpr (Q4<T>::offset) p = Mma<T>::run(xp, m24, p);
              p = Mma<T>::run(xp, dec.word(k), p);
            }
            const float f = half_at(sc[s].w[(j >> GSH) >> 1], (j >> GSH) & 1);
#pragma unroll
            for (int t = 0; t < NI; ++t) acc[0][t] = fmaf(f, p[t], acc[0][t]);
          }
        }
        if (i + kLinSlots < todo) {
          wait_lds();
          fetch(i + kLinSlots, s, sc[s]);
        }
      }
    }
  }
  __syncthreads();
  lin_finish<T, 1, NI, kLinWaves, 1>(a, (float*)&ring[0][0][0], row0, wave, 0, m, c, acc);
}

// More tokens, or long rows: x passes through LDS in blocks of 1024 columns, a chunk of 128
// for each wave; the next block's x and the weights of four blocks are asked for in registers
// meanwhile (writing x to LDS waits for all that was asked for before: the compiler keeps no count
// across the branches of the weights' loads).  16 weight rows per workgroup.  Two row tiles and more need over 128 registers (with
// that limit they spilled in the loop: 32 x 4096 x 8192 bf16, scales per 64, 23.0 us instead of
// 15.7); few rows leave a compute unit one workgroup anyway.
template <class T, int NT, int GSH>
__global__ __launch_bounds__(kLinWaves * kWave, NT == 1 ? 4 : 2) void k_linear_q4_wide(LinearArgs a) {
  constexpr int kThreads = kLinWaves * kWave, kCols = 128 * kLinWaves, kRow = kCols * 2 + 16;
  constexpr int kX = 16 * NT * kRow, kRed = kLinWaves * 16 * (16 * NT + 1) * 4;
  constexpr int kPass = 16 * NT * (kCols / 8) / kThreads;       // 16-byte pieces of x per thread and block
  constexpr int kAhead = 4;                                     // blocks of weights on the way (registers)
  __shared__ __attribute__((aligned(16))) uint8_t sh[kX > kRed ? kX : kRed];
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = lane & 15, c = lane >> 4;
  const int row0 = blockIdx.x * 16;
  const int ng = a.d >> 5, nblock = (ng + 4 * kLinWaves - 1) / (4 * kLinWaves);
  const int row = min(row0 + m, a.n - 1);
  const uint8_t* wrow = a.W + (size_t)row * (a.d >> 1);
  const uint16_t* srow = a.s + (size_t)row * (ng >> GSH);
  // thread's pieces of x: piece tid % 128 of tokens tid / 128 + 4 i
  const int piece = threadIdx.x & (kCols / 8 - 1), tok0 = threadIdx.x / (kCols / 8);
  constexpr int kStep = kThreads / (kCols / 8);
  Raw<16> xv[kPass];
  auto load_x = [&](int blk) {
    const int col = min(blk * kCols + piece * 8, a.d - 8);
#pragma unroll
    for (int i = 0; i < kPass; ++i)
      xv[i] = load_raw<16>(a.x + (size_t)min(tok0 + kStep * i, a.B - 1) * a.ldx + (size_t)col * 2);
  };
  LinChunk<GSH> w[kAhead];
  auto load_w = [&](int blk, LinChunk<GSH>& to) {
    const int ck = blk * kLinWaves + wave;
    if (4 * ck < ng) lin_load<GSH>(wrow, srow, ck, c, ng, to);
  };
  load_x(0);
#pragma unroll
  for (int u = 0; u < kAhead; ++u) load_w(u, w[u]);
  const uint8_t* xrow[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) xrow[t] = sh + min(16 * t + m, a.B - 1) * kRow + wave * 256 + c * 16;
  float acc[NT][4];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[t][i] = 0.f;
  const Q4<T> dec;
  const Raw<16> m24 = lin_offset<T>();
  for (int blk0 = 0; blk0 < nblock; blk0 += kAhead) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int blk = blk0 + u;
      if (blk < nblock) {
#pragma unroll
        for (int i = 0; i < kPass; ++i)
          *reinterpret_cast<Raw<16>*>(sh + (tok0 + kStep * i) * kRow + piece * 16) = lin_order(xv[i]);
        // x before the weights: loads are waited for in their order, and x is needed first
        if (blk + 1 < nblock) load_x(blk + 1);
        const LinChunk<GSH> now = w[u];
        load_w(blk + kAhead, w[u]);
        __syncthreads();
        const int groups = ng - 4 * (blk * kLinWaves + wave);
        if (groups >= 4) lin_chunk<T, NT, GSH>(now, xrow, 4, dec, m24, acc);
        else lin_chunk<T, NT, GSH>(now, xrow, groups, dec, m24, acc);
        __syncthreads();
      }
    }
  }
  lin_finish<T, NT, 4, kLinWaves, 1>(a, (float*)sh, row0, wave, 0, m, c, acc);
}

// Many weight rows: two groups of four waves, 16 rows each, over blocks of 512 columns.  Two
// blocks of x lie in LDS: while one is worked on, the next is written from registers and the
// one behind it is asked for, with one barrier a block; loads are waited for as above.
template <class T, int NT, int GSH>
__global__ __launch_bounds__(kLinWaves * kWave, 2) void k_linear_q4_rows(LinearArgs a) {
  constexpr int kThreads = kLinWaves * kWave, kChunks = 4, kCols = 128 * kChunks, kRow = kCols * 2 + 16;
  constexpr int kX = 16 * NT * kRow, kRed = kLinWaves * 16 * (16 * NT + 1) * 4;
  constexpr int kPass = 16 * NT * (kCols / 8) / kThreads;       // 16-byte pieces of x per thread and block
  constexpr int kAhead = 4;                                     // blocks of weights on the way (registers)
  __shared__ __attribute__((aligned(16))) uint8_t sh[2 * kX > kRed ? 2 * kX : kRed];
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kc = wave % kChunks, rg = wave / kChunks;
  const int m = lane & 15, c = lane >> 4;
  const int row0 = (blockIdx.x * 2 + rg) * 16;
  const int ng = a.d >> 5, nblock = (ng + 4 * kChunks - 1) / (4 * kChunks);
  const int row = min(row0 + m, a.n - 1);
  const uint8_t* wrow = a.W + (size_t)row * (a.d >> 1);
  const uint16_t* srow = a.s + (size_t)row * (ng >> GSH);
  // thread's pieces of x: piece tid % 64 of tokens tid / 64 + 8 i
  const int piece = threadIdx.x & (kCols / 8 - 1), tok0 = threadIdx.x / (kCols / 8);
  constexpr int kStep = kThreads / (kCols / 8);
  Raw<16> xv[kPass];
  auto load_x = [&](int blk) {
    const int col = min(blk * kCols + piece * 8, a.d - 8);
#pragma unroll
    for (int i = 0; i < kPass; ++i)
      xv[i] = load_raw<16>(a.x + (size_t)min(tok0 + kStep * i, a.B - 1) * a.ldx + (size_t)col * 2);
  };
  auto store_x = [&](int buf) {
#pragma unroll
    for (int i = 0; i < kPass; ++i)
      *reinterpret_cast<Raw<16>*>(sh + buf * kX + (tok0 + kStep * i) * kRow + piece * 16) = lin_order(xv[i]);
  };
  LinChunk<GSH> w[kAhead];
  auto load_w = [&](int blk, LinChunk<GSH>& to) {
    const int ck = blk * kChunks + kc;
    if (4 * ck < ng) lin_load<GSH>(wrow, srow, ck, c, ng, to);
  };
  load_x(0);
#pragma unroll
  for (int u = 0; u < kAhead; ++u) load_w(u, w[u]);
  int xoff[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) xoff[t] = min(16 * t + m, a.B - 1) * kRow + kc * 256 + c * 16;
  float acc[NT][4];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[t][i] = 0.f;
  const Q4<T> dec;
  const Raw<16> m24 = lin_offset<T>();
  store_x(0);
  if (nblock > 1) load_x(1);
  __syncthreads();
  for (int blk0 = 0; blk0 < nblock; blk0 += kAhead) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int blk = blk0 + u;
      if (blk < nblock) {
        if (blk + 1 < nblock) store_x((u + 1) & 1);
        // x before the weights: loads are waited for in their order, and x is needed first
        if (blk + 2 < nblock) load_x(blk + 2);
        const LinChunk<GSH> now = w[u];
        load_w(blk + kAhead, w[u]);
        const uint8_t* xrow[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) xrow[t] = sh + (u & 1) * kX + xoff[t];
        const int groups = ng - 4 * (blk * kChunks + kc);
        if (groups >= 4) lin_chunk<T, NT, GSH>(now, xrow, 4, dec, m24, acc);
        else lin_chunk<T, NT, GSH>(now, xrow, groups, dec, m24, acc);
        __syncthreads();
      }
    }
  }
  lin_finish<T, NT, 4, kChunks, 2>(a, (float*)sh, row0, kc, rg, m, c, acc);
}

// x is kept whole in LDS, beside the 32 KB ring, up to these sizes: with kLinXTwo two workgroups
// fit a compute unit's 160 KB, with kLinXOne one does.
constexpr int kLinXTwo = 48 << 10, kLinXOne = 128 << 10;

template <class T, int NI>
hipError_t lin_run(hipStream_t s, const LinearArgs& a, int gsh) {
  const dim3 grid((a.n + 15) / 16), blk(kLinWaves * kWave);
  const size_t lds = (size_t)a.B * (a.d * 2 + 16);
  if (gsh == 0) k_linear_q4<T, NI, 0><<<grid, blk, lds, s>>>(a);
  else if (gsh == 1) k_linear_q4<T, NI, 1><<<grid, blk, lds, s>>>(a);
  else k_linear_q4<T, NI, 2><<<grid, blk, lds, s>>>(a);
  return hipGetLastError();
}
template <class T, int NT>
hipError_t lin_run_wide(hipStream_t s, const LinearArgs& a, int gsh) {
  const dim3 grid((a.n + 15) / 16), blk(kLinWaves * kWave);
  if (gsh == 0) k_linear_q4_wide<T, NT, 0><<<grid, blk, 0, s>>>(a);
  else if (gsh == 1) k_linear_q4_wide<T, NT, 1><<<grid, blk, 0, s>>>(a);
  else k_linear_q4_wide<T, NT, 2><<<grid, blk, 0, s>>>(a);
  return hipGetLastError();
}
template <class T, int NT>
hipError_t lin_run_rows(hipStream_t s, const LinearArgs& a, int gsh) {
  const dim3 grid((a.n + 31) / 32), blk(kLinWaves * kWave);
  if (gsh == 0) k_linear_q4_rows<T, NT, 0><<<grid, blk, 0, s>>>(a);
  else if (gsh == 1) k_linear_q4_rows<T, NT, 1><<<grid, blk, 0, s>>>(a);
  else k_linear_q4_rows<T, NT, 2><<<grid, blk, 0, s>>>(a);
  return hipGetLastError();
}

template <class T>
hipError_t lin_launch(hipStream_t s, const LinearArgs& a, int gsh) {
  // Up to 8 tokens x is kept whole.  A workgroup that has a compute unit to itself pays where
  // there is no second one for it (up to 4096 rows), and for one or two tokens where there are
  // up to two.  us, x whole against x in blocks (f16, scales per 32):
  //   x 24..48 KB    4 x 4096 x 4096 6.0, 7.2;  2 x 8192 x 8192 13.5, 17.3;  4 x 28672 x 4096 20, 25
  //   x 48..128 KB   4096 rows: 8 x 4096 6.2, 7.2;  2 x 16384 17.0, 19.3;  1 x 28672 26.1, 31.3
  //                  8192 rows: 4 x 7168 17.1, 15.2;  8 x 4096 10.7, 9.5;  1 x 28672 47.8, 50.1
  //                  16384 rows: 4 x 7168 31.2, 21.0;  2 x 16384 56.7, 42.3;  1 x 28672 90, 70
  //   9..16 tokens   16 x 4096 x 1024 4.9, 3.6;  16 x 28672 x 1024 15.2, 8.4;  12 x 4096 x 4096 7.2, 7.4
  const size_t x = (size_t)a.B * (a.d * 2 + 16);
  if (a.B <= 8 && x <= (size_t)(a.n <= (a.B <= 2 ? 8192 : 4096) ? kLinXOne : kLinXTwo))
    return a.B <= 4 ? lin_run<T, 1>(s, a, gsh) : lin_run<T, 2>(s, a, gsh);
  // 16 rows per workgroup leave enough workgroups for few rows; above one per compute unit,
  // workgroups of 32 rows read x half as often (64 tokens: 4096 x 4096 14.4 us with 16 rows and
  // 16.7 with 32; 32: 4096 x 8192 15.7 and 17.8; 48: 6144 x 4096 20.6 and 13.5; 37: 8192 x 8192
  // 38.2 and 24.1; 12: 8192 x 4096 10.4 and 9.5, 8192 x 1024 4.5 and 4.8)
  const bool two = a.n > 16 * 256;
  if (a.B <= 16) return two ? lin_run_rows<T, 1>(s, a, gsh) : lin_run_wide<T, 1>(s, a, gsh);
  if (a.B <= 32) return two ? lin_run_rows<T, 2>(s, a, gsh) : lin_run_wide<T, 2>(s, a, gsh);
  if (a.B <= 48) return two ? lin_run_rows<T, 3>(s, a, gsh) : lin_run_wide<T, 3>(s, a, gsh);
  return two ? lin_run_rows<T, 4>(s, a, gsh) : lin_run_wide<T, 4>(s, a, gsh);
}

}  // namespace
}  // namespace sfx
