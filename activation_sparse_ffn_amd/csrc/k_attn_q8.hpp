// Attention over the paged int8 key/value cache: the last tokens of each sequence (one or many),
// Hq query heads sharing Hkv kv heads.
//
//   s_p = scale q . k_p,  p in [lo, hi);  o = sum_p e^(s_p - m) v_p / sum_p e^(s_p - m)
//
// A row is a (token, query head) pair of one kv head, token by token; sixteen rows share a pass
// over the cache.  A wave takes 32 positions (two blocks) at a time:
//   scores   16x16x32 products, 16 positions (rows) x 16 rows of queries (columns), on the codes
//            as fp16 (exact) and the queries scaled by a power of two per row to just below
//            2^15 (exact but for what is below 2^-39 of a row's largest); the block's fp32 scale
//            multiplies the fp32 sum;
//   weights  P = 2^(s + log2 vs - ref + 9) in fp32, as one fp16 operand: the scale of a block's
//            values rides in the exponent, so the second product takes the codes as they are
//            and its precision is relative to the largest contribution.  The sum of weights
//            takes P / vs in fp32;
//   output   value codes as rows of 16 dims x 32 positions.
// The lane that holds a score holds it in the place where the second product wants the weight.
// The reference is raised only when an exponent passes it by 6, so P stays below 2^15.
#pragma once
#include "sfx_kv8.hpp"
#include "sfx_launch.hpp"
#include "sfx_q4.hpp"

namespace sfx {
namespace {

constexpr int kTile8 = 32;             // positions a wave takes at a time
constexpr float kRefMin8 = -3.0e38f;
constexpr float kNoScale = 0x1p-64f;   // stands for the scale 0 of values that are all 0
constexpr int attn8_waves(int NG) { return NG <= 4 ? 8 : 4; }

struct Attn8Args {
  KvCache kv;
  Rows8 rows;
  const uint8_t* q;
  size_t ldq;               // bytes between tokens
  const int32_t* starts;
  uint8_t* out;             // [T][Hq][D] 16 bit
  float* lse;               // [T][Hq] or null
  float* parts;             // [B][Hkv][row tiles][S] x ([16][D] sums, [16][2] reference and weight sum)
  float k2;                 // scale log2(e)
  int Hq, G, window, RT, S;
};

template <int N>
__device__ __forceinline__ void load_words8(const uint8_t* p, uint32_t* w) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const Raw<16> r = load_raw<16>(p + 16 * i);
#pragma unroll
      for (int j = 0; j < 4; ++j) w[4 * i + j] = r.w[j];
    }
  } else {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const Raw<8> r = load_raw<8>(p + 8 * i);
      w[2 * i] = r.w[0];
      w[2 * i + 1] = r.w[1];
    }
  }
}

// Eight codes as fp16: u sits in the mantissa of 1024, 1152 taken off, both exact.
__device__ __forceinline__ Raw<16> codes8(uint32_t a, uint32_t b) {
  Raw<16> r;
  r.w[0] = pk_add(__builtin_amdgcn_perm(0x64646464u, a, 0x04010400u), 0xE480E480u);
  r.w[1] = pk_add(__builtin_amdgcn_perm(0x64646464u, a, 0x04030402u), 0xE480E480u);
  r.w[2] = pk_add(__builtin_amdgcn_perm(0x64646464u, b, 0x04010400u), 0xE480E480u);
  r.w[3] = pk_add(__builtin_amdgcn_perm(0x64646464u, b, 0x04030402u), 0xE480E480u);
  return r;
}
__device__ __forceinline__ uint32_t pack8_f16(float a, float b) {
  const half2_t h = {(_Float16)a, (_Float16)b};
  return __builtin_bit_cast(uint32_t, h);
}
__device__ __forceinline__ float quarters_max8(float v, int lane) {
  v = fmaxf(v, __uint_as_float(lane_xor_u32<32>(__float_as_uint(v), lane)));
  return fmaxf(v, __uint_as_float(lane_xor_u32<16>(__float_as_uint(v), lane)));
}
__device__ __forceinline__ float quarters_sum8(float v, int lane) {
  v += __uint_as_float(lane_xor_u32<32>(__float_as_uint(v), lane));
  return v + __uint_as_float(lane_xor_u32<16>(__float_as_uint(v), lane));
}

// First of the eight dims that a lane of quarter c feeds to product g of the scores.
template <int NG>
__device__ __forceinline__ int dim8(int g, int c) {
  return g < (NG & ~1) ? 64 * (g >> 1) + 16 * c + 8 * (g & 1) : 32 * g + 8 * c;
}

// A lane's part of 32 positions: K of position n of both blocks, V words of four positions of dims
// n NM .. n NM + NM - 1 (NM = D / 16), the blocks' scales.
template <int NG>
struct Tile8 {
  uint32_t k[2][2 * NG], v[2][2 * NG];
  float2 s[2];
};
template <int NG>
__device__ __forceinline__ void tile8_load(const uint8_t* const (&blk)[2], int n, int c, Tile8<NG>& t) {
  constexpr int D = 32 * NG;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
#pragma unroll
    for (int j = 0; j < NG / 2; ++j) load_words8<4>(blk[u] + n * D + 64 * j + 16 * c, t.k[u] + 4 * j);
    if constexpr (NG % 2) load_words8<2>(blk[u] + n * D + 32 * (NG - 1) + 8 * c, t.k[u] + 2 * (NG - 1));
    load_words8<2 * NG>(blk[u] + 16 * D + (c * D + n * 2 * NG) * 4, t.v[u]);
    t.s[u] = *(const float2*)(blk[u] + 32 * D);
  }
}

template <int NG>
struct State8 {
  float ref, sum;           // reference (all quarters alike), sum of this quarter's weights
  f32x4 acc[2 * NG];        // of product m: dims (4 c + i) 2 NG + m
};

// `on`: bit 4 u + i says that position 4 c + i of block u counts for this lane's row (all ones
// where `full`).
template <int NG>
__device__ __forceinline__ void tile8_run(const Tile8<NG>& t, const Raw<16> (&qf)[NG], float k2, float qs, bool full,
                                          uint32_t on, int lane, State8<NG>& st) {
  float s[8], lv[2], iv[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    f32x4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int g = 0; g < NG; ++g) p = Mma<TF16>::run(codes8(t.k[u][2 * g], t.k[u][2 * g + 1]), qf[g], p);
    const float kk = t.s[u].x * k2 * qs, vs = t.s[u].y != 0.f ? t.s[u].y : kNoScale;
    lv[u] = log2f(vs);
    iv[u] = 1.0f / vs;
#pragma unroll
    for (int i = 0; i < 4; ++i) s[4 * u + i] = fmaf(p[i], kk, lv[u]);
  }
  if (!full) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (!((on >> i) & 1u)) s[i] = -INFINITY;
    // a block none of whose positions counts may hold anything
    if (!(on & 0x0Fu)) iv[0] = 0.f;
    if (!(on & 0xF0u)) iv[1] = 0.f;
  }
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = fmaxf(top, s[i]);
  if (__any(top > st.ref + 6.f)) {
    const float next = fmaxf(quarters_max8(top, lane), st.ref), f = exp2f(st.ref - next);
    st.ref = next;
    st.sum *= f;
#pragma unroll
    for (int m = 0; m < 2 * NG; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) st.acc[m][i] *= f;
  }
  const float off = 9.f - st.ref;
  Raw<16> p;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float e0 = __builtin_amdgcn_exp2f(s[2 * i] + off), e1 = __builtin_amdgcn_exp2f(s[2 * i + 1] + off);
    st.sum = fmaf(e0, iv[i >> 1], st.sum);
    st.sum = fmaf(e1, iv[i >> 1], st.sum);
    p.w[i] = pack8_f16(e0, e1);
  }
#pragma unroll
  for (int m = 0; m < 2 * NG; ++m) st.acc[m] = Mma<TF16>::run(codes8(t.v[0][m], t.v[1][m]), p, st.acc[m]);
}

__device__ __forceinline__ int query8_exponent(float top) {
  return top > 0.f && top < INFINITY ? (int)((__float_as_uint(top) >> 23) & 255u) - 127 - 14 : 0;
}
// The row's eighths of queries for the score products, times 2^-e: returns 2^e.  A row that holds
// an infinity or a NaN is taken as it is.
template <class T, int NG>
__device__ __forceinline__ float query8(const uint8_t* row, bool real, int c, int lane, Raw<16> (&qf)[NG]) {
  float x[NG][8], top = 0.f;
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    const Raw<16> r = real ? load_raw<16>(row + 2 * dim8<NG>(g, c)) : zero16();
    unpack<T, 4>(r.w, x[g]);
#pragma unroll
    for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(x[g][j]));
  }
  const int e = query8_exponent(quarters_max8(top, lane));
#pragma unroll
  for (int g = 0; g < NG; ++g)
#pragma unroll
    for (int j = 0; j < 4; ++j) qf[g].w[j] = pack8_f16(ldexpf(x[g][2 * j], -e), ldexpf(x[g][2 * j + 1], -e));
  return ldexpf(1.f, e);
}

__device__ __forceinline__ float attn8_lse(float ref, float sum) {
  return sum != 0.f ? (ref - 9.f + log2f(sum)) * 0.69314718055994531f : -INFINITY;
}

// Positions [start, end) that some row of a tile covers, as tiles t0 .. t0 + ntile - 1 cut into
// `active` runs of `per`: S even runs, none shorter than a tile per wave.
struct Span8 {
  int start, end, t0, ntile, per, active;
};
__device__ __forceinline__ int row8_lo(const Attn8Args& a, int start, int pos) {
  return a.window ? max(start, pos + 1 - a.window) : start;
}
__device__ __forceinline__ Span8 span8(const Attn8Args& a, const Seq8& sq, int start, int rt, int W) {
  const int i0 = 16 * rt / a.G, i1 = min(sq.n - 1, (16 * rt + 15) / a.G);       // first and last token of the tile
  const int first = sq.len - sq.n;
  Span8 s;
  s.start = max(0, row8_lo(a, start, first + i0));
  s.end = min(first + i1 + 1, a.kv.max_pages << a.kv.page_shift);
  s.t0 = s.start / kTile8;
  s.ntile = s.end > s.start ? (s.end + kTile8 - 1) / kTile8 - s.t0 : 0;
  s.per = max(W, (s.ntile + a.S - 1) / a.S);
  s.active = max(1, (s.ntile + s.per - 1) / s.per);            // an empty tile has one: its zero rows
  return s;
}

// Page ids of a wave's next 32 tiles, one block per lane.
__device__ __forceinline__ int attn8_ids(const KvCache& kv, int b, int it, int W, int te, int lane) {
  const int t = min(it + (lane >> 1) * W, te - 1);
  return kv_page(kv, b, t * kTile8 + (lane & 1) * kBlk8);
}
__device__ __forceinline__ const uint8_t* attn8_block(const KvCache& kv, int h, int id, int pos) {
  return kv.base + kv8_block(kv, max(id, 0), h, (pos & ((1 << kv.page_shift) - 1)) >> 4);
}

template <class T, int NG>
__global__ __launch_bounds__(attn8_waves(NG) * kWave) void k_attn_q8(Attn8Args a) {
  constexpr int W = attn8_waves(NG), D = 32 * NG, kThreads = W * kWave;
  __shared__ float sh_ref[W][16], sh_sum[W][16];
  __shared__ __attribute__((aligned(16))) float sh_acc[W * 16 * (D + 4)];
  const int lane = opaque_lane(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, c = lane >> 4;
  const int split = blockIdx.x % a.S, rt = blockIdx.x / a.S, h = blockIdx.y, b = blockIdx.z;
  const Seq8 sq = rows8_seq(a.rows, b);
  const int rows = min(16, sq.n * a.G - 16 * rt);              // of this tile
  if (rows <= 0) return;
  const int start = a.starts ? max(a.starts[b], 0) : 0;
  const Span8 sp = span8(a, sq, start, rt, W);
  if (split >= sp.active) return;
  const int tb = sp.t0 + split * sp.per, te = min(sp.t0 + sp.ntile, tb + sp.per);

  // this lane's row
  const int r = 16 * rt + min(n, rows - 1), tok = r / a.G, head = h * a.G + r % a.G;
  const int pos = sq.len - sq.n + tok;
  const int lo = row8_lo(a, start, pos), hi = pos + 1;          // columns past the last row repeat it
  const int all_lo = row8_lo(a, start, sq.len - sq.n + (16 * rt + rows - 1) / a.G);   // what every row covers
  const int all_hi = sq.len - sq.n + 16 * rt / a.G + 1;
  Raw<16> qf[NG];
  const float qs = query8<T, NG>(a.q + (size_t)(sq.first + tok) * a.ldq + (size_t)head * D * 2, n < rows, c, lane, qf);
  State8<NG> st;
  st.ref = kRefMin8;
  st.sum = 0.f;
#pragma unroll
  for (int m = 0; m < 2 * NG; ++m) st.acc[m] = f32x4{0.f, 0.f, 0.f, 0.f};
  int it = tb + wave;
  if (it < te) {
    const int todo = (te - it + W - 1) / W;
    int ids = attn8_ids(a.kv, b, it, W, te, lane), next_ids = ids;
    Tile8<NG> cur, nxt;
    {
      const int p0 = it * kTile8;
      const uint8_t* blk[2] = {attn8_block(a.kv, h, __builtin_amdgcn_readlane(ids, 0), p0),
                               attn8_block(a.kv, h, __builtin_amdgcn_readlane(ids, 1), p0 + kBlk8)};
      tile8_load<NG>(blk, n, c, cur);
    }
    for (int i = 0; i < todo; ++i, it += W) {
      const int at = 2 * (i & 31), p0 = it * kTile8;
      const int id0 = __builtin_amdgcn_readlane(ids, at), id1 = __builtin_amdgcn_readlane(ids, at + 1);
      if (i + 1 < todo) {
        const int an = 2 * ((i + 1) & 31), pn = p0 + W * kTile8;
        if (an == 0) next_ids = attn8_ids(a.kv, b, it + W, W, te, lane);
        const uint8_t* blk[2] = {attn8_block(a.kv, h, __builtin_amdgcn_readlane(next_ids, an), pn),
                                 attn8_block(a.kv, h, __builtin_amdgcn_readlane(next_ids, an + 1), pn + kBlk8)};
        tile8_load<NG>(blk, n, c, nxt);
      }
      const bool full = p0 >= all_lo && p0 + kTile8 <= all_hi && id0 >= 0 && id1 >= 0;
      uint32_t on = 0xFFu;
      if (!full) {
        on = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int p = p0 + (e >> 2) * kBlk8 + 4 * c + (e & 3);
          if (p >= lo && p < hi && ((e >> 2) ? id1 : id0) >= 0) on |= 1u << e;
        }
      }
      tile8_run<NG>(cur, qf, a.k2, qs, full, on, lane, st);
      cur = nxt;
      ids = next_ids;
    }
  }

  // join the waves
  st.sum = quarters_sum8(st.sum, lane);
  if (c == 0) {
    sh_ref[wave][n] = st.ref;
    sh_sum[wave][n] = st.sum;
  }
#pragma unroll
  for (int m = 0; m < 2 * NG; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) sh_acc[(wave * 16 + n) * (D + 4) + (4 * c + i) * 2 * NG + m] = st.acc[m][i];
  __syncthreads();
  constexpr size_t run = 16 * (D + 2);
  float* part = a.parts + ((((size_t)b * a.kv.Hkv + h) * a.RT + rt) * a.S + split) * run;
  for (int e = threadIdx.x; e < rows * (D / 2); e += kThreads) {
    const int rr = e / (D / 2), d = 2 * (e % (D / 2));
    float ref = sh_ref[0][rr];
#pragma unroll
    for (int w = 1; w < W; ++w) ref = fmaxf(ref, sh_ref[w][rr]);
    float v0 = 0.f, v1 = 0.f, l = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float f = exp2f(sh_ref[w][rr] - ref);
      const float* p = sh_acc + (w * 16 + rr) * (D + 4) + d;
      v0 = fmaf(f, p[0], v0);
      v1 = fmaf(f, p[1], v1);
      l = fmaf(f, sh_sum[w][rr], l);
    }
    if (sp.active == 1) {
      const int q = 16 * rt + rr;
      const size_t o = (size_t)(sq.first + q / a.G) * a.Hq + h * a.G + q % a.G;
      const float inv = l != 0.f ? 1.0f / l : 0.f;
      ((uint32_t*)a.out)[(o * D + d) >> 1] = (uint32_t)to_16(T{}, v0 * inv) | ((uint32_t)to_16(T{}, v1 * inv) << 16);
      if (a.lse && d == 0) a.lse[o] = attn8_lse(ref, l);
    } else {
      *reinterpret_cast<float2*>(part + rr * D + d) = make_float2(v0, v1);
      if (d == 0) *reinterpret_cast<float2*>(part + 16 * D + 2 * rr) = make_float2(ref, l);
    }
  }
}

// Joins the runs of a row, one workgroup per row.  Four dims to a thread; the runs are dealt out
// over groups of D / 4 threads and the groups' sums added in order.
template <class T, int NG>
__global__ __launch_bounds__(256) void k_attn8_join(Attn8Args a) {
  constexpr int W = attn8_waves(NG), D = 32 * NG, kItems = D / 4, kGroups = 256 / kItems;
  __shared__ __attribute__((aligned(16))) float sh_v[kGroups][D];
  __shared__ float sh_l[kGroups], sh_r[kGroups];
  const int b = blockIdx.y, per_head = a.rows.most * a.G, h = blockIdx.x / per_head, q = blockIdx.x % per_head;
  const Seq8 sq = rows8_seq(a.rows, b);
  if (q >= sq.n * a.G) return;
  const int rt = q / 16, rr = q % 16;
  const Span8 sp = span8(a, sq, a.starts ? max(a.starts[b], 0) : 0, rt, W);
  if (sp.active == 1) return;                                   // the attention kernel wrote the row
  constexpr size_t run = 16 * (D + 2);
  const float* part = a.parts + (((size_t)b * a.kv.Hkv + h) * a.RT + rt) * a.S * run;
  const float* rs = part + 16 * D + 2 * rr;
  const int grp = threadIdx.x / kItems, d = 4 * (threadIdx.x % kItems);
  float r = kRefMin8;
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  float l = 0.f;
  if (grp < kGroups) {
#pragma unroll 4
    for (int k = grp; k < sp.active; k += kGroups) {
      const f32x4 pk = *reinterpret_cast<const f32x4*>(part + k * run + rr * D + d);
      const float2 rl = *reinterpret_cast<const float2*>(rs + k * run);
      const float next = fmaxf(r, rl.x), f0 = exp2f(r - next), f1 = exp2f(rl.x - next);
      r = next;
      l = fmaf(f1, rl.y, l * f0);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = fmaf(f1, pk[i], v[i] * f0);
    }
    *reinterpret_cast<f32x4*>(&sh_v[grp][d]) = v;
    if (d == 0) {
      sh_l[grp] = l;
      sh_r[grp] = r;
    }
  }
  __syncthreads();
  if (threadIdx.x < kItems) {
#pragma unroll
    for (int k = 0; k < kGroups; ++k) r = fmaxf(r, sh_r[k]);
    l = 0.f;
    v = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
      const float f = exp2f(sh_r[k] - r);
      const f32x4 o = *reinterpret_cast<const f32x4*>(&sh_v[k][d]);
      l = fmaf(f, sh_l[k], l);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = fmaf(f, o[i], v[i]);
    }
    const size_t o = (size_t)(sq.first + q / a.G) * a.Hq + h * a.G + q % a.G;
    const float inv = l != 0.f ? 1.0f / l : 0.f;
    uint32_t* dst = (uint32_t*)a.out + ((o * D + d) >> 1);
    dst[0] = (uint32_t)to_16(T{}, v[0] * inv) | ((uint32_t)to_16(T{}, v[1] * inv) << 16);
    dst[1] = (uint32_t)to_16(T{}, v[2] * inv) | ((uint32_t)to_16(T{}, v[3] * inv) << 16);
    if (a.lse && d == 0) a.lse[o] = attn8_lse(r, l);
  }
}

// ---- many rows of a sequence.  A workgroup takes 256 rows, a wave 32 of them as the columns of
// 32x32x16 products; 64 positions at a time go through LDS as fp16, decoded once for all waves: K as rows of
// positions (16 bytes more than D numbers long: 16 lanes that read one piece of 16 rows meet all banks),
// V as [block][c][dim] of the eight positions that lane quarter c of the second product holds.
constexpr int kRows8 = 256, kTileR8 = 64;

typedef float f32x16 __attribute__((ext_vector_type(16)));
__device__ __forceinline__ f32x16 mma32(const Raw<16>& a, const Raw<16>& b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8, a), __builtin_bit_cast(half8, b), c, 0, 0, 0);
}

template <class T, int NG>
__global__ __launch_bounds__(512) void k_attn_q8_rows(Attn8Args a) {
  constexpr int D = 32 * NG, kRow = 2 * D + 16, kK = kTileR8 * kRow, kV = kTileR8 * 2 * D, kPieces = 8 * D, PT = (kPieces + 511) / 512;
  __shared__ __attribute__((aligned(16))) uint8_t mem[2][kK + kV];
  __shared__ float4 consts[2][kTileR8 / kBlk8];                // of a block: ks k2, log2 vs, 1 / vs
  const int lane = opaque_lane(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n = lane & 31, c = lane >> 5;
  const int h = blockIdx.x % a.kv.Hkv, rt = a.RT - 1 - blockIdx.x / a.kv.Hkv, b = blockIdx.y;   // long tiles first
  const Seq8 sq = rows8_seq(a.rows, b);
  const int rows = min(kRows8, sq.n * a.G - kRows8 * rt);
  if (rows <= 0) return;
  const int start = a.starts ? max(a.starts[b], 0) : 0, first = sq.len - sq.n;
  const int i0 = kRows8 * rt / a.G, i1 = (kRows8 * rt + rows - 1) / a.G;
  const int p_lo = max(0, row8_lo(a, start, first + i0)), p_hi = min(first + i1 + 1, a.kv.max_pages << a.kv.page_shift);
  const int t0 = p_lo / kTileR8, t1 = p_hi > p_lo ? (p_hi + kTileR8 - 1) / kTileR8 : t0;

  // this wave's rows and this lane's
  const int w0 = kRows8 * rt + 32 * wave, wrows = min(32, kRows8 * rt + rows - w0);
  const int r = w0 + min(n, max(wrows, 1) - 1), tok = min(r / a.G, sq.n - 1), head = h * a.G + r % a.G;
  const int pos = first + tok, lo = row8_lo(a, start, pos), hi = pos + 1;
  const int any_lo = row8_lo(a, start, first + w0 / a.G), any_hi = first + (w0 + max(wrows, 1) - 1) / a.G + 1;
  const int all_lo = row8_lo(a, start, any_hi - 1), all_hi = first + w0 / a.G + 1;
  Raw<16> qf[2 * NG];
  float qs;
  {
    const uint8_t* row = a.q + (size_t)(sq.first + tok) * a.ldq + (size_t)head * D * 2;
    float top = 0.f;
#pragma unroll
    for (int g = 0; g < 2 * NG; ++g) {
      qf[g] = load_raw<16>(row + (16 * g + 8 * c) * 2);
      float x[8];
      unpack<T, 4>(qf[g].w, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(x[j]));
    }
    top = fmaxf(top, __uint_as_float(lane_xor_u32<32>(__float_as_uint(top), lane)));
    const int e = query8_exponent(top);
#pragma unroll
    for (int g = 0; g < 2 * NG; ++g) {
      float x[8];
      unpack<T, 4>(qf[g].w, x);
#pragma unroll
      for (int j = 0; j < 4; ++j) qf[g].w[j] = pack8_f16(ldexpf(x[2 * j], -e), ldexpf(x[2 * j + 1], -e));
    }
    qs = ldexpf(1.f, e);
  }
  float ref = kRefMin8, sum = 0.f;
  f32x16 acc[NG];
#pragma unroll
  for (int m = 0; m < NG; ++m) acc[m] = f32x16{0.f};

  // pieces of 16 bytes: K of the tile's four blocks, then V
  Raw<16> piece[PT];
  float2 scales = make_float2(0.f, 0.f);
  int ids = 0, next_consts = -1;
  const auto fetch = [&](int t) {
    if (((t - t0) & 15) == 0) {                                // page ids of 16 tiles, a block to a lane
      const int p = (min(t + (lane >> 2), t1 - 1)) * kTileR8 + (lane & 3) * kBlk8;
      ids = kv_page(a.kv, b, p);
    }
    const int at = ((t - t0) & 15) * 4;
#pragma unroll
    for (int j = 0; j < PT; ++j) {
      const int e = min(j * 512 + (int)threadIdx.x, kPieces - 1), part = e / (4 * D), u = (e % (4 * D)) / D;
      const int id = __shfl(ids, at + u);
      piece[j] = load_raw<16>(attn8_block(a.kv, h, id, t * kTileR8 + u * kBlk8) + part * 16 * D + 16 * (e % D));
    }
    next_consts = __shfl(ids, at + (lane & 3));
    if (threadIdx.x < kTileR8 / kBlk8)
      scales = *(const float2*)(attn8_block(a.kv, h, next_consts, t * kTileR8 + lane * kBlk8) + 32 * D);
  };
  const auto decode = [&](int buf) {
    uint8_t* kb = mem[buf];
    uint8_t* vb = kb + kK;
#pragma unroll
    for (int j = 0; j < PT; ++j) {
      const int e = j * 512 + threadIdx.x;
      if (e >= kPieces) continue;
      const int part = e / (4 * D), u = (e % (4 * D)) / D, o = 16 * (e % D);
      const Raw<16> x = codes8(piece[j].w[0], piece[j].w[1]), y = codes8(piece[j].w[2], piece[j].w[3]);
      if (part == 0) {
        uint8_t* to = kb + (u * kBlk8 + o / D) * kRow + (o % D) * 2;
        *(Raw<16>*)to = x;
        *(Raw<16>*)(to + 16) = y;
      } else {
        const int q = o / (4 * D), d = (o % (4 * D)) / 4;
        uint8_t* to = vb + ((u * 2 + (q & 1)) * D + d) * 16 + (q >> 1) * 8;
        *(Raw<8>*)to = Raw<8>{{x.w[0], x.w[1]}};
        *(Raw<8>*)(to + 16) = Raw<8>{{x.w[2], x.w[3]}};
        *(Raw<8>*)(to + 32) = Raw<8>{{y.w[0], y.w[1]}};
        *(Raw<8>*)(to + 48) = Raw<8>{{y.w[2], y.w[3]}};
      }
    }
    if (threadIdx.x < kTileR8 / kBlk8) {
      const float vs = scales.y != 0.f ? scales.y : kNoScale;
      // a block without a page counts nowhere
      consts[buf][threadIdx.x] = next_consts >= 0 ? make_float4(scales.x * a.k2, log2f(vs), 1.0f / vs, 1.f) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  };

  if (t0 < t1) fetch(t0);
  for (int t = t0; t < t1; ++t) {
    const int buf = (t - t0) & 1;
    decode(buf);
    __syncthreads();
    if (t + 1 < t1) fetch(t + 1);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int p0 = t * kTileR8 + 32 * s;
      if (wrows <= 0 || p0 >= any_hi || p0 + 32 <= any_lo) continue;
      const uint8_t* kr = mem[buf] + (32 * s + n) * kRow + 16 * c;
      f32x16 sc = {0.f};
#pragma unroll
      for (int g = 0; g < 2 * NG; ++g) sc = mma32(load_raw<16>(kr + 32 * g), qf[g], sc);
      const float4 k0 = consts[buf][2 * s], k1 = consts[buf][2 * s + 1];
      const float kk[2] = {k0.x * qs, k1.x * qs}, lv[2] = {k0.y, k1.y};
      float iv[2] = {k0.z, k1.z};
      float e[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) e[i] = fmaf(sc[i], kk[i >> 3], lv[i >> 3]);
      if (!(p0 >= all_lo && p0 + 32 <= all_hi && k0.w != 0.f && k1.w != 0.f)) {
        bool on[2] = {false, false};
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int p = p0 + 8 * (i >> 2) + 4 * c + (i & 3);
          const bool in = p >= lo && p < hi && (i < 8 ? k0.w : k1.w) != 0.f;
          on[i >> 3] |= in;
          if (!in) e[i] = -INFINITY;
        }
        if (!on[0]) iv[0] = 0.f;
        if (!on[1]) iv[1] = 0.f;
      }
      float top = e[0];
#pragma unroll
      for (int i = 1; i < 16; ++i) top = fmaxf(top, e[i]);
      if (__any(top > ref + 6.f)) {
        const float next = fmaxf(fmaxf(top, __uint_as_float(lane_xor_u32<32>(__float_as_uint(top), lane))), ref);
        const float f = exp2f(ref - next);
        ref = next;
        sum *= f;
#pragma unroll
        for (int m = 0; m < NG; ++m)
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[m][i] *= f;
      }
      const float off = 9.f - ref;
      Raw<16> p[2];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float e0 = __builtin_amdgcn_exp2f(e[2 * i] + off), e1 = __builtin_amdgcn_exp2f(e[2 * i + 1] + off);
        sum = fmaf(e0, iv[i >> 2], sum);
        sum = fmaf(e1, iv[i >> 2], sum);
        p[i >> 2].w[i & 3] = pack8_f16(e0, e1);
      }
      const uint8_t* vr = mem[buf] + kK + ((4 * s + c) * D + n) * 16;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int m = 0; m < NG; ++m) acc[m] = mma32(load_raw<16>(vr + (2 * j * D + 32 * m) * 16), p[j], acc[m]);
    }
  }

  if (n >= wrows) return;
  sum += __uint_as_float(lane_xor_u32<32>(__float_as_uint(sum), lane));
  const float inv = sum != 0.f ? 1.0f / sum : 0.f;
  const size_t o = (size_t)(sq.first + tok) * a.Hq + head;
#pragma unroll
  for (int m = 0; m < NG; ++m)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      Raw<8> w;
#pragma unroll
      for (int j = 0; j < 2; ++j)
        w.w[j] = (uint32_t)to_16(T{}, acc[m][4 * q + 2 * j] * inv) | ((uint32_t)to_16(T{}, acc[m][4 * q + 2 * j + 1] * inv) << 16);
      *(Raw<8>*)(a.out + (o * D + 32 * m + 8 * q + 4 * c) * 2) = w;
    }
  if (a.lse && c == 0) a.lse[o] = attn8_lse(ref, sum);
}

template <class T, int NG>
hipError_t attn8_run(hipStream_t s, const Attn8Args& a, bool rows) {
  if (rows) {
    k_attn_q8_rows<T, NG><<<dim3(a.RT * a.kv.Hkv, a.kv.B), dim3(512), 0, s>>>(a);
    return hipGetLastError();
  }
  k_attn_q8<T, NG><<<dim3(a.S * a.RT, a.kv.Hkv, a.kv.B), dim3(attn8_waves(NG) * kWave), 0, s>>>(a);
  if (a.S > 1) k_attn8_join<T, NG><<<dim3(a.kv.Hkv * a.rows.most * a.G, a.kv.B), dim3(256), 0, s>>>(a);
  return hipGetLastError();
}

template <class T>
hipError_t attn8_launch(hipStream_t s, const Attn8Args& a, bool rows) {
  switch (a.kv.D >> 5) {
    case 1: return attn8_run<T, 1>(s, a, rows);
    case 2: return attn8_run<T, 2>(s, a, rows);
    case 3: return attn8_run<T, 3>(s, a, rows);
    case 4: return attn8_run<T, 4>(s, a, rows);
    case 5: return attn8_run<T, 5>(s, a, rows);
    case 6: return attn8_run<T, 6>(s, a, rows);
    case 7: return attn8_run<T, 7>(s, a, rows);
    default: return attn8_run<T, 8>(s, a, rows);
  }
}

}  // namespace
}  // namespace sfx
