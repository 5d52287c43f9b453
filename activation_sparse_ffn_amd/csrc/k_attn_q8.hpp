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
//            takes P / vs in fp32.  That holds every weight down to 2^-39 of the largest while the scales of
//            a row's blocks lie within 2^-64 .. 2^32; from the first block outside on, a row's sum has a
//            reference of its own, the largest score, and takes a second exponential (State8::wide;
//            the test for it costs 1 to 4%).  One term for fp16 results too: they are off by 2.7e-4 of
//            themselves, 2.1e-4 of it their own rounding, which a second term (2^-22, as the int4 attention takes,
//            whose products are fewer) would leave alone; but then one token over 131072 positions takes 54 us
//            instead of 53, eight 115 instead of 103, 8192 tokens in one sequence 769 instead of 566;
//   output   value codes as rows of 16 dims x 32 positions.
// The lane that holds a score holds it in the place where the second product wants the weight.
// 131072 positions of 8 kv heads of 128 for 64 query heads: 56-58 us (270 MB, 4.7 TB/s of a streaming 5.3), the
// join 4.3.  8192 tokens of 32 / 8 heads of 128 in one sequence: 566 us (971 TFLOP/s).
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
constexpr float kNotWide = INFINITY;
// (In whole numbers, which scales that all lanes hold alike are for the scalar unit.)
__device__ __forceinline__ bool wide_scale8(uint32_t vs) { return vs != 0 && vs - 0x1F800000u > 0x4F800000u - 0x1F800000u; }
constexpr int attn8_waves(int NG) { return NG <= 4 ? 8 : 4; }

struct Attn8Args {
  KvCache kv;
  Rows8 rows;
  const uint8_t* q;
  size_t ldq;               // bytes between tokens
  const int32_t* starts;
  uint8_t* out;             // [T][Hq][D] 16 bit
  float* lse;               // [T][Hq] or null
  float* parts;             // [B][Hkv][row tiles][S] x ([R][D] sums, [R][4] their reference, that of the weights' sum, that sum), R rows a tile
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
__device__ __forceinline__ uint32_t quarters_or8(uint32_t v, int lane) {
  v |= lane_xor_u32<32>(v, lane);
  return v | lane_xor_u32<16>(v, lane);
}

// Adds weights of scores x (-inf: does not count) to a sum of weights 2^(x - wide + 9).
template <int N>
__device__ __forceinline__ void add_weights8(const float (&x)[N], float& wide, float& sum) {
  float next = wide;
#pragma unroll
  for (int i = 0; i < N; ++i) next = fmaxf(next, x[i]);
  sum *= __builtin_amdgcn_exp2f(wide - next);
#pragma unroll
  for (int i = 0; i < N; ++i) sum += __builtin_amdgcn_exp2f(x[i] - next + 9.f);
  wide = next;
}
// 2^x as f 2^e: results may lie below fp32's normal numbers.
struct Power8 {
  float f;
  int e;
};
__device__ __forceinline__ Power8 power8(float x) {
  const float i = floorf(x);
  return Power8{__builtin_amdgcn_exp2f(x - i), (int)i};
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
  float wide;               // the sum's own reference, or kNotWide: ref
  f32x4 acc[2 * NG];        // of product m: dims (4 c + i) 2 NG + m
};

// NC tiles of 16 rows at once, so that codes are decoded once for them.  `on`: bit 4 u + i says that
// position 4 c + i of block u counts for this lane's row (all ones where `full`).
// `any_wide`: a row of the wave has a reference of its own for its sum.
template <int NG, int NC>
__device__ __forceinline__ void tile8_run(const Tile8<NG>& t, const Raw<16> (&qf)[NC][NG], float k2, const float (&qs)[NC],
                                          bool full, const uint32_t (&on)[NC], int lane, State8<NG> (&st)[NC], bool& any_wide) {
  float s[NC][8], lv[2], inv[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    f32x4 p[NC];
#pragma unroll
    for (int j = 0; j < NC; ++j) p[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const Raw<16> k = codes8(t.k[u][2 * g], t.k[u][2 * g + 1]);
#pragma unroll
      for (int j = 0; j < NC; ++j) p[j] = Mma<TF16>::run(k, qf[j][g], p[j]);
    }
    const float vs = t.s[u].y != 0.f ? t.s[u].y : kNoScale;
    lv[u] = log2f(vs);
    inv[u] = 1.0f / vs;
#pragma unroll
    for (int j = 0; j < NC; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[j][4 * u + i] = fmaf(p[j][i], t.s[u].x * k2 * qs[j], lv[u]);
  }
  const bool apart[2] = {wide_scale8(__builtin_amdgcn_readfirstlane(__float_as_uint(t.s[0].y))),
                         wide_scale8(__builtin_amdgcn_readfirstlane(__float_as_uint(t.s[1].y)))};
  Raw<16> w[NC];
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    float iv[2] = {inv[0], inv[1]};
    if (!full) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (!((on[j] >> i) & 1u)) s[j][i] = -INFINITY;
      // a block none of whose positions counts may hold anything
      if (!(on[j] & 0x0Fu)) iv[0] = 0.f;
      if (!(on[j] & 0xF0u)) iv[1] = 0.f;
    }
    if (__builtin_expect(any_wide || apart[0] || apart[1], 0)) {
      const uint32_t row = quarters_or8(on[j], lane);
      if (st[j].wide == kNotWide && ((apart[0] && (row & 0x0Fu)) || (apart[1] && (row & 0xF0u)))) st[j].wide = st[j].ref;
      if (__any(st[j].wide != kNotWide)) any_wide = true;
      if (st[j].wide != kNotWide) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = (on[j] >> i) & 1u ? s[j][i] - lv[i >> 2] : -INFINITY;
        add_weights8(x, st[j].wide, st[j].sum);
        iv[0] = iv[1] = 0.f;
      }
    }
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, s[j][i]);
    if (__any(top > st[j].ref + 6.f)) {
      const float next = fmaxf(quarters_max8(top, lane), st[j].ref), f = exp2f(st[j].ref - next);
      st[j].ref = next;
      st[j].sum *= st[j].wide == kNotWide ? f : 1.f;
#pragma unroll
      for (int m = 0; m < 2 * NG; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) st[j].acc[m][i] *= f;
    }
    const float off = 9.f - st[j].ref;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float e0 = __builtin_amdgcn_exp2f(s[j][2 * i] + off), e1 = __builtin_amdgcn_exp2f(s[j][2 * i + 1] + off);
      st[j].sum = fmaf(e0, iv[i >> 1], st[j].sum);
      st[j].sum = fmaf(e1, iv[i >> 1], st[j].sum);
      w[j].w[i] = pack8_f16(e0, e1);
    }
  }
#pragma unroll
  for (int m = 0; m < 2 * NG; ++m) {
    const Raw<16> v = codes8(t.v[0][m], t.v[1][m]);
#pragma unroll
    for (int j = 0; j < NC; ++j) st[j].acc[m] = Mma<TF16>::run(v, w[j], st[j].acc[m]);
  }
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

// Positions [start, end) that some row of a tile of rows covers, as tiles t0 .. t0 + ntile - 1 cut into
// `active` runs of `per`: S even runs, none shorter than `least`.
struct Span8 {
  int start, end, t0, ntile, per, active;
};
// (The difference stays within 32 bits for rows in front of position 0 and any window too.)
__device__ __forceinline__ int row8_lo(const Attn8Args& a, int start, int pos) {
  return a.window && pos >= a.window ? max(start, pos + 1 - a.window) : start;
}
// The same for `R` rows at a time, `step` positions to a tile and runs of at least `least` tiles.
__device__ __forceinline__ Span8 span8(const Attn8Args& a, const Seq8& sq, int start, int rt, int R, int step, int least) {
  const int i0 = R * rt / a.G, i1 = min(sq.n - 1, (R * rt + R - 1) / a.G);      // first and last token of the tile
  Span8 s;
  s.start = max(0, row8_lo(a, start, sq.pos + i0));
  s.end = min(sq.pos + i1 + 1, a.kv.max_pages << a.kv.page_shift);
  s.t0 = s.start / step;
  s.ntile = s.end > s.start ? (s.end + step - 1) / step - s.t0 : 0;
  s.per = max(least, (s.ntile + a.S - 1) / a.S);
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

template <class T, int NG, int NC>
__global__ __launch_bounds__(attn8_waves(NG) * kWave) void k_attn_q8(Attn8Args a) {
  constexpr int W = attn8_waves(NG), D = 32 * NG, kThreads = W * kWave, R = 16 * NC;
  __shared__ float sh_ref[W][16], sh_wide[W][16], sh_sum[W][16];
  __shared__ __attribute__((aligned(8))) uint8_t sh_any[W];
  __shared__ __attribute__((aligned(16))) float sh_acc[W * 16 * (D + 4)];
  const int lane = opaque_lane(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, c = lane >> 4;
  const int split = blockIdx.x % a.S, rt = blockIdx.x / a.S, h = blockIdx.y, b = blockIdx.z;
  const Seq8 sq = rows8_seq(a.rows, b);
  const int rows = min(R, sq.n * a.G - R * rt);                // of this tile
  if (rows <= 0) return;
  const int start = a.starts ? max(a.starts[b], 0) : 0, first = sq.pos;
  const Span8 sp = span8(a, sq, start, rt, R, kTile8, W);
  if (split >= sp.active) return;
  const int tb = sp.t0 + split * sp.per, te = min(sp.t0 + sp.ntile, tb + sp.per);

  // this lane's rows; columns past the last one repeat it
  int lo[NC], hi[NC];
  float qs[NC];
  Raw<16> qf[NC][NG];
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    const int r = R * rt + min(16 * j + n, rows - 1), tok = r / a.G, head = h * a.G + r % a.G;
    lo[j] = row8_lo(a, start, first + tok);
    hi[j] = first + tok + 1;
    qs[j] = query8<T, NG>(a.q + (size_t)(sq.first + tok) * a.ldq + (size_t)head * D * 2, 16 * j + n < rows, c, lane, qf[j]);
  }
  // what every row covers
  const int all_lo = row8_lo(a, start, first + (R * rt + rows - 1) / a.G), all_hi = first + R * rt / a.G + 1;
  State8<NG> st[NC];
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    st[j].ref = kRefMin8;
    st[j].sum = 0.f;
    st[j].wide = kNotWide;
#pragma unroll
    for (int m = 0; m < 2 * NG; ++m) st[j].acc[m] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  bool any_wide = false;
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
      uint32_t on[NC];
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        on[j] = 0xFFu;
        if (!full) {
          on[j] = 0;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int p = p0 + (e >> 2) * kBlk8 + 4 * c + (e & 3);
            if (p >= lo[j] && p < hi[j] && ((e >> 2) ? id1 : id0) >= 0) on[j] |= 1u << e;
          }
        }
      }
      tile8_run<NG, NC>(cur, qf, a.k2, qs, full, on, lane, st, any_wide);
      cur = nxt;
      ids = next_ids;
    }
  }

  // join the waves, 16 rows at a time; without wide rows both references are the same
  if (lane == 0) sh_any[wave] = any_wide;
  constexpr size_t run = R * (D + 4);
  float* part = a.parts + ((((size_t)b * a.kv.Hkv + h) * a.RT + rt) * a.S + split) * run;
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    if (16 * j >= rows) break;
    if (j > 0) __syncthreads();
    float base = st[j].ref, sum = st[j].sum;
    if (any_wide) {                                            // quarters have references of their own
      const float mine = st[j].wide == kNotWide ? base : st[j].wide;
      base = quarters_max8(mine, lane);
      sum *= exp2f(mine - base);
    }
    sum = quarters_sum8(sum, lane);
    if (c == 0) {
      sh_ref[wave][n] = st[j].ref;
      sh_wide[wave][n] = base;
      sh_sum[wave][n] = sum;
    }
#pragma unroll
    for (int m = 0; m < 2 * NG; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) sh_acc[(wave * 16 + n) * (D + 4) + (4 * c + i) * 2 * NG + m] = st[j].acc[m][i];
    __syncthreads();
    using Flags = std::conditional_t<W == 8, uint64_t, uint32_t>;
    const bool apart = *(const Flags*)sh_any != 0;
    for (int e = threadIdx.x; e < min(16, rows - 16 * j) * (D / 2); e += kThreads) {
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
      float wide = ref;
      if (apart) {
        wide = sh_wide[0][rr];
#pragma unroll
        for (int w = 1; w < W; ++w) wide = fmaxf(wide, sh_wide[w][rr]);
        l = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) l = fmaf(exp2f(sh_wide[w][rr] - wide), sh_sum[w][rr], l);
      }
      if (sp.active == 1) {
        const int q = R * rt + 16 * j + rr;
        const size_t o = (size_t)(sq.first + q / a.G) * a.Hq + h * a.G + q % a.G;
        const Power8 up = power8(ref - wide);
        const float inv = l != 0.f ? up.f / l : 0.f;
        ((uint32_t*)a.out)[(o * D + d) >> 1] = (uint32_t)to_16(T{}, ldexpf(v0 * inv, up.e)) | ((uint32_t)to_16(T{}, ldexpf(v1 * inv, up.e)) << 16);
        if (a.lse && d == 0) a.lse[o] = attn8_lse(wide, l);
      } else {
        *reinterpret_cast<float2*>(part + (16 * j + rr) * D + d) = make_float2(v0, v1);
        if (d == 0) *reinterpret_cast<float4*>(part + R * D + 4 * (16 * j + rr)) = make_float4(ref, wide, l, 0.f);
      }
    }
  }
}

// Joins the runs of a row, one workgroup per row: the runs' references first, then four dims to a thread,
// the runs dealt out over groups of D / 4 threads and the groups' sums added in order.  Tiles of R
// rows as span8 cuts them.
template <class T, int NG>
__global__ __launch_bounds__(256) void k_attn8_join(Attn8Args a, int R, int step, int least) {
  constexpr int D = 32 * NG, kItems = D / 4, kGroups = 256 / kItems;
  __shared__ __attribute__((aligned(16))) float sh_v[kGroups][D];
  __shared__ float sh_f[256], sh_l[256 / kWave], sh_r[256 / kWave], sh_w[256 / kWave];
  const int b = blockIdx.y, per_head = a.rows.most * a.G, h = blockIdx.x / per_head, q = blockIdx.x % per_head;
  const Seq8 sq = rows8_seq(a.rows, b);
  if (q >= sq.n * a.G) return;
  const int rt = q / R, rr = q % R;
  const Span8 sp = span8(a, sq, a.starts ? max(a.starts[b], 0) : 0, rt, R, step, least);
  if (sp.active == 1) return;                                   // the attention kernel wrote the row
  const size_t run = (size_t)R * (D + 4);
  const float* part = a.parts + (((size_t)b * a.kv.Hkv + h) * a.RT + rt) * a.S * run;
  const float* rs = part + (size_t)R * D + 4 * rr;
  const int grp = threadIdx.x / kItems, d = 4 * (threadIdx.x % kItems), wave = threadIdx.x >> 6;
  float ref = kRefMin8, wide = kRefMin8, l = 0.f;
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  for (int k0 = 0; k0 < sp.active; k0 += 256) {                 // 256 runs at a time (there are hardly more)
    const int k = k0 + threadIdx.x;
    const float4 rl = k < sp.active ? *reinterpret_cast<const float4*>(rs + k * run) : make_float4(kRefMin8, kRefMin8, 0.f, 0.f);
    float top = rl.x, top_w = rl.y;
#pragma unroll
    for (int o = 32; o; o >>= 1) {
      top = fmaxf(top, __shfl_xor(top, o));
      top_w = fmaxf(top_w, __shfl_xor(top_w, o));
    }
    if ((threadIdx.x & 63) == 0) {
      sh_r[wave] = top;
      sh_w[wave] = top_w;
    }
    __syncthreads();
    float next = ref, next_w = wide;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      next = fmaxf(next, sh_r[w]);
      next_w = fmaxf(next_w, sh_w[w]);
    }
    const float f = exp2f(rl.x - next), back = exp2f(ref - next);
    sh_f[threadIdx.x] = f;
    float sum = exp2f(rl.y - next_w) * rl.z;
#pragma unroll
    for (int o = 32; o; o >>= 1) sum += __shfl_xor(sum, o);
    if ((threadIdx.x & 63) == 0) sh_l[wave] = sum;
    __syncthreads();
    l = l * exp2f(wide - next_w) + ((sh_l[0] + sh_l[1]) + (sh_l[2] + sh_l[3]));
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] *= back;
    ref = next;
    wide = next_w;
    if (grp < kGroups) {
      const int n = min(256, sp.active - k0);
#pragma unroll 8
      for (int k = grp; k < n; k += kGroups) {
        const f32x4 pk = *reinterpret_cast<const f32x4*>(part + (k0 + k) * run + rr * D + d);
        const float w = sh_f[k];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = fmaf(w, pk[i], v[i]);
      }
    }
    __syncthreads();
  }
  if (grp < kGroups) *reinterpret_cast<f32x4*>(&sh_v[grp][d]) = v;
  __syncthreads();
  if (threadIdx.x < kItems) {
    v = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
      const f32x4 o = *reinterpret_cast<const f32x4*>(&sh_v[k][d]);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += o[i];
    }
    const size_t o = (size_t)(sq.first + q / a.G) * a.Hq + h * a.G + q % a.G;
    const Power8 up = power8(ref - wide);
    const float inv = l != 0.f ? up.f / l : 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = ldexpf(v[i] * inv, up.e);
    uint32_t* dst = (uint32_t*)a.out + ((o * D + d) >> 1);
    dst[0] = (uint32_t)to_16(T{}, v[0]) | ((uint32_t)to_16(T{}, v[1]) << 16);
    dst[1] = (uint32_t)to_16(T{}, v[2]) | ((uint32_t)to_16(T{}, v[3]) << 16);
    if (a.lse && d == 0) a.lse[o] = attn8_lse(wide, l);
  }
}

// The same for few runs of many rows (at most kFewRuns8), a wave per row: D / 4 lanes read a run, the
// others the next ones.
constexpr int kFewRuns8 = 16;
template <class T, int NG>
__global__ __launch_bounds__(256) void k_attn8_join_few(Attn8Args a, int R, int step, int least) {
  constexpr int D = 32 * NG, kItems = D / 4, kGroups = kWave / kItems;
  const int lane = opaque_lane(), b = blockIdx.y, per_head = a.rows.most * a.G;
  const int x = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), h = x / per_head, q = x % per_head;
  const Seq8 sq = rows8_seq(a.rows, b);
  if (h >= a.kv.Hkv || q >= sq.n * a.G) return;
  const int rt = q / R, rr = q % R;
  const Span8 sp = span8(a, sq, a.starts ? max(a.starts[b], 0) : 0, rt, R, step, least);
  if (sp.active == 1) return;                                   // the attention kernel wrote the row
  const size_t run = (size_t)R * (D + 4);
  const float* part = a.parts + (((size_t)b * a.kv.Hkv + h) * a.RT + rt) * a.S * run;
  const float4 rl = lane < sp.active ? *reinterpret_cast<const float4*>(part + (size_t)R * D + 4 * rr + lane * run)
                                     : make_float4(kRefMin8, kRefMin8, 0.f, 0.f);
  float ref = rl.x, wide = rl.y;
#pragma unroll
  for (int o = 8; o; o >>= 1) {
    ref = fmaxf(ref, __shfl_xor(ref, o));
    wide = fmaxf(wide, __shfl_xor(wide, o));
  }
  ref = __shfl(ref, 0);
  wide = __shfl(wide, 0);
  const float f = exp2f(rl.x - ref);
  float l = exp2f(rl.y - wide) * rl.z;
#pragma unroll
  for (int o = 8; o; o >>= 1) l += __shfl_xor(l, o);
  l = __shfl(l, 0);
  const int grp = lane / kItems, d = 4 * (lane % kItems);
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int k = 0; k < sp.active; k += kGroups) {
    const int mine = k + grp;
    const bool in = grp < kGroups && mine < sp.active;
    const f32x4 pk = *reinterpret_cast<const f32x4*>(part + (in ? mine : 0) * run + rr * D + d);
    const float w = __shfl(f, mine & (kWave - 1));
    if (in)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = fmaf(w, pk[i], v[i]);
  }
  f32x4 o4 = v;
#pragma unroll
  for (int k = 1; k < kGroups; ++k)
#pragma unroll
    for (int i = 0; i < 4; ++i) o4[i] += __shfl(v[i], (lane + k * kItems) & (kWave - 1));
  if (lane >= kItems) return;
  const size_t o = (size_t)(sq.first + q / a.G) * a.Hq + h * a.G + q % a.G;
  const Power8 up = power8(ref - wide);
  const float inv = l != 0.f ? up.f / l : 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) o4[i] = ldexpf(o4[i] * inv, up.e);
  uint32_t* dst = (uint32_t*)a.out + ((o * D + d) >> 1);
  dst[0] = (uint32_t)to_16(T{}, o4[0]) | ((uint32_t)to_16(T{}, o4[1]) << 16);
  dst[1] = (uint32_t)to_16(T{}, o4[2]) | ((uint32_t)to_16(T{}, o4[3]) << 16);
  if (a.lse && d == 0) a.lse[o] = attn8_lse(wide, l);
}

// ---- many rows of a sequence.  A workgroup takes 128 or 256 rows (attn8_rows), a wave 32 of them as the
// columns of 32x32x16 products; 64 positions at a time go through LDS as fp16, decoded once for all waves: K as rows of
// positions (16 bytes more than D numbers long: 16 lanes that read one piece of 16 rows meet all banks),
// V as [block][c][dim] of the eight positions that lane half c of the second product holds.
constexpr int kTileR8 = 64, kLeastR8 = 4;         // and tiles of positions that a run has at least

typedef float f32x16 __attribute__((ext_vector_type(16)));
__device__ __forceinline__ f32x16 mma32(const Raw<16>& a, const Raw<16>& b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8, a), __builtin_bit_cast(half8, b), c, 0, 0, 0);
}

template <class T, int NG>
__global__ __launch_bounds__(2 * attn8_rows(NG), 2) void k_attn_q8_rows(Attn8Args a) {
  constexpr int kRows8 = attn8_rows(NG), NTH = 2 * kRows8;
  constexpr int D = 32 * NG, kRow = 2 * D + 16, kK = kTileR8 * kRow, kV = kTileR8 * 2 * D, kPieces = 4 * D, PT = (kPieces + NTH - 1) / NTH;
  constexpr bool kWhole = D % 64 == 0;                         // a wave's pieces are of one block
  __shared__ __attribute__((aligned(16))) uint8_t mem[2][kK + kV];
  __shared__ float4 consts[2][kTileR8 / kBlk8];                // of a block: ks k2, log2 vs, 1 / vs, 1 (0: no page, 2: wide_scale8)
  const int lane = opaque_lane(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n = lane & 31, c = lane >> 5;
  // a head's tiles on one XCD where heads are a multiple of 8; tiles with many positions first
  const int h = blockIdx.x % a.kv.Hkv, split = blockIdx.x / a.kv.Hkv % a.S, rt = a.RT - 1 - blockIdx.x / a.kv.Hkv / a.S, b = blockIdx.y;
  const Seq8 sq = rows8_seq(a.rows, b);
  const int rows = min(kRows8, sq.n * a.G - kRows8 * rt);
  if (rows <= 0) return;
  const int start = a.starts ? max(a.starts[b], 0) : 0, first = sq.pos;
  const Span8 sp = span8(a, sq, start, rt, kRows8, kTileR8, kLeastR8);
  if (split >= sp.active) return;
  const int t0 = sp.t0 + split * sp.per, t1 = min(sp.t0 + sp.ntile, t0 + sp.per);

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
  float ref = kRefMin8, sum = 0.f, wide = kNotWide;            // see State8
  bool any_wide = false;
  f32x16 acc[NG];
#pragma unroll
  for (int m = 0; m < NG; ++m) acc[m] = f32x16{0.f};

  // Pieces of 16 bytes of the tile's four blocks, K by the threads from the first on, V by the same
  // threads half the workgroup further, so that narrow heads give every thread one.
  Raw<16> pk[PT], pv8[PT];
  float2 scales = make_float2(0.f, 0.f);
  int ids = 0, const_id = -1;
  const auto place = [&](int j, int turn) { return j * NTH + (((int)threadIdx.x + turn) & (NTH - 1)); };   // piece number
  const auto fetch = [&](int t) {
    if (((t - t0) & 15) == 0) {                                // page ids of 16 tiles, a block to a lane
      const int p = (min(t + (lane >> 2), t1 - 1)) * kTileR8 + (lane & 3) * kBlk8;
      ids = kv_page(a.kv, b, p);
    }
    const int at = ((t - t0) & 15) * 4;
#pragma unroll
    for (int j = 0; j < PT; ++j)
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        const int e = min(place(j, part * (NTH / 2)), kPieces - 1);
        int u = e / D, id;
        if constexpr (kWhole) {
          u = __builtin_amdgcn_readfirstlane(u);
          id = __builtin_amdgcn_readlane(ids, at + u);
        } else {
          id = __shfl(ids, at + u);
        }
        const uint8_t* src = attn8_block(a.kv, h, id, t * kTileR8 + u * kBlk8);
        if (part == 0) {
          pk[j] = load_raw<16>(src + (size_t)(uint32_t)(16 * (e % D)));
        } else {                                               // quarters cq and cq + 2 of two dims
          const uint32_t at8 = 16 * D + ((e % D) / (D / 2) * D + (e % D) % (D / 2) * 2) * 4;
          const Raw<8> v0 = load_raw<8>(src + (size_t)at8), v1 = load_raw<8>(src + (size_t)at8 + 8 * D);
          pv8[j] = Raw<16>{{v0.w[0], v0.w[1], v1.w[0], v1.w[1]}};
        }
      }
    const_id = __shfl(ids, at + (lane & 3));
    if (threadIdx.x < kTileR8 / kBlk8)
      scales = *(const float2*)(attn8_block(a.kv, h, const_id, t * kTileR8 + lane * kBlk8) + 32 * D);
  };
  const auto decode = [&](int buf) {
    uint8_t* kb = mem[buf];
    uint8_t* vb = kb + kK;
#pragma unroll
    for (int j = 0; j < PT; ++j) {
      int e = place(j, 0);
      if (e < kPieces) {
        const int u = e / D, o = 16 * (e % D);
        uint8_t* to = kb + (u * kBlk8 + o / D) * kRow + (o % D) * 2;
        *(Raw<16>*)to = codes8(pk[j].w[0], pk[j].w[1]);
        *(Raw<16>*)(to + 16) = codes8(pk[j].w[2], pk[j].w[3]);
      }
      e = place(j, NTH / 2);
      if (e < kPieces) {
        uint8_t* to = vb + e * 32;                             // [block][c][dim] of 16 bytes
        *(Raw<16>*)to = codes8(pv8[j].w[0], pv8[j].w[2]);
        *(Raw<16>*)(to + 16) = codes8(pv8[j].w[1], pv8[j].w[3]);
      }
    }
    if (threadIdx.x < kTileR8 / kBlk8) {
      const float vs = scales.y != 0.f ? scales.y : kNoScale;
      // a block without a page counts nowhere
      consts[buf][threadIdx.x] = const_id >= 0 ? make_float4(scales.x * a.k2, log2f(vs), 1.0f / vs, wide_scale8(__float_as_uint(vs)) ? 2.f : 1.f) : make_float4(0.f, 0.f, 0.f, 0.f);
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
      float iv[2] = {k0.z, k1.z}, e[16];
      const float base = 9.f - ref;
#pragma unroll
      for (int i = 0; i < 16; ++i) e[i] = fmaf(sc[i], kk[i >> 3], lv[i >> 3] + base);
      if (!(p0 >= all_lo && p0 + 32 <= all_hi && k0.w == 1.f && k1.w == 1.f && !any_wide)) {
        bool on[2] = {false, false};
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int p = p0 + 8 * (i >> 2) + 4 * c + (i & 3);
          const bool in = (int)(p >= lo) & (int)(p < hi) & (int)((i < 8 ? k0.w : k1.w) != 0.f);
          on[i >> 3] |= in;
          e[i] = in ? e[i] : -INFINITY;
        }
        iv[0] = on[0] ? iv[0] : 0.f;
        iv[1] = on[1] ? iv[1] : 0.f;
        if (wide == kNotWide && ((k0.w > 1.f && p0 + kBlk8 > lo && p0 < hi) || (k1.w > 1.f && p0 + 2 * kBlk8 > lo && p0 + kBlk8 < hi)))
          wide = ref;
        if (__any(wide != kNotWide)) {
          any_wide = true;
          if (wide != kNotWide) {                              // eight at a time: registers
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              float x[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) x[i] = e[8 * u + i] == -INFINITY ? -INFINITY : sc[8 * u + i] * kk[u];
              add_weights8(x, wide, sum);
            }
            iv[0] = iv[1] = 0.f;
          }
        }
      }
      float top = e[0];
#pragma unroll
      for (int i = 1; i < 16; ++i) top = fmaxf(top, e[i]);
      if (__any(top > 15.f)) {
        // the scores themselves, what does not count left at -inf
        top = -INFINITY;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          e[i] = e[i] == -INFINITY ? -INFINITY : fmaf(sc[i], kk[i >> 3], lv[i >> 3]);
          top = fmaxf(top, e[i]);
        }
        const float next = fmaxf(fmaxf(top, __uint_as_float(lane_xor_u32<32>(__float_as_uint(top), lane))), ref);
        const float f = exp2f(ref - next), off = 9.f - next;
        ref = next;
        sum *= wide == kNotWide ? f : 1.f;
#pragma unroll
        for (int m = 0; m < NG; ++m)
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[m][i] *= f;
#pragma unroll
        for (int i = 0; i < 16; ++i) e[i] += off;
      }
      Raw<16> p[2];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float e0 = __builtin_amdgcn_exp2f(e[2 * i]), e1 = __builtin_amdgcn_exp2f(e[2 * i + 1]);
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
  float base = ref;
  if (any_wide) {                                              // the row's halves have references of their own
    const float mine = wide == kNotWide ? ref : wide;
    base = fmaxf(mine, __uint_as_float(lane_xor_u32<32>(__float_as_uint(mine), lane)));
    sum *= exp2f(mine - base);
  }
  sum += __uint_as_float(lane_xor_u32<32>(__float_as_uint(sum), lane));
  if (sp.active > 1) {
    const int rr = 32 * wave + n;
    float* part = a.parts + ((((size_t)b * a.kv.Hkv + h) * a.RT + rt) * a.S + split) * (size_t)(kRows8 * (D + 4));
#pragma unroll
    for (int m = 0; m < NG; ++m)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x4 v = {acc[m][4 * q], acc[m][4 * q + 1], acc[m][4 * q + 2], acc[m][4 * q + 3]};
        *reinterpret_cast<f32x4*>(part + rr * D + 32 * m + 8 * q + 4 * c) = v;
      }
    if (c == 0) *reinterpret_cast<float4*>(part + kRows8 * D + 4 * rr) = make_float4(ref, base, sum, 0.f);
    return;
  }
  const Power8 up = power8(ref - base);
  const float inv = sum != 0.f ? up.f / sum : 0.f;
  const size_t o = (size_t)(sq.first + tok) * a.Hq + head;
#pragma unroll
  for (int m = 0; m < NG; ++m)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      Raw<8> w;
#pragma unroll
      for (int j = 0; j < 2; ++j)
        w.w[j] = (uint32_t)to_16(T{}, ldexpf(acc[m][4 * q + 2 * j] * inv, up.e)) |
                 ((uint32_t)to_16(T{}, ldexpf(acc[m][4 * q + 2 * j + 1] * inv, up.e)) << 16);
      *(Raw<8>*)(a.out + (o * D + 32 * m + 8 * q + 4 * c) * 2) = w;
    }
  if (a.lse && c == 0) a.lse[o] = attn8_lse(base, sum);
}

template <class T, int NG, int NC>
void attn8_few(hipStream_t s, const Attn8Args& a) {
  k_attn_q8<T, NG, NC><<<dim3(a.S * a.RT, a.kv.Hkv, a.kv.B), dim3(attn8_waves(NG) * kWave), 0, s>>>(a);
}
template <class T, int NG>
hipError_t attn8_run(hipStream_t s, const Attn8Args& a, int R) {
  constexpr int kRows8 = attn8_rows(NG);
  if (R == kRows8) k_attn_q8_rows<T, NG><<<dim3(a.RT * a.S * a.kv.Hkv, a.kv.B), dim3(2 * kRows8), 0, s>>>(a);
  else if (R == 32) attn8_few<T, NG, 2>(s, a);
  else attn8_few<T, NG, 1>(s, a);
  const int step = R == kRows8 ? kTileR8 : kTile8, least = R == kRows8 ? kLeastR8 : attn8_waves(NG);
  const int rows = a.kv.Hkv * a.rows.most * a.G;
  if (a.S > kFewRuns8) k_attn8_join<T, NG><<<dim3(rows, a.kv.B), dim3(256), 0, s>>>(a, R, step, least);
  else if (a.S > 1) k_attn8_join_few<T, NG><<<dim3((rows + 3) / 4, a.kv.B), dim3(256), 0, s>>>(a, R, step, least);
  return hipGetLastError();
}

template <class T>
hipError_t attn8_launch(hipStream_t s, const Attn8Args& a, int R) {
  switch (a.kv.D >> 5) {
    case 1: return attn8_run<T, 1>(s, a, R);
    case 2: return attn8_run<T, 2>(s, a, R);
    case 3: return attn8_run<T, 3>(s, a, R);
    case 4: return attn8_run<T, 4>(s, a, R);
    case 5: return attn8_run<T, 5>(s, a, R);
    case 6: return attn8_run<T, 6>(s, a, R);
    case 7: return attn8_run<T, 7>(s, a, R);
    default: return attn8_run<T, 8>(s, a, R);
  }
}

}  // namespace
}  // namespace sfx
