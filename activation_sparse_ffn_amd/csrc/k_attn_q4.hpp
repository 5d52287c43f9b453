// Decode attention over the paged int4 key/value cache: one query token per sequence,
// Hq query heads sharing Hkv kv heads.
//
//   s_p = scale q . k_p,  p in [start, len);  o = sum_p e^(s_p - m) v_p / sum_p e^(s_p - m)
//
// One pass with a running reference and sum.  A wave takes 32 positions at a time:
//   scores   two 16x16x32 products per group of 32 dims, 16 positions (rows) x 16 query
//            heads (columns) each, on the codes (sfx_q4.hpp); the key's fp32 scale multiplies
//            each group's fp32 sum;
//   weights  P = 2^(s - ref + 9) in fp32, rounded to fp16 as the second product's operand (the
//            sum of weights keeps the fp32 values); the lane that holds a score holds it in
//            the place where the product wants the weight, so nothing crosses lanes;
//   output   codes times scale, rounded once to fp16, as rows of 16 dims x 32 positions.
// The reference is raised only when a score passes it by 6 (in powers of two), so P stays
// below 2^15; the 2^9 keeps weights down to 2^-33 of the largest above fp16's last bit.
#pragma once
#include "sfx_kv.hpp"
#include "sfx_launch.hpp"
#include "sfx_q4.hpp"

namespace sfx {
namespace {

constexpr int kAttnTile = 32;          // positions a wave takes at a time
constexpr float kRefMin = -3.0e38f;
// Waves of a workgroup, and whether the next tile's registers are loaded while one is worked
// on: from 160 dims on, two tiles do not fit the registers of two waves per SIMD.
constexpr int attn_waves(int NG) { return NG <= 4 ? 8 : 4; }
constexpr bool attn_ahead(int NG) { return NG <= 4; }

struct AttnArgs {
  KvCache kv;
  const uint8_t* q;
  size_t ldq;               // bytes between sequences
  const int32_t *starts, *lens;
  uint8_t* out;             // [B][Hq][D] 16 bit
  float* lse;               // [B][Hq] or null
  uint32_t* tickets;        // [B][Hkv][head tiles]
  float* parts;             // [B][Hkv][head tiles][S][HG][D + 4]
  float k2;                 // scale log2(e)
  int Hq, G, HT, HG, S;     // HG = heads of a full head tile, min(G, 16)
};

template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t* w) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const Raw<16> r = load_raw<16>(p + 16 * i);
#pragma unroll
      for (int j = 0; j < 4; ++j) w[4 * i + j] = r.w[j];
    }
  } else if constexpr (N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const Raw<8> r = load_raw<8>(p + 8 * i);
      w[2 * i] = r.w[0];
      w[2 * i + 1] = r.w[1];
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = *(const uint32_t*)(p + 4 * i);
  }
}

__device__ __forceinline__ uint32_t pk_add24(uint32_t a) {
  const half2_t k = {(_Float16)-24.0f, (_Float16)-24.0f};
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2_t, a) + k);
}
__device__ __forceinline__ uint32_t pk_mul(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2_t, a) * __builtin_bit_cast(half2_t, b));
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  const half2_t h = {(_Float16)a, (_Float16)b};
  return __builtin_bit_cast(uint32_t, h);
}
// Maximum / sum over the four quarters of a wave (lanes L, L ^ 16, L ^ 32, L ^ 48).
__device__ __forceinline__ float quarters_max(float v, int lane) {
  v = fmaxf(v, __uint_as_float(lane_xor_u32<32>(__float_as_uint(v), lane)));
  return fmaxf(v, __uint_as_float(lane_xor_u32<16>(__float_as_uint(v), lane)));
}
__device__ __forceinline__ float quarters_sum(float v, int lane) {
  v += __uint_as_float(lane_xor_u32<32>(__float_as_uint(v), lane));
  return v + __uint_as_float(lane_xor_u32<16>(__float_as_uint(v), lane));
}

// What a lane holds of 32 positions: K rows of position n % 4 (+ 4) of octet n / 4, words of
// quarter c; V unit n and the scales of octet c.
template <int NG>
struct AttnTile {
  uint32_t k[2][NG], v[2 * NG];
  Raw<16> ks[NG], vs[NG];
  uint32_t on;              // bit i: position i of octet c counts
};

// Pages of the two octets a lane reads in tile `it` (-1: none).
struct AttnPages {
  int k, v;
};
__device__ __forceinline__ AttnPages attn_pages(const AttnArgs& a, int b, int it, int n, int c) {
  return AttnPages{kv_page(a.kv, b, it * kAttnTile + 8 * (n >> 2)), kv_page(a.kv, b, it * kAttnTile + 8 * c)};
}

template <int NG>
__device__ __forceinline__ void attn_load(const AttnArgs& a, int h, int it, AttnPages id, int start, int end, int n, int c,
                                          AttnTile<NG>& x) {
  constexpr int D = 32 * NG;
  const int page_mask = (1 << a.kv.page_shift) - 1;
  const int pk = it * kAttnTile + 8 * (n >> 2), pv = it * kAttnTile + 8 * c;
  const uint8_t* bk = a.kv.base + kv_block(a.kv, max(id.k, 0), h, (pk & page_mask) >> 3);
  const uint8_t* bv = a.kv.base + kv_block(a.kv, max(id.v, 0), h, (pv & page_mask) >> 3);
#pragma unroll
  for (int t = 0; t < 2; ++t) load_words<NG>(bk + (4 * t + (n & 3)) * (D / 2) + c * 4 * NG, x.k[t]);
#pragma unroll
  for (int g = 0; g < NG; ++g) x.ks[g] = load_raw<16>(bv + 8 * D + 16 * g);
  load_words<2 * NG>(bv + 4 * D + n * 8 * NG, x.v);
#pragma unroll
  for (int g = 0; g < NG; ++g) x.vs[g] = load_raw<16>(bv + 8 * D + D / 2 + 16 * g);
  uint32_t on = id.v < 0 ? 0u : 0xFFu;
  const int lo = start - pv, hi = end - pv;
  if (lo > 0) on &= lo >= 8 ? 0u : 0xFFu << lo;
  if (hi < 8) on &= hi <= 0 ? 0u : (1u << hi) - 1u;
  x.on = on;
}

// Running state of a wave: per lane the head n, of products m the dims 16 m + 4 c + i.
template <int NG>
struct AttnState {
  float ref, sum;           // reference (all quarters alike), sum of this quarter's weights
  f32x4 acc[2 * NG];
};

template <class T, int NG>
__device__ __forceinline__ void attn_tile(AttnTile<NG>& x, const Raw<16> (&qf)[NG], float k2, int lane,
                                          AttnState<NG>& st) {
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  float s[8];
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      // the -24 sum(q) of the codes' offset as a product of its own: the matrix cores have
      // the time, and its result would hold 4 registers per group
      f32x4 p = Mma<T>::run(q4_minus24<T>(), qf[g], zero);
      p = Mma<T>::run(q4_word<T>(x.k[t][g]), qf[g], p);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float sc = half_at(x.ks[g].w[2 * t + (i >> 1)], i & 1);
        s[4 * t + i] = g == 0 ? sc * p[i] : fmaf(sc, p[i], s[4 * t + i]);
      }
    }
#pragma unroll
  for (int i = 0; i < 8; ++i) s[i] *= k2;
  if (!__all(x.on == 0xFFu)) {
    // some position does not count: its weight is 0 and so is its value, whatever is held there
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (!((x.on >> i) & 1u)) s[i] = -INFINITY;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t keep =
          ((x.on >> (2 * i)) & 1u ? 0xFFFFu : 0u) | ((x.on >> (2 * i + 1)) & 1u ? 0xFFFF0000u : 0u);
#pragma unroll
      for (int g = 0; g < NG; ++g) x.vs[g].w[i] &= keep;
    }
  }
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = fmaxf(top, s[i]);
  if (__any(top > st.ref + 6.f)) {
    const float next = fmaxf(quarters_max(top, lane), st.ref);
    const float f = exp2f(st.ref - next);
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
    st.sum += e0 + e1;
    p.w[i] = pack_f16(e0, e1);
  }
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    Raw<16> lo, hi;
    const uint32_t w0 = x.v[2 * g], w1 = x.v[2 * g + 1];
    lo.w[0] = q4_pair<TF16, 0>(w0);
    hi.w[0] = q4_pair<TF16, 1>(w0);
    lo.w[1] = q4_pair<TF16, 2>(w0);
    hi.w[1] = q4_pair<TF16, 3>(w0);
    lo.w[2] = q4_pair<TF16, 0>(w1);
    hi.w[2] = q4_pair<TF16, 1>(w1);
    lo.w[3] = q4_pair<TF16, 2>(w1);
    hi.w[3] = q4_pair<TF16, 3>(w1);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo.w[i] = pk_mul(pk_add24(lo.w[i]), x.vs[g].w[i]);
      hi.w[i] = pk_mul(pk_add24(hi.w[i]), x.vs[g].w[i]);
    }
    st.acc[2 * g] = Mma<TF16>::run(lo, p, st.acc[2 * g]);
    st.acc[2 * g + 1] = Mma<TF16>::run(hi, p, st.acc[2 * g + 1]);
  }
}

__device__ __forceinline__ float attn_lse(float ref, float sum) {
  return sum != 0.f ? (ref - 9.f + log2f(sum)) * 0.69314718055994531f : -INFINITY;
}

template <class T, int NG>
__global__ __launch_bounds__(attn_waves(NG) * kWave) void k_attn_q4(AttnArgs a) {
  constexpr int kAttnWaves = attn_waves(NG);
  constexpr int D = 32 * NG, kThreads = kAttnWaves * kWave;
  __shared__ float sh_ref[kAttnWaves][16], sh_sum[kAttnWaves][16];
  __shared__ __attribute__((aligned(16))) float sh_acc[kAttnWaves * 16 * (D + 4)];
  __shared__ uint32_t sh_last;
  const int lane = opaque_lane(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, c = lane >> 4;
  const int split = blockIdx.x, ht = blockIdx.y % a.HT, h = blockIdx.y / a.HT, b = blockIdx.z;
  const int heads = min(16, a.G - 16 * ht);                    // query heads of this workgroup
  const int max_len = a.kv.max_pages << a.kv.page_shift;
  const int end = min(a.lens[b], max_len);
  const int start = a.starts ? max(a.starts[b], 0) : 0;

  // this workgroup's tiles of 32 positions: the sequence's tiles in S even runs
  const int t0 = start / kAttnTile, t1 = (end + kAttnTile - 1) / kAttnTile;
  const int ntile = end > start ? t1 - t0 : 0;
  const int per = max(kAttnWaves, (ntile + a.S - 1) / a.S);
  const int active = max(1, (ntile + per - 1) / per);          // workgroups with work (one writes an empty row)
  if (split >= active) return;
  const int tb = t0 + split * per, te = min(t0 + ntile, tb + per);

  const int hq0 = h * a.G + 16 * ht;
  Raw<16> qf[NG];
#pragma unroll
  for (int g = 0; g < NG; ++g)
    qf[g] = n < heads ? load_raw<16>(a.q + (size_t)b * a.ldq + ((size_t)(hq0 + n) * D + 32 * g + 8 * c) * 2) : zero16();
  AttnState<NG> st;
  st.ref = kRefMin;
  st.sum = 0.f;
#pragma unroll
  for (int m = 0; m < 2 * NG; ++m) st.acc[m] = f32x4{0.f, 0.f, 0.f, 0.f};

  // two tiles in registers: the next one's loads are under way while one is worked on, the
  // pages of the one behind it are looked up before
  int it = tb + wave;
  if constexpr (!attn_ahead(NG)) {
    AttnTile<NG> x;
    for (; it < te; it += kAttnWaves) {
      attn_load<NG>(a, h, it, attn_pages(a, b, it, n, c), start, end, n, c, x);
      attn_tile<T, NG>(x, qf, a.k2, lane, st);
    }
  } else if (it < te) {
    AttnTile<NG> x, y;
    AttnPages id = attn_pages(a, b, it, n, c);
    AttnPages id1 = attn_pages(a, b, min(it + kAttnWaves, te - 1), n, c);
    attn_load<NG>(a, h, it, id, start, end, n, c, x);
    while (true) {
      int nx = it + kAttnWaves;
      if (nx < te) attn_load<NG>(a, h, nx, id1, start, end, n, c, y);
      id = attn_pages(a, b, min(nx + kAttnWaves, te - 1), n, c);
      __builtin_amdgcn_sched_barrier(0);
      attn_tile<T, NG>(x, qf, a.k2, lane, st);
      if (nx >= te) break;
      it = nx;
      nx += kAttnWaves;
      if (nx < te) attn_load<NG>(a, h, nx, id, start, end, n, c, x);
      id1 = attn_pages(a, b, min(nx + kAttnWaves, te - 1), n, c);
      __builtin_amdgcn_sched_barrier(0);
      attn_tile<T, NG>(y, qf, a.k2, lane, st);
      if (nx >= te) break;
      it = nx;
    }
  }

  // join the waves
  st.sum = quarters_sum(st.sum, lane);
  if (c == 0) {
    sh_ref[wave][n] = st.ref;
    sh_sum[wave][n] = st.sum;
  }
#pragma unroll
  for (int m = 0; m < 2 * NG; ++m)
    *reinterpret_cast<f32x4*>(sh_acc + (wave * 16 + n) * (D + 4) + 16 * m + 4 * c) = st.acc[m];
  __syncthreads();
  const size_t unit = (size_t)b * gridDim.y + blockIdx.y;
  const size_t run = (size_t)a.HG * (D + 4);                   // one run's part: [HG][D] and [HG] (ref, sum)
  float* part = a.parts + (unit * a.S + split) * run;
  for (int e = threadIdx.x; e < heads * (D / 2); e += kThreads) {
    const int hd = e / (D / 2), d = 2 * (e % (D / 2));
    float r = sh_ref[0][hd];
#pragma unroll
    for (int w = 1; w < kAttnWaves; ++w) r = fmaxf(r, sh_ref[w][hd]);
    float v0 = 0.f, v1 = 0.f, l = 0.f;
#pragma unroll
    for (int w = 0; w < kAttnWaves; ++w) {
      const float f = exp2f(sh_ref[w][hd] - r);
      const float* p = sh_acc + (w * 16 + hd) * (D + 4) + d;
      v0 = fmaf(f, p[0], v0);
      v1 = fmaf(f, p[1], v1);
      l = fmaf(f, sh_sum[w][hd], l);
    }
    if (active == 1) {
      const size_t o = (size_t)b * a.Hq + hq0 + hd;
      const float inv = l != 0.f ? 1.0f / l : 0.f;
      ((uint32_t*)a.out)[(o * D + d) >> 1] = (uint32_t)to_16(T{}, v0 * inv) | ((uint32_t)to_16(T{}, v1 * inv) << 16);
      if (a.lse && d == 0) a.lse[o] = attn_lse(r, l);
    } else {
      store_through2(part + hd * D + d, v0, v1);
      if (d == 0) store_through2(part + a.HG * D + 2 * hd, r, l);
    }
  }
  if (active == 1) return;
  // the last workgroup of the unit joins the runs, in their order
  wait_memory();
  __syncthreads();
  if (threadIdx.x == 0) sh_last = take_ticket(a.tickets + unit) == (uint32_t)(active - 1) ? 1u : 0u;
  __syncthreads();
  if (!sh_last) return;
  acquire_agent();
  part = a.parts + unit * a.S * run;
  // `items` threads hold 4 dims of a head each; where there are fewer items than threads
  // the runs are dealt out over groups of threads and their sums added in group order
  const int items = heads * (D / 4);
  const int ngroup = max(1, min(kThreads / items, kAttnWaves));
  for (int e0 = 0; e0 < items; e0 += kThreads) {
    const int grp = ngroup > 1 ? threadIdx.x / items : 0;
    const int e = ngroup > 1 ? threadIdx.x % items : e0 + threadIdx.x;
    const bool mine = grp < ngroup && e < items;
    const int hd = mine ? e / (D / 4) : 0, d = 4 * (e % (D / 4));
    const float* rs = part + a.HG * D + 2 * hd;
    float r = kRefMin;
    for (int k = 0; k < active; ++k) r = fmaxf(r, rs[k * run]);
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    float l = 0.f;
    if (mine) {
#pragma unroll 8
      for (int k = grp; k < active; k += ngroup) {
        const f32x4 pk = *reinterpret_cast<const f32x4*>(part + k * run + hd * D + d);
        const float f = exp2f(rs[k * run] - r);
        l = fmaf(f, rs[k * run + 1], l);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = fmaf(f, pk[i], v[i]);
      }
    }
    if (ngroup > 1) {
      __syncthreads();
      if (mine) {
        *reinterpret_cast<f32x4*>(sh_acc + (grp * items + e) * 4) = v;
        if (d == 0) sh_acc[kThreads * 4 + grp * 16 + hd] = l;
      }
      __syncthreads();
      if (grp == 0) {
        for (int k = 1; k < ngroup; ++k) {
          const f32x4 o = *reinterpret_cast<const f32x4*>(sh_acc + (k * items + e) * 4);
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] += o[i];
        }
        l = 0.f;
        for (int k = 0; k < ngroup; ++k) l += sh_acc[kThreads * 4 + k * 16 + hd];
      }
    }
    if (mine && grp == 0) {
      const size_t o = (size_t)b * a.Hq + hq0 + hd;
      const float inv = l != 0.f ? 1.0f / l : 0.f;
      uint32_t* dst = (uint32_t*)a.out + ((o * D + d) >> 1);
      dst[0] = (uint32_t)to_16(T{}, v[0] * inv) | ((uint32_t)to_16(T{}, v[1] * inv) << 16);
      dst[1] = (uint32_t)to_16(T{}, v[2] * inv) | ((uint32_t)to_16(T{}, v[3] * inv) << 16);
      if (a.lse && d == 0) a.lse[o] = attn_lse(r, l);
    }
  }
  if (threadIdx.x == 0) store_through(a.tickets + unit, 0u);
}

template <class T>
hipError_t attn_launch(hipStream_t s, const AttnArgs& a) {
  const dim3 grid(a.S, a.kv.Hkv * a.HT, a.kv.B), blk(attn_waves(a.kv.D >> 5) * kWave);
  switch (a.kv.D >> 5) {
    case 1: k_attn_q4<T, 1><<<grid, blk, 0, s>>>(a); break;
    case 2: k_attn_q4<T, 2><<<grid, blk, 0, s>>>(a); break;
    case 3: k_attn_q4<T, 3><<<grid, blk, 0, s>>>(a); break;
    case 4: k_attn_q4<T, 4><<<grid, blk, 0, s>>>(a); break;
    case 5: k_attn_q4<T, 5><<<grid, blk, 0, s>>>(a); break;
    case 6: k_attn_q4<T, 6><<<grid, blk, 0, s>>>(a); break;
    case 7: k_attn_q4<T, 7><<<grid, blk, 0, s>>>(a); break;
    default: k_attn_q4<T, 8><<<grid, blk, 0, s>>>(a); break;
  }
  return hipGetLastError();
}

}  // namespace
}  // namespace sfx
