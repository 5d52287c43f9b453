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

constexpr int kAttnWaves = 4;
constexpr int kAttnTile = 32;          // positions a wave takes at a time
constexpr float kRefMin = -3.0e38f;

struct AttnArgs {
  KvCache kv;
  const uint8_t* q;
  size_t ldq;               // bytes between sequences
  const int32_t *starts, *lens;
  uint8_t* out;             // [B][Hq][D] 16 bit
  float* lse;               // [B][Hq] or null
  uint32_t* tickets;        // [B][Hkv][head tiles]
  float* parts;             // [B][Hkv][head tiles][S][HG][D + 2]
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

template <class T, int NG>
__global__ __launch_bounds__(kAttnWaves * kWave) void k_attn_q4(AttnArgs a) {
  constexpr int D = 32 * NG;
  __shared__ float sh_ref[kAttnWaves][16], sh_sum[kAttnWaves][16];
  __shared__ float sh_acc[kAttnWaves][16][D + 1];
  __shared__ uint32_t sh_last;
  const int lane = opaque_lane(), wave = threadIdx.x >> 6;
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
  f32x4 c24[NG];
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    qf[g] = n < heads ? load_raw<16>(a.q + (size_t)b * a.ldq + ((size_t)(hq0 + n) * D + 32 * g + 8 * c) * 2) : zero16();
    c24[g] = Mma<T>::run(q4_minus24<T>(), qf[g], zero);
  }
  float ref = kRefMin, sum = 0.f;
  f32x4 acc[2 * NG];
#pragma unroll
  for (int m = 0; m < 2 * NG; ++m) acc[m] = zero;

  const int page_mask = (1 << a.kv.page_shift) - 1;
  for (int it = tb + wave; it < te; it += kAttnWaves) {
    // K rows: lane n reads position n % 4 (+ 4 in the second product) of octet n / 4;
    // scales, scores and V: octet c
    const int pk = it * kAttnTile + 8 * (n >> 2), pv = it * kAttnTile + 8 * c;
    const int idk = kv_page(a.kv, b, pk), idv = kv_page(a.kv, b, pv);
    const uint8_t* bk = a.kv.base + kv_block(a.kv, max(idk, 0), h, (pk & page_mask) >> 3);
    const uint8_t* bv = a.kv.base + kv_block(a.kv, max(idv, 0), h, (pv & page_mask) >> 3);
    uint32_t kw[2][NG], vw[2 * NG];
    Raw<16> ks[NG], vs[NG];
#pragma unroll
    for (int t = 0; t < 2; ++t) load_words<NG>(bk + (4 * t + (n & 3)) * (D / 2) + c * 4 * NG, kw[t]);
#pragma unroll
    for (int g = 0; g < NG; ++g) ks[g] = load_raw<16>(bv + 8 * D + 16 * g);
    load_words<2 * NG>(bv + 4 * D + n * 8 * NG, vw);
#pragma unroll
    for (int g = 0; g < NG; ++g) vs[g] = load_raw<16>(bv + 8 * D + D / 2 + 16 * g);

    float s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = 0.f;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const f32x4 p = Mma<T>::run(q4_word<T>(kw[t][g]), qf[g], c24[g]);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[4 * t + i] = fmaf(half_at(ks[g].w[2 * t + (i >> 1)], i & 1), p[i], s[4 * t + i]);
      }
    // positions of this lane that count
    uint32_t on = 0xFFu;
    if (idv < 0) on = 0u;
    const int lo = start - pv, hi = end - pv;
    if (lo > 0) on &= lo >= 8 ? 0u : 0xFFu << lo;
    if (hi < 8) on &= hi <= 0 ? 0u : (1u << hi) - 1u;
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      s[i] = (on >> i) & 1u ? s[i] * a.k2 : -INFINITY;
      top = fmaxf(top, s[i]);
    }
    if (__any(top > ref + 6.f)) {
      const float next = fmaxf(quarters_max(top, lane), ref);
      const float f = exp2f(ref - next);
      ref = next;
      sum *= f;
#pragma unroll
      for (int m = 0; m < 2 * NG; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][i] *= f;
    }
    Raw<16> p;
    const float off = 9.f - ref;
    float e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      e[i] = __builtin_amdgcn_exp2f(s[i] + off);
      sum += e[i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) p.w[i] = pack_f16(e[2 * i], e[2 * i + 1]);
    // masked positions: scales to zero, whatever the cache holds there
    uint32_t keep[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      keep[i] = ((on >> (2 * i)) & 1u ? 0xFFFFu : 0u) | ((on >> (2 * i + 1)) & 1u ? 0xFFFF0000u : 0u);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      Raw<16> lo16, hi16;
      const uint32_t w0 = vw[2 * g], w1 = vw[2 * g + 1];
      lo16.w[0] = q4_pair<TF16, 0>(w0);
      hi16.w[0] = q4_pair<TF16, 1>(w0);
      lo16.w[1] = q4_pair<TF16, 2>(w0);
      hi16.w[1] = q4_pair<TF16, 3>(w0);
      lo16.w[2] = q4_pair<TF16, 0>(w1);
      hi16.w[2] = q4_pair<TF16, 1>(w1);
      lo16.w[3] = q4_pair<TF16, 2>(w1);
      hi16.w[3] = q4_pair<TF16, 3>(w1);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t sc = vs[g].w[i] & keep[i];
        lo16.w[i] = pk_mul(pk_add24(lo16.w[i]), sc);
        hi16.w[i] = pk_mul(pk_add24(hi16.w[i]), sc);
      }
      acc[2 * g] = Mma<TF16>::run(lo16, p, acc[2 * g]);
      acc[2 * g + 1] = Mma<TF16>::run(hi16, p, acc[2 * g + 1]);
    }
  }

  // join the waves: rows 4 c + i of product m are dims 16 m + 4 c + i of head n
  sum = quarters_sum(sum, lane);
  if (c == 0) {
    sh_ref[wave][n] = ref;
    sh_sum[wave][n] = sum;
  }
#pragma unroll
  for (int m = 0; m < 2 * NG; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) sh_acc[wave][n][16 * m + 4 * c + i] = acc[m][i];
  __syncthreads();
  const size_t unit = (size_t)b * gridDim.y + blockIdx.y;
  const size_t run = (size_t)a.HG * (D + 2);
  float* part = a.parts + (unit * a.S + split) * run;
  for (int e = threadIdx.x; e < heads * D; e += kAttnWaves * kWave) {
    const int hd = e / D, d = e % D;
    float r = sh_ref[0][hd];
#pragma unroll
    for (int w = 1; w < kAttnWaves; ++w) r = fmaxf(r, sh_ref[w][hd]);
    float v = 0.f, l = 0.f;
#pragma unroll
    for (int w = 0; w < kAttnWaves; ++w) {
      const float f = exp2f(sh_ref[w][hd] - r);
      v = fmaf(f, sh_acc[w][hd][d], v);
      l = fmaf(f, sh_sum[w][hd], l);
    }
    if (active == 1) {
      const size_t o = ((size_t)b * a.Hq + hq0 + hd);
      ((uint16_t*)a.out)[o * D + d] = to_16(T{}, l != 0.f ? v / l : 0.f);
      if (a.lse && d == 0) a.lse[o] = l != 0.f ? (r - 9.f + log2f(l)) * 0.69314718055994531f : -INFINITY;
    } else {
      store_through(part + hd * (D + 2) + d, v);
      if (d == 0) {
        store_through(part + hd * (D + 2) + D, r);
        store_through(part + hd * (D + 2) + D + 1, l);
      }
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
  for (int e = threadIdx.x; e < heads * D; e += kAttnWaves * kWave) {
    const int hd = e / D, d = e % D;
    const float* p = part + hd * (D + 2);
    float r = kRefMin;
    for (int k = 0; k < active; ++k) r = fmaxf(r, p[k * run + D]);
    float v = 0.f, l = 0.f;
    for (int k = 0; k < active; ++k) {
      const float* pk = p + k * run;
      const float f = exp2f(pk[D] - r);
      v = fmaf(f, pk[d], v);
      l = fmaf(f, pk[D + 1], l);
    }
    const size_t o = ((size_t)b * a.Hq + hq0 + hd);
    ((uint16_t*)a.out)[o * D + d] = to_16(T{}, l != 0.f ? v / l : 0.f);
    if (a.lse && d == 0) a.lse[o] = l != 0.f ? (r - 9.f + log2f(l)) * 0.69314718055994531f : -INFINITY;
  }
  if (threadIdx.x == 0) store_through(a.tickets + unit, 0u);
}

template <class T>
hipError_t attn_launch(hipStream_t s, const AttnArgs& a) {
  const dim3 grid(a.S, a.kv.Hkv * a.HT, a.kv.B), blk(kAttnWaves * kWave);
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
