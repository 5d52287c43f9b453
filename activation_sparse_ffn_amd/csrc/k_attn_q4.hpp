// Decode attention over the paged int4 key/value cache: one query token per sequence,
// Hq query heads sharing Hkv kv heads.
//
//   s_p = scale q . k_p,  p in [start, len);  o = sum_p e^(s_p - m) v_p / sum_p e^(s_p - m)
//
// One pass with a running reference and sum.  A wave takes 32 positions at a time:
//   scores   two 16x16x32 products per group of 32 dims, 16 positions (rows) x 16 query
//            heads (columns) each, on the codes (sfx_q4.hpp); the key's fp32 scale multiplies
//            each group's fp32 sum;
//   weights  P = 2^(s - ref + 9) in fp32, as one fp16 operand of the second product (bf16
//            results) or two (fp16 results); the sum of weights keeps the fp32 values.  The
//            lane that holds a score holds it in the place where the product wants the
//            weight, so nothing crosses lanes;
//   output   codes times scale, rounded once to fp16, as rows of 16 dims x 32 positions.
// The reference is raised only when a score passes it by 6 (in powers of two), so P stays
// below 2^15; the 2^9 keeps weights down to 2^-33 of the largest above fp16's last bit.
//
// Bound by reading the cache (D + D / 8 bytes per position and kv head, keys and values
// together); the codes' way into matrix operands is the second load (331 vector operations
// per wave and tile of 32 positions at D = 128, 45% of the time at 131072 positions).  The
// cache is copied into LDS without passing through registers, so a wave holds only what it
// works on and four waves fit a SIMD.  131072 positions x 8 kv heads, step by step: two tiles in
// registers, the last workgroup joining behind a cache invalidation, 66 us; through LDS, joined
// without the invalidation, 45; joined by a kernel of its own, 41 (35.0, 4.3 TB/s, and 4.7).
// 64 sequences of up to 4096 x 8 kv heads of 64: 26 us, with sequences of different lengths paired
// on a compute unit (31 in the caller's order).
#pragma once
#include "sfx_kv.hpp"
#include "sfx_launch.hpp"
#include "sfx_q4.hpp"

namespace sfx {
namespace {

constexpr int kAttnTile = 32;          // positions a wave takes at a time
constexpr int kAttnUnits = 256;        // compute units
constexpr int kAttnOrder = 1024;       // positions of a table from which sequences are ordered
constexpr float kRefMin = -3.0e38f;
// Waves of a workgroup and tiles of LDS per wave: two workgroups fit a compute unit's 160 KB.
// The next tiles are asked for before a tile is waited for.  The counted waits are what a tile
// needs; the compiler adds a wait for all copies into LDS before the tile's first LDS read, so
// as compiled a wave's copies overlap with other waves' work and not with its own.
constexpr int attn_waves(int NG) { return NG <= 4 ? 8 : 4; }
constexpr int attn_slots(int NG) { return NG <= 2 ? 4 : NG == 5 ? 3 : 2; }

struct AttnArgs {
  KvCache kv;
  const uint8_t* q;
  size_t ldq;               // bytes between sequences
  const int32_t *starts, *lens;
  uint8_t* out;             // [B][Hq][D] 16 bit
  float* lse;               // [B][Hq] or null
  float* parts;             // [B][Hkv][head tiles][S] x ([HG][D] sums, [HG][2] reference and weight sum)
  float k2;                 // scale log2(e), times the unit of the decoded codes
  int Hq, G, HT, HG, S;     // HG = heads of a full head tile, min(G, 16)
  int pass;                 // attn_sequence; 0: sequences in their order
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

// ---- the cache's way into LDS.  A tile of 32 positions is NP pieces of the cache, contiguous
// bytes of one page each (1: pages of 32 or more, 2: 16, 4: 8), copied without passing
// through registers.

template <int NG, int NP>
struct AttnPieces {
  static constexpr int chunks = 72 * NG / NP;                  // of 16 bytes, per piece
  static constexpr int loads = (chunks + kWave - 1) / kWave;   // instructions per piece
  static constexpr int count = NP * loads;                     // per tile
};

// Page ids of a wave's next 64 / NP tiles, one piece per lane; tile `it` of the sequence is
// the wave's tile (it - first) / W from lane 0.
template <int NP>
__device__ __forceinline__ int attn_ids(const KvCache& kv, int b, int it, int W, int te, int lane) {
  const int t = min(it + (lane / NP) * W, te - 1);
  return kv_page(kv, b, t * kAttnTile + (lane % NP) * (kAttnTile / NP));
}

template <int NG, int NP>
__device__ __forceinline__ void attn_copy(const KvCache& kv, int h, int it, int ids, int at, uint8_t* dst, int lane) {
  using P = AttnPieces<NG, NP>;
  memory_order();                                              // tiles are waited for in this order
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int pos = it * kAttnTile + p * (kAttnTile / NP);
    const int id = max(__builtin_amdgcn_readlane(ids, at * NP + p), 0);
    const uint32_t blk = ((uint32_t)(id * kv.Hkv + h) << (kv.page_shift - 3)) +
                         (uint32_t)((pos & ((1 << kv.page_shift) - 1)) >> 3);
    const uint8_t* src = kv.base + (size_t)blk * (288 * NG);
#pragma unroll
    for (int j = 0; j < P::loads; ++j) {
      const int left = P::chunks - j * kWave;
      if (left >= kWave || lane < left)
        __builtin_amdgcn_global_load_lds((const void*)(src + (size_t)(uint32_t)((j * kWave + lane) * 16)),
                                         (__attribute__((address_space(3))) void*)(dst + (p * P::chunks + j * kWave) * 16),
                                         16, 0, 0);
    }
  }
}

// Running state of a wave: per lane the head n, of products m the dims 16 m + 4 c + i.
template <int NG>
struct AttnState {
  float ref, sum;           // reference (all quarters alike), sum of this quarter's weights
  f32x4 acc[2 * NG];
};

// One tile, from LDS.  A lane takes K rows of position n % 4 (+ 4) of octet n / 4, words of
// quarter c; V unit n and the scales of octet c.  `on`: bit i says that position i of octet
// c counts (all ones where `full`).
template <class T, int NG>
__device__ __forceinline__ void attn_tile(const uint8_t* tile, const Raw<16> (&qf)[NG], const Q4<T>& kc,
                                          const Q4<TF16>& vc, float k2, bool full, uint32_t on, int lane,
                                          AttnState<NG>& st) {
  constexpr int D = 32 * NG;
  const int n = lane & 15, c = lane >> 4;
  const uint8_t *bk = tile + (n >> 2) * 9 * D, *bv = tile + c * 9 * D;
  uint32_t kw[2][NG], vw[2 * NG];
  Raw<16> ks[NG], vs[NG];
#pragma unroll
  for (int t = 0; t < 2; ++t) load_words<NG>(bk + (4 * t + (n & 3)) * (D / 2) + c * 4 * NG, kw[t]);
#pragma unroll
  for (int g = 0; g < NG; ++g) ks[g] = load_raw<16>(bv + 8 * D + 16 * g);
  float s[8];
  Raw<16> m24;
  if constexpr (Q4<T>::offset) m24 = Q4<T>::minus24();
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    f32x4 from = {0.f, 0.f, 0.f, 0.f};
    if constexpr (Q4<T>::offset) from = Mma<T>::run(m24, qf[g], from);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const f32x4 p = Mma<T>::run(kc.word(kw[t][g]), qf[g], from);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float sc = half_at(ks[g].w[2 * t + (i >> 1)], i & 1);
        s[4 * t + i] = g == 0 ? sc * p[i] : fmaf(sc, p[i], s[4 * t + i]);
      }
    }
  }
  // the values' part is read only now: its registers are the scores' until here
  __builtin_amdgcn_sched_barrier(0);
  load_words<2 * NG>(bv + 4 * D + n * 8 * NG, vw);
#pragma unroll
  for (int g = 0; g < NG; ++g) vs[g] = load_raw<16>(bv + 8 * D + D / 2 + 16 * g);
  const float off = 9.f - st.ref;
  float e[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) e[i] = fmaf(s[i], k2, off);
  if (!full) {
    // some position does not count: its weight is 0 and so is its value, whatever is held there
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (!((on >> i) & 1u)) e[i] = -INFINITY;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t keep = ((on >> (2 * i)) & 1u ? 0xFFFFu : 0u) | ((on >> (2 * i + 1)) & 1u ? 0xFFFF0000u : 0u);
#pragma unroll
      for (int g = 0; g < NG; ++g) vs[g].w[i] &= keep;
    }
  }
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = fmaxf(top, e[i]);
  if (__any(top > 15.f)) {
    // raise the reference to the largest score so far
    float most = -INFINITY;
#pragma unroll
    for (int i = 0; i < 8; ++i) most = fmaxf(most, e[i] == -INFINITY ? e[i] : s[i] * k2);
    const float next = fmaxf(quarters_max(most, lane), st.ref);
    const float f = exp2f(st.ref - next);
    st.ref = next;
    st.sum *= f;
#pragma unroll
    for (int m = 0; m < 2 * NG; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) st.acc[m][i] *= f;
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = e[i] == -INFINITY ? e[i] : fmaf(s[i], k2, 9.f - next);
  }
  // fp16 queries get results of 11 bits: their weights' rounding errors are kept as a second
  // fp16 term (products the matrix cores have time for), else they would add half of the
  // result's own rounding to it; bf16 results have 8 bits
  constexpr bool kTwo = !Q4<T>::offset;
  Raw<16> p, p2;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float e0 = __builtin_amdgcn_exp2f(e[2 * i]), e1 = __builtin_amdgcn_exp2f(e[2 * i + 1]);
    st.sum += e0 + e1;
    p.w[i] = pack_f16(e0, e1);
    if constexpr (kTwo) p2.w[i] = pack_f16(e0 - half_at(p.w[i], 0), e1 - half_at(p.w[i], 1));
  }
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    Raw<16> lo, hi;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const Raw<16> u = vc.word(vw[2 * g + j]);               // (dim n, dim n + 16) of positions 4 j + (0 1), (2 3)
      lo.w[2 * j] = pk_mul(u.w[0], vs[g].w[2 * j]);
      hi.w[2 * j] = pk_mul(u.w[1], vs[g].w[2 * j]);
      lo.w[2 * j + 1] = pk_mul(u.w[2], vs[g].w[2 * j + 1]);
      hi.w[2 * j + 1] = pk_mul(u.w[3], vs[g].w[2 * j + 1]);
    }
    st.acc[2 * g] = Mma<TF16>::run(lo, p, st.acc[2 * g]);
    st.acc[2 * g + 1] = Mma<TF16>::run(hi, p, st.acc[2 * g + 1]);
    if constexpr (kTwo) {
      st.acc[2 * g] = Mma<TF16>::run(lo, p2, st.acc[2 * g]);
      st.acc[2 * g + 1] = Mma<TF16>::run(hi, p2, st.acc[2 * g + 1]);
    }
  }
}

__device__ __forceinline__ float attn_lse(float ref, float sum) {
  return sum != 0.f ? (ref - 9.f + log2f(sum)) * 0.69314718055994531f : -INFINITY;
}

// A sequence's positions [start, end) as tiles t0 .. t0 + ntile - 1, cut into `active` runs of
// `per` tiles: S even runs, but none shorter than a tile per wave.
struct AttnSpan {
  int start, end, t0, ntile, per, active;
};
__device__ __forceinline__ int attn_start(const AttnArgs& a, int b) { return a.starts ? max(a.starts[b], 0) : 0; }
__device__ __forceinline__ int attn_end(const AttnArgs& a, int b) {
  return min(a.lens[b], a.kv.max_pages << a.kv.page_shift);
}
__device__ __forceinline__ AttnSpan attn_span(const AttnArgs& a, int start, int end, int W) {
  AttnSpan s;
  s.end = end;
  s.start = start;
  s.t0 = s.start / kAttnTile;
  s.ntile = s.end > s.start ? (s.end + kAttnTile - 1) / kAttnTile - s.t0 : 0;
  s.per = max(W, (s.ntile + a.S - 1) / a.S);
  s.active = max(1, (s.ntile + s.per - 1) / s.per);            // an empty sequence has one: its zero row
  return s;
}

// The sequence that launch position z works on, and its span.  Workgroups are handed out in
// order, so with two to a compute unit positions z and z + pass share one: the first `pass`
// positions take the longest sequences, longest first, the others the rest, shortest first.
// Ranks by counting (equal lengths by index); at most 64 sequences, one to a lane, each wave
// counting a share of them.  Lengths spread evenly up to 4096, 64 sequences x 8 kv heads of
// 64: 31.3 us in their order, 27.6 so; up to 2048 of 128: 26.3 and 22.8.  It costs 0.5 us: all
// 64 of 1500 positions 30.1 and 30.7; up to 600 positions 11.8 and 11.6, up to 300 8.8 and 9.7.
// Behind more than 512 workgroups the next one starts where one has ended, and the order
// gains nothing (1024: 19.2 in their order, 21.5 so).
template <int W>
__device__ __forceinline__ int attn_sequence(const AttnArgs& a, uint8_t (&count)[W][kWave], int wave, int lane,
                                             int& start, int& end) {
  const int B = a.kv.B, z = blockIdx.z;
  if (a.pass == 0) {
    start = attn_start(a, z);
    end = attn_end(a, z);
    return z;
  }
  const int from = lane < B ? attn_start(a, lane) : 0, to = lane < B ? attn_end(a, lane) : 0;
  const int len = lane >= B ? -1 : to > from ? to - from : 0;
  int more = 0;
#pragma unroll
  for (int i = 0; i < kWave / W; ++i) {
    const int j = wave * (kWave / W) + i, other = __builtin_amdgcn_readlane(len, j);
    more += other > len || (other == len && j < lane);
  }
  count[wave][lane] = (uint8_t)more;
  __syncthreads();
  int rank = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) rank += count[w][lane];
  const int want = z < a.pass ? z : B - 1 - (z - a.pass);
  const int b = __builtin_ctzll(__ballot(rank == want));       // ranks are 0..63, each once
  start = __builtin_amdgcn_readlane(from, b);
  end = __builtin_amdgcn_readlane(to, b);
  return b;
}

// The tiles of one wave: tb + wave, then every W-th.
template <class T, int NG, int NP>
__device__ __forceinline__ void attn_wave(const AttnArgs& a, int b, int h, int it, int te, int start, int end, int lane,
                                          uint8_t* ring, const Raw<16> (&qf)[NG], AttnState<NG>& st) {
  constexpr int W = attn_waves(NG), SL = attn_slots(NG), bytes = kAttnTile / 8 * 288 * NG;
  constexpr int kCount = AttnPieces<NG, NP>::count, kHold = kWave / NP;   // loads per tile, tiles per look-up
  const int c = lane >> 4;
  const int todo = (te - it + W - 1) / W;
  const Q4<T> kc;
  const Q4<TF16> vc;
  int ids = attn_ids<NP>(a.kv, b, it, W, te, lane);
#pragma unroll
  for (int i = 0; i < SL - 1; ++i)
    if (i < todo) attn_copy<NG, NP>(a.kv, h, it + i * W, ids, i, ring + i * bytes, lane);
  // tile i + SL - 1 is asked for before tile i is worked on, into the slot tile i - 1 has left
  int slot = 0, next = SL - 1, base = 0;                       // ids hold tiles base .. base + kHold - 1
  int ids0 = ids, base0 = 0;                                   // the look-up that tile i came from
  for (int i = 0; i < todo; ++i) {
    const int ahead = i + SL - 1;
    if (ahead < todo) {
      if (ahead - base == kHold) {
        base = ahead;
        ids = attn_ids<NP>(a.kv, b, it + ahead * W, W, te, lane);
      }
      wait_lds();
      attn_copy<NG, NP>(a.kv, h, it + ahead * W, ids, ahead - base, ring + next * bytes, lane);
      wait_vm<(SL - 1) * kCount>();
    } else {
      wait_vm<0>();
    }
    if (i - base0 == kHold) {
      base0 = base;
      ids0 = ids;
    }
    const int pos = (it + i * W) * kAttnTile;
    bool full = pos >= start && pos + kAttnTile <= end;
#pragma unroll
    for (int p = 0; p < NP; ++p) full = full && __builtin_amdgcn_readlane(ids0, (i - base0) * NP + p) >= 0;
    uint32_t on = 0xFFu;
    if (!full) {
      const int id = __shfl(ids0, (i - base0) * NP + c * NP / 4);
      const int lo = start - pos - 8 * c, hi = end - pos - 8 * c;
      if (lo > 0) on &= lo >= 8 ? 0u : 0xFFu << lo;
      if (hi < 8) on &= hi <= 0 ? 0u : (1u << hi) - 1u;
      if (id < 0) on = 0u;
    }
    attn_tile<T, NG>(ring + slot * bytes, qf, kc, vc, a.k2, full, on, lane, st);
    slot = slot + 1 == SL ? 0 : slot + 1;
    next = next + 1 == SL ? 0 : next + 1;
  }
}

template <class T, int NG>
__global__ __launch_bounds__(attn_waves(NG) * kWave, NG <= 4 ? 4 : 2) void k_attn_q4(AttnArgs a) {
  constexpr int W = attn_waves(NG), D = 32 * NG, kThreads = W * kWave;
  constexpr int kRing = W * attn_slots(NG) * (kAttnTile / 8) * 9 * D, kJoin = W * 16 * (D + 4) * 4;
  __shared__ float sh_ref[W][16], sh_sum[W][16];
  __shared__ uint8_t sh_count[W][kWave];
  __shared__ __attribute__((aligned(16))) uint8_t sh_mem[kRing > kJoin ? kRing : kJoin];
  float* sh_acc = (float*)sh_mem;
  const int lane = opaque_lane(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, c = lane >> 4;
  const int split = blockIdx.x, ht = blockIdx.y % a.HT, h = blockIdx.y / a.HT;
  const int heads = min(16, a.G - 16 * ht);                    // query heads of this workgroup
  int start, end;
  const int b = attn_sequence<W>(a, sh_count, wave, lane, start, end);
  const AttnSpan sp = attn_span(a, start, end, W);
  const int active = sp.active;
  if (split >= active) return;
  const int tb = sp.t0 + split * sp.per, te = min(sp.t0 + sp.ntile, tb + sp.per);

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
  uint8_t* ring = sh_mem + wave * (kRing / W);
  if (tb + wave < te) {
    if (a.kv.page_shift >= 5) attn_wave<T, NG, 1>(a, b, h, tb + wave, te, sp.start, sp.end, lane, ring, qf, st);
    else if (a.kv.page_shift == 4) attn_wave<T, NG, 2>(a, b, h, tb + wave, te, sp.start, sp.end, lane, ring, qf, st);
    else attn_wave<T, NG, 4>(a, b, h, tb + wave, te, sp.start, sp.end, lane, ring, qf, st);
  }

  __syncthreads();                                             // the rings become the join's memory
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
  const size_t run = (size_t)a.HG * (D + 4);
  float* part = a.parts + (((size_t)b * gridDim.y + blockIdx.y) * a.S + split) * run;
  for (int e = threadIdx.x; e < heads * (D / 2); e += kThreads) {
    const int hd = e / (D / 2), d = 2 * (e % (D / 2));
    float r = sh_ref[0][hd];
#pragma unroll
    for (int w = 1; w < W; ++w) r = fmaxf(r, sh_ref[w][hd]);
    float v0 = 0.f, v1 = 0.f, l = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
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
      *reinterpret_cast<float2*>(part + hd * D + d) = make_float2(v0, v1);
      if (d == 0) *reinterpret_cast<float2*>(part + a.HG * D + 2 * hd) = make_float2(r, l);
    }
  }
}

// Joins the runs of a sequence, one workgroup per query head.  Four dims to a thread; the
// runs are dealt out over groups of D / 4 threads and the groups' sums added in order.
template <class T, int NG>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs a) {
  constexpr int W = attn_waves(NG), D = 32 * NG, kItems = D / 4, kGroups = 256 / kItems;
  __shared__ __attribute__((aligned(16))) float sh_v[kGroups][D];
  __shared__ float sh_l[kGroups], sh_r[kGroups];
  const AttnSpan sp = attn_span(a, attn_start(a, blockIdx.y), attn_end(a, blockIdx.y), W);
  if (sp.active == 1) return;                                   // the attention kernel wrote the row
  const int hq = blockIdx.x, h = hq / a.G, ht = (hq % a.G) / 16, hd = (hq % a.G) % 16, b = blockIdx.y;
  const size_t run = (size_t)a.HG * (D + 4);
  const float* part = a.parts + ((size_t)b * (a.kv.Hkv * a.HT) + h * a.HT + ht) * a.S * run;
  const float* rs = part + a.HG * D + 2 * hd;
  const int grp = threadIdx.x / kItems, d = 4 * (threadIdx.x % kItems);
  float r = kRefMin;
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  float l = 0.f;
  if (grp < kGroups) {
    // one pass: the group's reference goes up with its runs
#pragma unroll 4
    for (int k = grp; k < sp.active; k += kGroups) {
      const f32x4 pk = *reinterpret_cast<const f32x4*>(part + k * run + hd * D + d);
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
    const size_t o = (size_t)b * a.Hq + hq;
    const float inv = l != 0.f ? 1.0f / l : 0.f;
    uint32_t* dst = (uint32_t*)a.out + ((o * D + d) >> 1);
    dst[0] = (uint32_t)to_16(T{}, v[0] * inv) | ((uint32_t)to_16(T{}, v[1] * inv) << 16);
    dst[1] = (uint32_t)to_16(T{}, v[2] * inv) | ((uint32_t)to_16(T{}, v[3] * inv) << 16);
    if (a.lse && d == 0) a.lse[o] = attn_lse(r, l);
  }
}

template <class T, int NG>
hipError_t attn_run(hipStream_t s, AttnArgs a) {
  const int each = a.S * a.kv.Hkv * a.HT, all = each * a.kv.B;  // workgroups of a sequence, of the call
  const bool order = all > kAttnUnits && all <= 2 * kAttnUnits && a.kv.max_pages << a.kv.page_shift >= kAttnOrder;
  a.pass = order ? kAttnUnits / each : 0;
  k_attn_q4<T, NG><<<dim3(a.S, a.kv.Hkv * a.HT, a.kv.B), dim3(attn_waves(NG) * kWave), 0, s>>>(a);
  if (a.S > 1) k_attn_join<T, NG><<<dim3(a.Hq, a.kv.B), dim3(256), 0, s>>>(a);
  return hipGetLastError();
}

template <class T>
hipError_t attn_launch(hipStream_t s, AttnArgs a) {
  a.k2 *= Q4<T>::unit;
  switch (a.kv.D >> 5) {
    case 1: return attn_run<T, 1>(s, a);
    case 2: return attn_run<T, 2>(s, a);
    case 3: return attn_run<T, 3>(s, a);
    case 4: return attn_run<T, 4>(s, a);
    case 5: return attn_run<T, 5>(s, a);
    case 6: return attn_run<T, 6>(s, a);
    case 7: return attn_run<T, 7>(s, a);
    default: return attn_run<T, 8>(s, a);
  }
}

}  // namespace
}  // namespace sfx
