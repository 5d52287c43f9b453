// Append to and read back from the paged int4 key/value cache.
//
//   k' = R(pos) k,  s = fp16(max |k'| / 7) per 32 dims,  q = clamp(rne(k' / s), -8, 7)
//   v alike without the rotation;  q_out = R(pos) q
//
// R turns pairs of the first `rot` dims by the angles whose cosines and sines the caller's
// fp32 table holds for the position.  The two products and their sum are taken in 64 bits
// (the products are exact there) and rounded once to fp32: a quotient next to a rounding
// border then falls the same way wherever it is computed.  max / 7 and k' / s are
// correctly rounded fp32 quotients.
#include "sfx_kv.hpp"
#include "sfx_launch.hpp"
#include "sfx_q4.hpp"

namespace sfx {
namespace {

template <int DT>
__device__ __forceinline__ float load_elem(const void* p, size_t i) {
  if constexpr (DT == DT_F32) return ((const float*)p)[i];
  else if constexpr (DT == DT_F16) return (float)((const _Float16*)p)[i];
  else return __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16);
}
template <int DT>
__device__ __forceinline__ void store_elem(void* p, size_t i, float v) {
  if constexpr (DT == DT_F32) ((float*)p)[i] = v;
  else if constexpr (DT == DT_F16) ((_Float16*)p)[i] = (_Float16)v;
  else ((__bf16*)p)[i] = (__bf16)v;
}

struct AppendArgs {
  KvCache kv;
  const void *q, *k, *v;
  size_t ldq, ldk, ldv;     // elements between tokens
  const int32_t *pos, *seq;
  const float* cs;          // [max_pos][rot]: cosines, then sines
  void* q_out;
  int T, Hq, rot, max_pos, pairs;
};

// Dim d of a head after the rotation (`head`: the head's first element).
template <int DT>
__device__ __forceinline__ float rotated(const AppendArgs& a, const void* p, size_t head, int d, const float* cs) {
  const float x = load_elem<DT>(p, head + d);
  if (cs == nullptr || d >= a.rot) return x;
  const int half = a.rot >> 1;
  int i, other;
  bool first;
  if (a.pairs) {
    i = d >> 1;
    other = d ^ 1;
    first = (d & 1) == 0;
  } else {
    first = d < half;
    i = first ? d : d - half;
    other = first ? d + half : d - half;
  }
  const double o = (double)load_elem<DT>(p, head + other), co = (double)cs[i], si = (double)cs[half + i];
  const double turn = first ? -(o * si) : o * si;
  // the fp32 value is what is rounded on to 16 bits or quantised: the copy keeps the
  // compiler from converting the 64-bit sum to 16 bits directly
  float y = (float)((double)x * co + turn);
  asm volatile("" : "+v"(y));
  return y;
}

// Scale (fp16 bits) and the codes u = q + 8 of a lane's two values; the 16 lanes of a
// quarter hold one group of 32.  A group with a NaN or an infinity takes a NaN scale;
// `top` is the largest scale.
__device__ __forceinline__ void quant_pair(float a, float b, float top, int lane, uint16_t* s_out, uint32_t* ua,
                                           uint32_t* ub) {
  uint32_t m = max(__float_as_uint(a) & 0x7FFFFFFFu, __float_as_uint(b) & 0x7FFFFFFFu);
  m = max(m, lane_xor_u32<8>(m, lane));
  m = max(m, lane_xor_u32<4>(m, lane));
  m = max(m, lane_xor_u32<2>(m, lane));
  m = max(m, lane_xor_u32<1>(m, lane));
  if (m >= 0x7F800000u) {
    *s_out = 0x7E00;
    *ua = *ub = 8u;
    return;
  }
  const _Float16 s = (_Float16)fminf(__uint_as_float(m) / 7.0f, top);
  const float sf = (float)s;
  const float qa = sf > 0.f ? fminf(fmaxf(rintf(a / sf), -8.f), 7.f) : 0.f;
  const float qb = sf > 0.f ? fminf(fmaxf(rintf(b / sf), -8.f), 7.f) : 0.f;
  *s_out = __builtin_bit_cast(uint16_t, s);
  *ua = (uint32_t)((int)qa + 8);
  *ub = (uint32_t)((int)qb + 8);
}

// Largest scales.  The attention takes V values as fp16 (code times scale), which stay
// finite up to 8 x 8188 = 65504; K scales multiply fp32 sums.
constexpr float kTopK = 65504.f, kTopV = 8188.f;

// One wave per token and head: first the query heads, then the kv heads.
template <int DT, int QDT>
__global__ __launch_bounds__(kBlock) void k_kv_append(AppendArgs a) {
  const int lane = threadIdx.x & (kWave - 1);
  const int t = blockIdx.x;
  const int unit = blockIdx.y * kWavesPerBlock + (threadIdx.x >> 6);
  const int Hkv = a.kv.Hkv, D = a.kv.D, NG = D >> 5;
  if (unit >= a.Hq + Hkv) return;
  const int pos = a.pos[t], b = a.seq ? a.seq[t] : t;
  if (pos < 0 || (unsigned)b >= (unsigned)a.kv.B || (a.cs && pos >= a.max_pos)) return;
  const int id = kv_page(a.kv, b, pos);
  if (id < 0) return;
  const float* cs = a.cs ? a.cs + (size_t)pos * a.rot : nullptr;
  const int n = lane & 15;
  if (unit < a.Hq) {
    const size_t head = (size_t)t * a.ldq + (size_t)unit * D;
    const size_t out = ((size_t)t * a.Hq + unit) * D;
    for (int d = lane; d < D; d += kWave) store_elem<QDT>(a.q_out, out + d, rotated<DT>(a, a.q, head, d, cs));
    return;
  }
  const int h = unit - a.Hq, in_page = pos & ((1 << a.kv.page_shift) - 1), i = in_page & 7;
  uint8_t* blk = a.kv.base + kv_block(a.kv, id, h, in_page >> 3);
  const size_t khead = (size_t)t * a.ldk + (size_t)h * D, vhead = (size_t)t * a.ldv + (size_t)h * D;
  for (int g = lane >> 4; g < NG; g += 4) {
    uint16_t s;
    uint32_t ua, ub;
    const int dk = 32 * g + 2 * n;
    const float k0 = rotated<DT>(a, a.k, khead, dk, cs), k1 = rotated<DT>(a, a.k, khead, dk + 1, cs);
    quant_pair(k0, k1, kTopK, lane, &s, &ua, &ub);
    uint32_t w = (ua << (4 * (n & 3))) | (ub << (16 + 4 * (n & 3)));
    w |= lane_xor_u32<1>(w, lane);
    w |= lane_xor_u32<2>(w, lane);
    if ((n & 3) == 0) *(uint32_t*)(blk + i * (D >> 1) + ((n >> 2) * NG + g) * 4) = w;
    if (n == 0) *(uint16_t*)(blk + 8 * D + g * 16 + i * 2) = s;
    const float v0 = load_elem<DT>(a.v, vhead + 32 * g + n), v1 = load_elem<DT>(a.v, vhead + 32 * g + 16 + n);
    quant_pair(v0, v1, kTopV, lane, &s, &ua, &ub);
    blk[4 * D + n * 8 * NG + g * 8 + kv_byte(i)] = (uint8_t)(ua | (ub << 4));
    if (n == 0) *(uint16_t*)(blk + 8 * D + (D >> 1) + g * 16 + i * 2) = s;
  }
}

struct ReadArgs {
  KvCache kv;
  const int32_t *pos, *seq;
  void *k, *v;              // [T][Hkv][D]
  int T;
};

// One wave per token and kv head.
template <int DT>
__global__ __launch_bounds__(kBlock) void k_kv_read(ReadArgs a) {
  const int lane = threadIdx.x & (kWave - 1);
  const int t = blockIdx.x;
  const int h = blockIdx.y * kWavesPerBlock + (threadIdx.x >> 6);
  const int D = a.kv.D, NG = D >> 5;
  if (h >= a.kv.Hkv) return;
  const int pos = a.pos[t], b = a.seq ? a.seq[t] : t;
  const int id = pos >= 0 && (unsigned)b < (unsigned)a.kv.B ? kv_page(a.kv, b, pos) : -1;
  const int n = lane & 15;
  const size_t out = ((size_t)t * a.kv.Hkv + h) * D;
  const int in_page = max(pos, 0) & ((1 << a.kv.page_shift) - 1), i = in_page & 7;
  const uint8_t* blk = a.kv.base + kv_block(a.kv, max(id, 0), h, in_page >> 3);
  for (int g = lane >> 4; g < NG; g += 4) {
    float k0 = 0.f, k1 = 0.f, v0 = 0.f, v1 = 0.f;
    if (id >= 0) {
      const uint32_t w = *(const uint32_t*)(blk + i * (D >> 1) + ((n >> 2) * NG + g) * 4) >> (4 * (n & 3));
      const float ks = half_at(*(const uint16_t*)(blk + 8 * D + g * 16 + i * 2), 0);
      const float vs = half_at(*(const uint16_t*)(blk + 8 * D + (D >> 1) + g * 16 + i * 2), 0);
      const uint32_t u = blk[4 * D + n * 8 * NG + g * 8 + kv_byte(i)];
      k0 = (float)((int)(w & 15u) - 8) * ks;
      k1 = (float)((int)((w >> 16) & 15u) - 8) * ks;
      v0 = (float)((int)(u & 15u) - 8) * vs;
      v1 = (float)((int)(u >> 4) - 8) * vs;
    }
    store_elem<DT>(a.k, out + 32 * g + 2 * n, k0);
    store_elem<DT>(a.k, out + 32 * g + 2 * n + 1, k1);
    store_elem<DT>(a.v, out + 32 * g + n, v0);
    store_elem<DT>(a.v, out + 32 * g + 16 + n, v1);
  }
}

KvCache make_cache(const KvGeom& g, const void* cache, const int32_t* table) {
  return KvCache{(uint8_t*)cache, table, g.Hkv, g.D, g.page_shift, g.num_pages, g.max_pages, g.B};
}

template <int DT>
void run_append(hipStream_t s, dim3 grid, const AppendArgs& a, int qdt) {
  if (qdt == DT_F16) k_kv_append<DT, DT_F16><<<grid, dim3(kBlock), 0, s>>>(a);
  else k_kv_append<DT, DT_BF16><<<grid, dim3(kBlock), 0, s>>>(a);
}

}  // namespace

hipError_t launch_kv_append_q4(hipStream_t s, const KvGeom& g, int xdt, int qdt, int T, int Hq, const void* q, size_t ldq,
                               const void* k, size_t ldk, const void* v, size_t ldv, const int32_t* pos,
                               const int32_t* seq, const float* cos_sin, int rot, int max_pos, int pairs,
                               const int32_t* table, void* cache, void* q_out) {
  const AppendArgs a{make_cache(g, cache, table), q, k, v, ldq, ldk, ldv, pos, seq, cos_sin, q_out, T, Hq, rot,
                     max_pos, pairs};
  const dim3 grid(T, (Hq + g.Hkv + kWavesPerBlock - 1) / kWavesPerBlock);
  if (xdt == DT_F32) run_append<DT_F32>(s, grid, a, qdt);
  else if (xdt == DT_F16) run_append<DT_F16>(s, grid, a, qdt);
  else run_append<DT_BF16>(s, grid, a, qdt);
  return hipGetLastError();
}

hipError_t launch_kv_read_q4(hipStream_t s, const KvGeom& g, int odt, int T, const int32_t* pos, const int32_t* seq,
                             const int32_t* table, const void* cache, void* k, void* v) {
  const ReadArgs a{make_cache(g, cache, table), pos, seq, k, v, T};
  const dim3 grid(T, (g.Hkv + kWavesPerBlock - 1) / kWavesPerBlock);
  if (odt == DT_F32) k_kv_read<DT_F32><<<grid, dim3(kBlock), 0, s>>>(a);
  else if (odt == DT_F16) k_kv_read<DT_F16><<<grid, dim3(kBlock), 0, s>>>(a);
  else k_kv_read<DT_BF16><<<grid, dim3(kBlock), 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace sfx
