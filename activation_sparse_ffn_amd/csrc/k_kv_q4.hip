// Append to and read back from the paged int4 key/value cache.
//
//   k' = R(pos) k,  s = fp16(max |k'| / 7) per 32 dims,  q = clamp(rne(k' / s), -8, 7)
//   v alike without the rotation;  q_out = R(pos) q
//
// The rotation is that of sfx_turn.hpp; max / 7 and k' / s are correctly rounded fp32 quotients.
//
// Both move mostly the 16- or 32-bit rows they read or write; of a thread's 28 vector loads in a
// bf16 prompt's append 16 are 4-byte loads of the angle table.  Measured (one MI355X): 4095
// tokens of 64 query and 8 kv heads of 128, bf16: append 45 us for 155 MB, of which the 64-bit
// rotation costs 2.4; one head per wave and token, each lane two dims, took 107, bound by the
// chain from position to page to data.  Reading 16384 positions of 8 heads of 128 back: 19 us
// for 86 MB (34 with a wave per head and token).  Eight tokens: 4.2 and 2.2 us, launch latency.
#include <algorithm>

#include "sfx_kv.hpp"
#include "sfx_launch.hpp"
#include "sfx_turn.hpp"

namespace sfx {
namespace {

struct AppendArgs : Rotation {
  KvCache kv;
  const void *q, *k, *v;
  size_t ldq, ldk, ldv;     // elements between tokens
  const int32_t *pos, *seq;
  void* q_out;
  int T, Hq;
};

// Scale (fp16 bits) and the codes u = q + 8, one per nibble of the result in element order;
// the 4 lanes of a quad hold one group of 32.  A group with a NaN or an infinity takes a NaN
// scale; `top` is the largest scale.
__device__ __forceinline__ uint32_t quant8(const float (&x)[8], float top, int lane, uint16_t* s_out) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(x[j]) & 0x7FFFFFFFu);
  m = max(m, lane_xor_u32<2>(m, lane));
  m = max(m, lane_xor_u32<1>(m, lane));
  if (m >= 0x7F800000u) {
    *s_out = 0x7E00;
    return 0x88888888u;
  }
  const _Float16 s = (_Float16)fminf(__uint_as_float(m) / 7.0f, top);
  const float sf = (float)s;
  *s_out = __builtin_bit_cast(uint16_t, s);
  if (!(sf > 0.f)) return 0x88888888u;
  uint32_t u = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) u |= (uint32_t)((int)fminf(fmaxf(rintf(x[j] / sf), -8.f), 7.f) + 8) << (4 * j);
  return u;
}

// Largest scales.  The attention takes V values as fp16 (code times scale), which stay
// finite up to 8 x 8188 = 65504; K scales multiply fp32 sums.
constexpr float kTopK = 65504.f, kTopV = 8188.f;

// A thread takes 8 dims of HP heads of one token, queries or keys and values by the
// workgroup's column: all its loads go out before the position is looked up.
template <int DT, int QDT, bool VEC, int HP>
__global__ __launch_bounds__(kBlock) void k_kv_append(AppendArgs a, int qcols) {
  const int D = a.kv.D, NG = D >> 5, slices = D >> 3, heads = kBlock / slices;
  const int mine = threadIdx.x / slices, slice = threadIdx.x - mine * slices;
  // workgroups 8 apart are on one XCD: the eight tokens of a block of positions are, so its
  // bytes meet in one cache
  const int blk = blockIdx.x, t = ((blk >> 6) * 8 + (blk & 7)) * 8 + ((blk >> 3) & 7);
  if (t >= a.T || mine >= heads) return;
  const int lane = threadIdx.x & (kWave - 1), d0 = 8 * slice, c = slice & 3, g = slice >> 2;
  const bool query = (int)blockIdx.y < qcols;
  const int unit0 = (query ? blockIdx.y : blockIdx.y - qcols) * heads * HP + mine, units = query ? a.Hq : a.kv.Hkv;
  if (unit0 >= units) return;
  const void* src = query ? a.q : a.k;
  const size_t row = (size_t)t * (query ? a.ldq : a.ldk);
  const bool apart = VEC && turn_apart(a, d0);
  Eight<DT> own[HP], oth[HP], val[HP];
#pragma unroll
  for (int k = 0; k < HP; ++k) {
    const size_t head = (size_t)min(unit0 + k * heads, units - 1) * D;
    own[k] = load8<DT, VEC>(src, row + head + d0);
    if (apart) oth[k] = load8<DT, VEC>(src, row + head + turn_other(a, d0));
    if (!query) val[k] = load8<DT, VEC>(a.v, (size_t)t * a.ldv + head + d0);
  }
  const int pos = a.pos[t], b = a.seq ? a.seq[t] : t;
  if (pos < 0 || (unsigned)b >= (unsigned)a.kv.B || (a.cs && pos >= a.max_pos)) return;
  const int id = kv_page(a.kv, b, pos);
  Turn turn;
  if (a.cs && d0 < a.rot) load_turn(a, a.cs + (size_t)pos * a.rot, d0, turn);
  if (id < 0) return;
  const int in_page = pos & ((1 << a.kv.page_shift) - 1), i = in_page & 7;
#pragma unroll
  for (int k = 0; k < HP; ++k) {
    const int unit = unit0 + k * heads;
    if (unit >= units) break;
    float y[8];
    turn8<DT, VEC>(a, src, row + (size_t)unit * D, d0, own[k], oth[k], turn, y);
    if (query) {
      const size_t out = ((size_t)t * a.Hq + unit) * D + d0;
      if constexpr (VEC) {
        store8<QDT>(a.q_out, out, y);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) store_elem<QDT>(a.q_out, out + j, y[j]);
      }
      continue;
    }
    uint8_t* at = a.kv.base + kv_block(a.kv, id, unit, in_page >> 3);
    uint16_t s;
    uint32_t u = quant8(y, kTopK, lane, &s);
    // dims 2 j and 2 j + 1 to nibbles j and j + 4
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) w |= ((u >> (8 * j)) & 15u) << (4 * j) | ((u >> (8 * j + 4)) & 15u) << (16 + 4 * j);
    *(uint32_t*)(at + i * (D >> 1) + (c * NG + g) * 4) = w;
    if (c == 0) *(uint16_t*)(at + 8 * D + g * 16 + i * 2) = s;
    float v[8];
    widen<DT>(val[k], v);
    u = quant8(v, kTopV, lane, &s);
    // dims n and 16 + n share a byte: the quad's lanes c and c + 2 hold them, each writes half
    const uint32_t other = lane_xor_u32<2>(u, lane);
    const uint32_t lo = (c & 2) ? other >> 16 : u & 0xFFFFu, hi = (c & 2) ? u >> 16 : other & 0xFFFFu;
    const int n0 = 8 * (c & 1) + ((c & 2) ? 4 : 0);
    uint8_t* bv = at + 4 * D + g * 8 + kv_byte(i);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      bv[(n0 + j) * 8 * NG] = (uint8_t)(((lo >> (4 * j)) & 15u) | (((hi >> (4 * j)) & 15u) << 4));
    if (c == 0) *(uint16_t*)(at + 8 * D + (D >> 1) + g * 16 + i * 2) = s;
  }
}

struct ReadArgs {
  KvCache kv;
  const int32_t *pos, *seq;
  void *k, *v;              // [T][Hkv][D]
  int T;
};

// A thread takes 8 dims of HP heads of one token; tokens on XCDs as in the append.
template <int DT, int HP>
__global__ __launch_bounds__(kBlock) void k_kv_read(ReadArgs a) {
  const int D = a.kv.D, NG = D >> 5, slices = D >> 3, heads = kBlock / slices;
  const int mine = threadIdx.x / slices, slice = threadIdx.x - mine * slices;
  const int blk = blockIdx.x, t = ((blk >> 6) * 8 + (blk & 7)) * 8 + ((blk >> 3) & 7);
  if (t >= a.T || mine >= heads) return;
  const int h0 = blockIdx.y * heads * HP + mine;
  if (h0 >= a.kv.Hkv) return;
  const int lane = threadIdx.x & (kWave - 1), d0 = 8 * slice, c = slice & 3, g = slice >> 2;
  const int pos = a.pos[t], b = a.seq ? a.seq[t] : t;
  const int id = pos >= 0 && (unsigned)b < (unsigned)a.kv.B ? kv_page(a.kv, b, pos) : -1;
  const int in_page = max(pos, 0) & ((1 << a.kv.page_shift) - 1), i = in_page & 7;
  uint32_t w[HP], u[HP][4];
  uint16_t ks[HP], vs[HP];
#pragma unroll
  for (int k = 0; k < HP; ++k) {
    const uint8_t* at = a.kv.base + kv_block(a.kv, max(id, 0), min(h0 + k * heads, a.kv.Hkv - 1), in_page >> 3);
    w[k] = *(const uint32_t*)(at + i * (D >> 1) + (c * NG + g) * 4);
    ks[k] = *(const uint16_t*)(at + 8 * D + g * 16 + i * 2);
    vs[k] = *(const uint16_t*)(at + 8 * D + (D >> 1) + g * 16 + i * 2);
    // the bytes of dims n and 16 + n, n = 8 (c & 1) + 0..7, serve lanes c and c + 2: each
    // loads four of them
    const uint8_t* bv = at + 4 * D + (8 * (c & 1) + 2 * (c & 2)) * 8 * NG + g * 8 + kv_byte(i);
#pragma unroll
    for (int j = 0; j < 4; ++j) u[k][j] = bv[j * 8 * NG];
  }
#pragma unroll
  for (int k = 0; k < HP; ++k) {
    const int h = h0 + k * heads;
    if (h >= a.kv.Hkv) break;
    // a padding token's values are zero whatever was read
    const float ksf = half_at(ks[k], 0), vsf = half_at(vs[k], 0);
    const uint32_t own = u[k][0] | u[k][1] << 8 | u[k][2] << 16 | u[k][3] << 24, oth = lane_xor_u32<2>(own, lane);
    const int nib = c & 2 ? 4 : 0;
    const uint32_t v0 = (c & 2 ? oth : own) >> nib, v1 = (c & 2 ? own : oth) >> nib;
    float kf[8], vf[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int ku = (int)((w[k] >> (4 * ((j >> 1) + 4 * (j & 1)))) & 15u);
      const int vu = (int)(((j < 4 ? v0 : v1) >> (8 * (j & 3))) & 15u);
      kf[j] = id >= 0 ? (float)(ku - 8) * ksf : 0.f;
      vf[j] = id >= 0 ? (float)(vu - 8) * vsf : 0.f;
    }
    const size_t out = ((size_t)t * a.kv.Hkv + h) * D + d0;
    store8<DT>(a.k, out, kf);
    store8<DT>(a.v, out, vf);
  }
}

// Lengths that a decode step's attention covers, one sequence per thread.
__global__ __launch_bounds__(kBlock) void k_kv_lens(KvCache kv, const int32_t* pos, int max_pos, int window, int32_t* lens,
                                                    int32_t* starts) {
  const int b = blockIdx.x * kBlock + threadIdx.x;
  if (b >= kv.B) return;
  const int p = pos[b];
  // stored by the append: the same conditions
  const bool stored = p >= 0 && (max_pos == 0 || p < max_pos) && kv_page(kv, b, p) >= 0;
  const int n = stored ? p + 1 : 0;
  lens[b] = n;
  if (starts) starts[b] = max(n - window, 0);
}

KvCache make_cache(const KvGeom& g, const void* cache, const int32_t* table) {
  return KvCache{(uint8_t*)cache, table, g.Hkv, g.D, g.page_shift, g.num_pages, g.max_pages, g.B};
}

// Workgroups in x: the mapping to tokens permutes each 64 of them and leaves the last of the 64
// in its place, so the one that would be workgroup kKvMaxTokens stands for no token of a call.
int token_groups(int T) { return std::min((T + 63) / 64 * 64, kKvMaxTokens); }

template <int DT, int QDT, bool VEC>
void run_append(hipStream_t s, const AppendArgs& a) {
  const int heads = kBlock / (a.kv.D >> 3);
  const auto columns = [&](int hp, int n) { return (n + heads * hp - 1) / (heads * hp); };
  const int tokens = token_groups(a.T);
  // four heads to a thread where that leaves four workgroups per compute unit
  if ((long long)a.T * (columns(4, a.Hq) + columns(4, a.kv.Hkv)) >= 1024) {
    const int qc = columns(4, a.Hq);
    k_kv_append<DT, QDT, VEC, 4><<<dim3(tokens, qc + columns(4, a.kv.Hkv)), dim3(kBlock), 0, s>>>(a, qc);
  } else {
    const int qc = columns(1, a.Hq);
    k_kv_append<DT, QDT, VEC, 1><<<dim3(tokens, qc + columns(1, a.kv.Hkv)), dim3(kBlock), 0, s>>>(a, qc);
  }
}
template <int DT>
void run_append(hipStream_t s, const AppendArgs& a, int qdt, bool vec) {
  if (qdt == DT_F16) vec ? run_append<DT, DT_F16, true>(s, a) : run_append<DT, DT_F16, false>(s, a);
  else vec ? run_append<DT, DT_BF16, true>(s, a) : run_append<DT, DT_BF16, false>(s, a);
}

template <int DT>
void run_read(hipStream_t s, const ReadArgs& a) {
  const int heads = kBlock / (a.kv.D >> 3), tokens = token_groups(a.T);
  const auto columns = [&](int hp) { return (a.kv.Hkv + heads * hp - 1) / (heads * hp); };
  if (a.kv.Hkv >= 2 * heads && (long long)a.T * columns(2) >= 1024)
    k_kv_read<DT, 2><<<dim3(tokens, columns(2)), dim3(kBlock), 0, s>>>(a);
  else
    k_kv_read<DT, 1><<<dim3(tokens, columns(1)), dim3(kBlock), 0, s>>>(a);
}

}  // namespace

hipError_t launch_kv_append_q4(hipStream_t s, const KvGeom& g, int xdt, int qdt, int T, int Hq, const void* q, size_t ldq,
                               const void* k, size_t ldk, const void* v, size_t ldv, const int32_t* pos,
                               const int32_t* seq, const float* cos_sin, int rot, int max_pos, int pairs,
                               const int32_t* table, void* cache, void* q_out) {
  const AppendArgs a{{cos_sin, rot, max_pos, pairs}, make_cache(g, cache, table), q, k, v, ldq, ldk, ldv, pos, seq,
                     q_out, T, Hq};
  const uintptr_t row = xdt == DT_F32 ? 4 : 8;                  // elements of 16 bytes
  const bool vec = (((uintptr_t)q | (uintptr_t)k | (uintptr_t)v | (uintptr_t)q_out) & 15u) == 0 &&
                   ((ldq | ldk | ldv) & (row - 1)) == 0 && (!cos_sin || (pairs ? rot % 8 == 0 : rot % 16 == 0));
  if (xdt == DT_F32) run_append<DT_F32>(s, a, qdt, vec);
  else if (xdt == DT_F16) run_append<DT_F16>(s, a, qdt, vec);
  else run_append<DT_BF16>(s, a, qdt, vec);
  return hipGetLastError();
}

hipError_t launch_kv_lens_q4(hipStream_t s, const KvGeom& g, const int32_t* pos, int max_pos, int window,
                             const int32_t* table, int32_t* lens, int32_t* starts) {
  k_kv_lens<<<dim3((g.B + kBlock - 1) / kBlock), dim3(kBlock), 0, s>>>(make_cache(g, nullptr, table), pos, max_pos, window,
                                                                       lens, starts);
  return hipGetLastError();
}

hipError_t launch_kv_read_q4(hipStream_t s, const KvGeom& g, int odt, int T, const int32_t* pos, const int32_t* seq,
                             const int32_t* table, const void* cache, void* k, void* v) {
  const ReadArgs a{make_cache(g, cache, table), pos, seq, k, v, T};
  if (odt == DT_F32) run_read<DT_F32>(s, a);
  else if (odt == DT_F16) run_read<DT_F16>(s, a);
  else run_read<DT_BF16>(s, a);
  return hipGetLastError();
}

}  // namespace sfx
