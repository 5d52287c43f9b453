// Append to and read back from the paged int8 key/value cache.
//
//   k' = R(pos) k;  per block of 16 positions and head: s = max(s of the positions it keeps,
//   max |k'| / 127),  q = rne(k' / s);  where s grows, kept codes become rne(q s_old / s);
//   v alike without the rotation;  q_out = R(pos) q
//
// A quotient is decided by an fp32 product with 1 / s unless that comes to rest within 2^-13 of a
// border, where it is taken in 64 bits: codes are those of the exact quotient.
//
// 4095 tokens of 64 query and 8 kv heads of 128 dims, bf16: 34-40 us (160 MB, 4.0-4.7 TB/s); 8 single tokens of 32
// heads: 6.0 us, offsets, page, rows, scale and kept codes one behind the other.  Where a half of the rotated
// dims is no whole slice of 8, or rows are not aligned, elements are loaded one by one: 40 of 128 dims rotated 53 us (64
// of them 36), 24 of 96 50 (32 of them 34), single tokens 7.0.  Reading 4109 positions of 8 heads back: 8 us (25 MB).
//
// A workgroup takes one block of one head (several heads of fewer than 128 dims): the scale needs
// all of a block's new rows.  Sequences' blocks are numbered one behind the other, so no
// workgroup looks for rows that are not there.
#include <algorithm>

#include "sfx_kv8.hpp"
#include "sfx_launch.hpp"
#include "sfx_turn.hpp"

namespace sfx {
namespace {

struct Append8Args : Rotation {
  KvCache kv;
  Rows8 rows;
  const void *q, *k, *v;
  size_t ldq, ldk, ldv;     // elements between tokens
  void* q_out;
  int Hq, blocks, hgroups;  // bound on blocks of all sequences; workgroups per block
};

// The sequence that block number x of the call belongs to, and which of its blocks it is; b < 0:
// none.  Each wave finds it for itself, 64 sequences at a time.
struct Found {
  int b, j;
  Seq8 s;
};
__device__ __forceinline__ Found find_block(const Append8Args& a, int x, int lane) {
  int before = 0;
  for (int b0 = 0; b0 < a.kv.B; b0 += kWave) {
    const int b = b0 + lane;
    Seq8 s{};
    int nb = 0;
    if (b < a.kv.B) {
      s = rows8_seq(a.rows, b);
      const int n = min(s.n, s.len);
      if (n > 0) nb = (s.len - 1) / kBlk8 - (s.len - n) / kBlk8 + 1;
    }
    const int upto = before + (int)wave_inclusive_scan_u32((uint32_t)nb);
    const uint64_t after = __ballot(upto > x);
    if (after) {
      const int l = __builtin_ctzll(after);
      Found f;
      f.b = b0 + l;
      f.j = x - (__builtin_amdgcn_readlane(upto, l) - __builtin_amdgcn_readlane(nb, l));
      f.s.first = __builtin_amdgcn_readlane(s.first, l);
      f.s.n = __builtin_amdgcn_readlane(s.n, l);
      f.s.len = __builtin_amdgcn_readlane(s.len, l);
      return f;
    }
    before = __builtin_amdgcn_readlane(upto, kWave - 1);
  }
  return Found{-1, 0, {}};
}

// u[j] = rne(x[j] a / s) + 128, a = 1 or the scale that integer x[j] had; r: a / s in fp32.
__device__ __forceinline__ void codes8(const float (&x)[8], float a, float s, float r, uint32_t (&w)[2]) {
  w[0] = w[1] = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float t = x[j] * r;
    float c = rintf(t);
    if (!(fabsf(fabsf(t - c) - 0.5f) >= 0x1p-13f)) c = (float)rint((double)x[j] * (double)a / (double)s);
    w[j >> 2] |= (uint32_t)((int)fminf(fmaxf(c, -127.f), 127.f) + 128) << (8 * (j & 3));
  }
}

// The larger of the kept scale and the new rows' (m: bits of their largest size).
__device__ __forceinline__ float scale8(float old, uint32_t m) {
  if (m >= 0x7F800000u || old != old) return __uint_as_float(0x7FC00000u);
  return fmaxf(old, __uint_as_float(m) / 127.0f);
}

template <int DT, bool VEC>
__device__ __forceinline__ void append_block(const Append8Args& a, int x, int hg, uint8_t* codes, uint32_t (*sh_max)[2]) {
  const int D = a.kv.D, slices = D >> 3, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int PL = min(16, kBlock / slices), HP = max(1, kBlock / (16 * slices)), passes = (16 + PL - 1) / PL;
  const Found f = find_block(a, x, lane);
  if (f.b < 0) return;
  const int n = min(f.s.n, f.s.len), pos0 = f.s.len - n;       // the sequence's first new position
  const int block = pos0 / kBlk8 + f.j, base = block * kBlk8;
  const int i0 = max(pos0 - base, 0), i1 = min(f.s.len - base, kBlk8);   // new positions of this block
  const int id = kv_page(a.kv, f.b, base);
  if (id < 0) return;
  const int hs = threadIdx.x / (slices * PL), rest = threadIdx.x - hs * slices * PL;
  const int pl = rest / slices, slice = rest - pl * slices, d0 = 8 * slice;
  const int h = hg * HP + hs;
  const bool mine = hs < HP && h < a.kv.Hkv;
  uint8_t* blk = a.kv.base + kv8_block(a.kv, id, mine ? h : 0, (base & ((1 << a.kv.page_shift) - 1)) / kBlk8);
  const int last = a.cs ? min(i1, a.max_pos - base) : i1;      // positions without angles are padding
  if (last <= i0) return;
  float y[2][8], v[2][8];
  uint32_t mk = 0, mv = 0;
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const int i = p * PL + pl;
    if (p >= passes || !mine || i < i0 || i >= last) continue;
    // the last n rows of the sequence's: rows in front of position 0 have none
    const size_t t = (size_t)f.s.first + (f.s.n - n) + (base + i - pos0);
    const size_t row = t * a.ldk, head = (size_t)h * D;
    const bool apart = VEC && turn_apart(a, d0);
    const Eight<DT> own = load8<DT, VEC>(a.k, row + head + d0), val = load8<DT, VEC>(a.v, t * a.ldv + head + d0);
    Eight<DT> oth = {};
    if (apart) oth = load8<DT, VEC>(a.k, row + head + turn_other(a, d0));
    Turn turn;
    if (a.cs && d0 < a.rot) load_turn(a, a.cs + (size_t)(base + i) * a.rot, d0, turn);
    turn8<DT, VEC>(a, a.k, row + head, d0, own, oth, turn, y[p]);
    widen<DT>(val, v[p]);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      mk = max(mk, __float_as_uint(y[p][j]) & 0x7FFFFFFFu);
      mv = max(mv, __float_as_uint(v[p][j]) & 0x7FFFFFFFu);
    }
  }
#pragma unroll
  for (int o = 32; o; o >>= 1) {
    mk = max(mk, (uint32_t)__shfl_xor((int)mk, o));
    mv = max(mv, (uint32_t)__shfl_xor((int)mv, o));
  }
  if (lane == 0) {
    sh_max[wave][0] = mk;
    sh_max[wave][1] = mv;
  }
  __syncthreads();
  // a head's threads are whole waves where a workgroup takes several
  const int span = HP > 1 ? slices * 16 / kWave : kWavesPerBlock, w0 = HP > 1 ? min(hs, HP - 1) * span : 0;
  mk = mv = 0;
  for (int w = w0; w < w0 + span; ++w) {
    mk = max(mk, sh_max[w][0]);
    mv = max(mv, sh_max[w][1]);
  }
  const bool fresh = i0 == 0;
  float2 old = make_float2(0.f, 0.f);
  if (!fresh && mine) old = *(const float2*)(blk + 32 * D);
  const float ks = scale8(old.x, mk), vs = scale8(old.y, mv);
  // the scales are read before they are written
  __syncthreads();
  // where a scale grows, and in a fresh block, every position is written
  const bool allk = fresh || ks != old.x, allv = fresh || vs != old.y;
  uint8_t* cv = codes + (mine ? hs : 0) * 16 * D;
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const int i = p * PL + pl;
    if (p >= passes || !mine || i >= kBlk8) continue;
    const bool is_new = i >= i0 && i < last;
    uint32_t kw[2] = {0x80808080u, 0x80808080u}, vw[2] = {0x80808080u, 0x80808080u};
    uint8_t *kp = blk + i * D + d0, *vp = blk + 16 * D + ((i >> 2) * D + d0) * 4 + (i & 3);
    if (is_new) {
      if (ks > 0.f) codes8(y[p], 1.0f, ks, 1.0f / ks, kw);
      if (vs > 0.f) codes8(v[p], 1.0f, vs, 1.0f / vs, vw);
    } else if (!fresh) {
      float was[8];
      if (allk && ks > 0.f) {
        const Raw<8> c = load_raw<8>(kp);
#pragma unroll
        for (int j = 0; j < 8; ++j) was[j] = (float)((int)((c.w[j >> 2] >> (8 * (j & 3))) & 255u) - 128);
        codes8(was, old.x, ks, old.x / ks, kw);
      }
      if (allv && vs > 0.f) {
#pragma unroll
        for (int j = 0; j < 8; ++j) was[j] = (float)((int)vp[4 * j] - 128);
        codes8(was, old.y, vs, old.y / vs, vw);
      }
    }
    if (allk || is_new) *(Raw<8>*)kp = Raw<8>{{kw[0], kw[1]}};
    if (allv) {
      *(Raw<8>*)(cv + i * D + d0) = Raw<8>{{vw[0], vw[1]}};
    } else if (is_new) {
#pragma unroll
      for (int j = 0; j < 8; ++j) vp[4 * j] = (uint8_t)(vw[j >> 2] >> (8 * (j & 3)));
    }
  }
  __syncthreads();
  if (!mine) return;
  if (allv)
    for (int e = rest; e < 4 * D; e += slices * PL) {          // a word: positions 4 c .. 4 c + 3 of a dim
      const int c = e / D, d = e - c * D;
      const uint8_t* s = cv + 4 * c * D + d;
      ((uint32_t*)(blk + 16 * D))[e] = s[0] | (uint32_t)s[D] << 8 | (uint32_t)s[2 * D] << 16 | (uint32_t)s[3 * D] << 24;
    }
  if (rest == 0) *(float2*)(blk + 32 * D) = make_float2(ks, vs);
}

// Position of row t where the append stores it (angles for max_pos positions; 0: no angles), else -1.  Each wave
// finds it for itself, 64 sequences at a time.
__device__ __forceinline__ int stored_pos(const KvCache& kv, const Rows8& rows, int max_pos, int t, int lane) {
  for (int b0 = 0; b0 < kv.B; b0 += kWave) {
    Seq8 s{};
    if (b0 + lane < kv.B) s = rows8_seq(rows, b0 + lane);
    const uint64_t in = __ballot(t >= s.first && t < s.first + s.n);
    if (!in) continue;
    const int l = __builtin_ctzll(in);
    const int pos = __builtin_amdgcn_readlane(s.pos, l) + t - __builtin_amdgcn_readlane(s.first, l);
    return pos < 0 || (max_pos && pos >= max_pos) || kv_page(kv, b0 + l, pos) < 0 ? -1 : pos;
  }
  return -1;
}

// Queries of one token.
template <int DT, int QDT, bool VEC>
__device__ __forceinline__ void append_query(const Append8Args& a, int t) {
  const int D = a.kv.D, slices = D >> 3;
  const int pos = stored_pos(a.kv, a.rows, a.cs ? a.max_pos : 0, t, threadIdx.x & 63);
  if (pos < 0) return;
  const int step = kBlock / slices, slice = threadIdx.x % slices, d0 = 8 * slice;
  if ((int)threadIdx.x >= step * slices) return;
  Turn turn;
  if (a.cs && d0 < a.rot) load_turn(a, a.cs + (size_t)pos * a.rot, d0, turn);
  const bool apart = VEC && turn_apart(a, d0);
  constexpr int U = 4;                                         // heads on their way
  for (int h0 = threadIdx.x / slices; h0 < a.Hq; h0 += U * step) {
    Eight<DT> own[U], oth[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const size_t row = (size_t)t * a.ldq + (size_t)min(h0 + u * step, a.Hq - 1) * D;
      own[u] = load8<DT, VEC>(a.q, row + d0);
      oth[u] = {};
      if (apart) oth[u] = load8<DT, VEC>(a.q, row + turn_other(a, d0));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * step;
      if (h >= a.Hq) break;
      float y[8];
      turn8<DT, VEC>(a, a.q, (size_t)t * a.ldq + (size_t)h * D, d0, own[u], oth[u], turn, y);
      const size_t out = ((size_t)t * a.Hq + h) * D + d0;
      if constexpr (VEC) {
        store8<QDT>(a.q_out, out, y);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) store_elem<QDT>(a.q_out, out + j, y[j]);
      }
    }
  }
}

template <int DT, int QDT, bool VEC>
__global__ __launch_bounds__(kBlock) void k_kv_append8(Append8Args a) {
  __shared__ __attribute__((aligned(8))) uint8_t codes[16 * 256];
  __shared__ uint32_t sh_max[kWavesPerBlock][2];
  const int kv_groups = a.blocks * a.hgroups;
  if ((int)blockIdx.x < kv_groups) append_block<DT, VEC>(a, blockIdx.x / a.hgroups, blockIdx.x % a.hgroups, codes, sh_max);
  else append_query<DT, QDT, VEC>(a, blockIdx.x - kv_groups);
}

struct Blank8Args {
  KvCache kv;
  Rows8 rows;
  uint8_t* x;
  int max_pos, bytes;       // bytes of a row
};

// A wave per row.  8192 rows of 16 KiB of one sequence: 5.9 us a call where all are tokens (the launch), 21 where none is.
__global__ __launch_bounds__(kBlock) void k_kv_blank8(Blank8Args a) {
  const int lane = threadIdx.x & 63, t = blockIdx.x * kWavesPerBlock + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (t >= a.rows.T || stored_pos(a.kv, a.rows, a.max_pos, t, lane) >= 0) return;
  for (int e = lane * 16; e < a.bytes; e += kWave * 16) *(Raw<16>*)(a.x + (size_t)t * a.bytes + e) = zero16();
}

struct Read8Args {
  KvCache kv;
  const int32_t *pos, *seq;
  void *k, *v;              // [T][Hkv][D]
  int T;
};

// A thread takes 8 dims of one token and head, a workgroup four neighbouring tokens: their V codes
// share words.
template <int DT>
__global__ __launch_bounds__(kBlock) void k_kv_read8(Read8Args a) {
  const int D = a.kv.D, slices = D >> 3, heads = kBlock / 4 / slices;
  const int r = threadIdx.x >> 2, hl = r / slices, slice = r - hl * slices, d0 = 8 * slice;
  const int t = blockIdx.x * 4 + (threadIdx.x & 3), h = blockIdx.y * heads + hl;
  if (t >= a.T || hl >= heads || h >= a.kv.Hkv) return;
  const int pos = a.pos[t], b = a.seq ? a.seq[t] : t;
  const int id = pos >= 0 && (unsigned)b < (unsigned)a.kv.B ? kv_page(a.kv, b, pos) : -1;
  float kf[8], vf[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) kf[j] = vf[j] = 0.f;
  if (id >= 0) {
    const int in_page = pos & ((1 << a.kv.page_shift) - 1), i = in_page & 15;
    const uint8_t* blk = a.kv.base + kv8_block(a.kv, id, h, in_page >> 4);
    const Raw<8> kw = load_raw<8>(blk + i * D + d0);
    const uint8_t* vp = blk + 16 * D + ((i >> 2) * D + d0) * 4;
    const Raw<16> v0 = load_raw<16>(vp), v1 = load_raw<16>(vp + 16);
    const float2 s = *(const float2*)(blk + 32 * D);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      kf[j] = (float)((int)((kw.w[j >> 2] >> (8 * (j & 3))) & 255u) - 128) * s.x;
      vf[j] = (float)((int)(((j < 4 ? v0.w[j & 3] : v1.w[j & 3]) >> (8 * (i & 3))) & 255u) - 128) * s.y;
    }
  }
  const size_t out = ((size_t)t * a.kv.Hkv + h) * D + d0;
  store8<DT>(a.k, out, kf);
  store8<DT>(a.v, out, vf);
}

template <int DT, int QDT>
void run_append8(hipStream_t s, const Append8Args& a, unsigned grid, bool vec) {
  if (vec) k_kv_append8<DT, QDT, true><<<dim3(grid), dim3(kBlock), 0, s>>>(a);
  else k_kv_append8<DT, QDT, false><<<dim3(grid), dim3(kBlock), 0, s>>>(a);
}
template <int DT>
void run_append8(hipStream_t s, const Append8Args& a, unsigned grid, int qdt, bool vec) {
  if (qdt == DT_F16) run_append8<DT, DT_F16>(s, a, grid, vec);
  else run_append8<DT, DT_BF16>(s, a, grid, vec);
}

}  // namespace

// T rows of B sequences touch at most T blocks, and at most two more than whole ones each.
static int append_blocks(const KvGeom& g, int T) { return (int)std::min<long long>(T, (long long)T / kBlk8 + 2ll * g.B); }
static int append_heads(const KvGeom& g) { return std::max(1, kBlock / (2 * g.D)); }   // of a workgroup
long long kv_append_q8_groups(const KvGeom& g, int T, bool queries) {
  return (long long)append_blocks(g, T) * ((g.Hkv + append_heads(g) - 1) / append_heads(g)) + (queries ? T : 0);
}

hipError_t launch_kv_append_q8(hipStream_t s, const KvGeom& g, int xdt, int qdt, int T, int Hq, const void* q, size_t ldq,
                               const void* k, size_t ldk, const void* v, size_t ldv, const int32_t* q_start,
                               const int32_t* lens, const float* cos_sin, int rot, int max_pos, int pairs,
                               const int32_t* table, void* cache, void* q_out) {
  const int heads = append_heads(g);
  const Append8Args a{{cos_sin, rot, max_pos, pairs},
                      {(uint8_t*)cache, table, g.Hkv, g.D, g.page_shift, g.num_pages, g.max_pages, g.B},
                      {q_start, lens, T, T}, q, k, v, ldq, ldk, ldv,
                      q_out, Hq, append_blocks(g, T),
                      (g.Hkv + heads - 1) / heads};
  const uintptr_t row = xdt == DT_F32 ? 4 : 8;                  // elements of 16 bytes
  const bool vec = (((uintptr_t)q | (uintptr_t)k | (uintptr_t)v | (uintptr_t)q_out) & 15u) == 0 &&
                   ((ldq | ldk | ldv) & (row - 1)) == 0 && (!cos_sin || (pairs ? rot % 8 == 0 : rot % 16 == 0));
  const unsigned grid = (unsigned)kv_append_q8_groups(g, T, q != nullptr);
  if (xdt == DT_F32) run_append8<DT_F32>(s, a, grid, qdt, vec);
  else if (xdt == DT_F16) run_append8<DT_F16>(s, a, grid, qdt, vec);
  else run_append8<DT_BF16>(s, a, grid, qdt, vec);
  return hipGetLastError();
}

hipError_t launch_kv_blank_q8(hipStream_t s, const KvGeom& g, int T, int n, void* x, const int32_t* q_start,
                              const int32_t* lens, int max_pos, int max_q, const int32_t* table) {
  const Blank8Args a{{nullptr, table, g.Hkv, g.D, g.page_shift, g.num_pages, g.max_pages, g.B}, {q_start, lens, T, max_q},
                     (uint8_t*)x, max_pos, 2 * n};
  k_kv_blank8<<<dim3((T + kWavesPerBlock - 1) / kWavesPerBlock), dim3(kBlock), 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_kv_read_q8(hipStream_t s, const KvGeom& g, int odt, int T, const int32_t* pos, const int32_t* seq,
                             const int32_t* table, const void* cache, void* k, void* v) {
  const Read8Args a{{(uint8_t*)cache, table, g.Hkv, g.D, g.page_shift, g.num_pages, g.max_pages, g.B}, pos, seq, k, v, T};
  const int heads = kBlock / 4 / (g.D >> 3);
  const dim3 grid((T + 3) / 4, (g.Hkv + heads - 1) / heads), block(kBlock);
  if (odt == DT_F32) k_kv_read8<DT_F32><<<grid, block, 0, s>>>(a);
  else if (odt == DT_F16) k_kv_read8<DT_F16><<<grid, block, 0, s>>>(a);
  else k_kv_read8<DT_BF16><<<grid, block, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace sfx
