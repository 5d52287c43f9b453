// C ABI of libsfx: host-side argument checks, workspace queries, status strings.
// Every check runs before anything is enqueued, and no check touches the GPU
// except the CU-count query that sizes persistent grids.
#include <hip/hip_runtime.h>

#include <atomic>
#include <cmath>

#include "../../include/sfx.h"
#include "sfx_launch.hpp"
#include "sfx_step.hpp"

namespace sfx {

int device_cu_count() {
  static std::atomic<int> cache[64];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) return 0;
  if (dev < 64) {
    const int c = cache[dev].load(std::memory_order_relaxed);
    if (c > 0) return c;
  }
  int cus = 0;
  if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess) return 0;
  if (dev < 64) cache[dev].store(cus, std::memory_order_relaxed);
  return cus;
}

// Runs per sequence: two workgroups of eight waves per compute unit, and no run shorter than
// a tile per wave.  256 units of up to 2048 positions are left whole: eight sequences of 32 kv
// heads take 20.8 us in one run and 23.4 in two at 2048 positions each, 68 and 67 at 8192,
// and 61 and 48 where their lengths are spread up to 8192.
AttnPlan attn_plan(int B, int Hq, int Hkv, int max_len) {
  AttnPlan p;
  p.Hq = Hq;
  p.G = Hq / Hkv;
  p.HT = (p.G + 15) / 16;
  p.HG = p.G < 16 ? p.G : 16;
  const int units = B * Hkv * p.HT;
  const int most = (max_len + 255) / 256;
  p.S = units >= 256 && max_len <= 2048 ? 1 : (512 + units - 1) / units;
  if (p.S > most) p.S = most;
  return p;
}

size_t attn_ws_bytes(const AttnPlan& p, int B, int Hkv, int D) {
  if (p.S <= 1) return 0;
  return (size_t)B * Hkv * p.HT * p.S * p.HG * (D + 4) * 4;
}

// Rows of a tile and runs of its positions.  Up to 96 rows of a sequence and kv head: 16 or 32 at a time,
// waves deal the positions among themselves, at least 512 workgroups and no run shorter than a tile of
// positions per wave; 256 units are left whole.  By registers one workgroup of eight waves fits a compute unit at
// heads of 96 and 128 and with two tiles of heads of 64, two or three fit below: 512 are two rounds there, and
// whether one round of 256 is better goes by how runs fill it.  8 kv heads of 128, one token, by 512 and 256: 1 x
// 131072 64.7 and 60.4 us, 8 x 4096 24.7 and 21.2, 17 x 4096 43 and 46, 20 x 4096 52 and 53, 28 x 4096 64 and 61
// (by 768: 70, 28, 46, 56, 67).  More rows: 128 or 256 at a time, no run shorter than 256 positions, and a
// workspace of at most 64 MiB.  16 sequences of 4096 with 8 kv heads of 64, 48, 80 and 112 rows: 32, 58 and 61 us by 32 rows, 48,
// 51 and 55 by 128; 80 rows of lengths up to 4096 behind a window of 1500: 16 and 26; 131072 positions, 8
// kv heads of 128, 64 and 120 rows: 100 and 161, 124 and 134.
Attn8Plan attn8_plan(int B, int max_q, int Hq, int Hkv, int D, int max_len) {
  Attn8Plan p;
  p.Hq = Hq;
  p.G = Hq / Hkv;
  const long long rows = (long long)max_q * p.G;
  const int many = attn8_rows(D / 32);
  p.R = rows <= 16 ? 16 : rows <= 96 ? 32 : many;
  p.RT = (int)((rows + p.R - 1) / p.R);
  const long long units = (long long)B * Hkv * p.RT;
  const int most = (max_len + 255) / 256;
  const long long want = p.R == many ? 63488 / many / units : units >= 256 ? 1 : (512 + units - 1) / units;
  p.S = (int)(want < 1 ? 1 : want > most ? most : want);
  return p;
}

// Workgroups of a call, also of rows that its sequences do not have.
bool attn8_fits(const Attn8Plan& p, int B, int Hkv) { return (long long)B * Hkv * p.RT * p.S < (1 << 24); }

size_t attn8_ws_bytes(const Attn8Plan& p, int B, int Hkv, int D) {
  if (p.S <= 1) return 0;
  return (size_t)B * Hkv * p.RT * p.S * p.R * (D + 4) * 4;
}

}  // namespace sfx

namespace {

int elem_bytes(int wdt) {
  switch (wdt) {
    case SFX_F32: return 4;
    case SFX_F16: return 2;
    case SFX_BF16: return 2;
    default: return 0;
  }
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }
bool aligned256(const void* p) { return ((uintptr_t)p & 255u) == 0; }

int check_ws(void* ws, size_t ws_bytes, size_t need) {
  if (need == 0) return SFX_OK;
  if (ws == nullptr || !aligned256(ws) || ws_bytes < need) return SFX_E_WORKSPACE;
  return SFX_OK;
}

int launch_status(hipError_t e) { return e == hipSuccess ? SFX_OK : SFX_E_LAUNCH; }

// Row of `n` stored elements of `wdt` (Q4: n codes) spans a multiple of 16 bytes.
bool row_ok(int wdt, long long n) {
  if (wdt == SFX_Q4G32) return n % 32 == 0;
  return (n * elem_bytes(wdt)) % 16 == 0;
}

// Shape of a paged int4 cache; fills `g` when it is one the kernels take.
int kv_geom(int B, int Hkv, int D, int page, int num_pages, int max_pages, sfx::KvGeom* g) {
  if (B < 1 || Hkv < 1 || Hkv > sfx::kAttnMaxHeads || D < 32 || D > 256 || D % 32 != 0) return SFX_E_SHAPE;
  if (page < 8 || page > 1024 || (page & (page - 1)) != 0 || num_pages < 1 || max_pages < 1) return SFX_E_SHAPE;
  if ((long long)max_pages * page > (1ll << 30)) return SFX_E_SHAPE;
  // blocks of 8 positions are counted in 31 bits (of 288 bytes and more: beyond any device)
  if ((long long)num_pages * Hkv * (page / 8) > 0x7FFFFFFFll) return SFX_E_SHAPE;
  *g = sfx::KvGeom{B, Hkv, D, __builtin_ctz((unsigned)page), num_pages, max_pages};
  return SFX_OK;
}

// The same of an int8 cache (blocks of 16 positions; q4's limits hold for it too).
int kv_geom8(int B, int Hkv, int D, int page, int num_pages, int max_pages, sfx::KvGeom* g) {
  if (page < 16 || B > sfx::kQ8MaxSeqs) return SFX_E_SHAPE;
  return kv_geom(B, Hkv, D, page, num_pages, max_pages, g);
}

bool dt16_or_32(int dt) { return dt == SFX_F32 || dt == SFX_F16 || dt == SFX_BF16; }
bool aligned_elem(const void* p, int dt) { return ((uintptr_t)p & (uintptr_t)(elem_bytes(dt) - 1)) == 0; }

}  // namespace

extern "C" {

const char* sfx_status_str(int status) {
  switch (status) {
    case SFX_OK: return "ok";
    case SFX_E_NULL: return "required pointer is NULL";
    case SFX_E_SHAPE: return "size out of range or inconsistent";
    case SFX_E_DTYPE: return "unknown or unsupported dtype / activation for this call";
    case SFX_E_ALIGN: return "pointer or row not 16-byte aligned";
    case SFX_E_WORKSPACE: return "workspace NULL, misaligned or too small";
    case SFX_E_LAUNCH: return "HIP reported a launch error";
    case SFX_E_UNSUPPORTED: return "combination not built";
    case SFX_E_DEVICE: return "no current HIP device";
    case SFX_E_SCRATCH: return "needs more scratch than the static maximum (SFX_DOWN_SCRATCH_BYTES)";
    default: return "unknown status";
  }
}

int sfx_abi_version(void) { return SFX_ABI_VERSION; }

// ------------------------------------------------------------------------------ predict

size_t sfx_predict_ws(int wdt, int B, int d, int h, int f) {
  if (B < 1 || B > SFX_MAX_B || h < 1) return 0;
  if (wdt < SFX_F32 || wdt > SFX_Q4G32) return 0;
  return sfx::predict_ws_bytes(wdt, B, d, h, f);
}

int sfx_predict(void* stream, int wdt, int B, int d, int h, int f, const void* x, const void* W1,
                const void* W2, float* scores, void* ws, size_t ws_bytes) {
  if (wdt != SFX_F32 && wdt != SFX_F16 && wdt != SFX_BF16) return SFX_E_DTYPE;
  if (B < 1 || B > SFX_MAX_B || d < 1 || h < 1 || f < 1) return SFX_E_SHAPE;
  if (!x || !W1 || !W2 || !scores) return SFX_E_NULL;
  if (!row_ok(wdt, d) || !row_ok(wdt, h)) return SFX_E_ALIGN;
  if (!aligned16(x) || !aligned16(W1) || !aligned16(W2) || !aligned16(scores)) return SFX_E_ALIGN;
  const int w = check_ws(ws, ws_bytes, sfx::predict_ws_bytes(wdt, B, d, h, f));
  if (w != SFX_OK) return w;
  return launch_status(
      sfx::launch_predict((hipStream_t)stream, wdt, B, d, h, f, x, W1, W2, scores, ws));
}

int sfx_predict_q4(void* stream, int B, int d, int h, int f, const void* x, const void* W1, const void* W1_scales,
                   const void* W2, const void* W2_scales, float* scores, void* ws, size_t ws_bytes) {
  if (B < 1 || B > SFX_MAX_B || d < 1 || h < 1 || f < 1) return SFX_E_SHAPE;
  if (d % 32 != 0 || h % 32 != 0) return SFX_E_SHAPE;
  if (!x || !W1 || !W1_scales || !W2 || !W2_scales || !scores) return SFX_E_NULL;
  if (!aligned16(x) || !aligned16(W1) || !aligned16(W2) || !aligned16(scores)) return SFX_E_ALIGN;
  if (((uintptr_t)W1_scales & 1u) != 0 || ((uintptr_t)W2_scales & 1u) != 0) return SFX_E_ALIGN;
  const int w = check_ws(ws, ws_bytes, sfx::predict_ws_bytes(SFX_Q4G32, B, d, h, f));
  if (w != SFX_OK) return w;
  return launch_status(
      sfx::launch_predict_q4((hipStream_t)stream, B, d, h, f, x, W1, W1_scales, W2, W2_scales, scores, ws));
}

// ------------------------------------------------------------------------------ compact

size_t sfx_compact_ws(int B, int f) {
  if (B < 1 || f < 1) return 0;
  return sfx::compact_ws_bytes(B, f);
}

int sfx_compact(void* stream, int B, int f, const float* scores, float threshold, uint32_t* tok_bits,
                uint32_t* union_bits, int32_t* idx, int kmax, int32_t* count, void* ws, size_t ws_bytes) {
  if (B < 1 || B > SFX_MAX_B || f < 1) return SFX_E_SHAPE;
  if (kmax < f) return SFX_E_SHAPE;
  if (!scores || !union_bits || !idx || !count) return SFX_E_NULL;
  if (!aligned16(scores) || !aligned4(union_bits) || !aligned4(idx) || (tok_bits && !aligned4(tok_bits)))
    return SFX_E_ALIGN;
  const int w = check_ws(ws, ws_bytes, sfx::compact_ws_bytes(B, f));
  if (w != SFX_OK) return w;
  return launch_status(sfx::launch_compact((hipStream_t)stream, B, f, scores, threshold, tok_bits, union_bits,
                                           idx, kmax, count, ws));
}

// ------------------------------------------------------------------------------ up

int sfx_sparse_up(void* stream, int wdt, int act, int B, int d, int f, const void* x, const void* Wa,
                  const void* Wa_scales, const float* ba, const void* Wl, const void* Wl_scales,
                  const int32_t* idx, const int32_t* count, int kmax, float* hact) {
  if (wdt < SFX_F32 || wdt > SFX_Q4G32) return SFX_E_DTYPE;
  if (act != SFX_RELU && act != SFX_REGLU && act != SFX_RELU2) return SFX_E_DTYPE;
  if (B < 1 || B > SFX_MAX_B || d < 1 || f < 1 || kmax < 1) return SFX_E_SHAPE;
  if (!x || !Wa || !idx || !count || !hact) return SFX_E_NULL;
  if (act == SFX_REGLU && !Wl) return SFX_E_NULL;
  if (wdt == SFX_Q4G32 && (!Wa_scales || (act == SFX_REGLU && !Wl_scales))) return SFX_E_NULL;
  if (!row_ok(wdt, d)) return wdt == SFX_Q4G32 ? SFX_E_SHAPE : SFX_E_ALIGN;
  if (!aligned16(x) || !aligned16(Wa) || !aligned16(hact) || (Wl && !aligned16(Wl))) return SFX_E_ALIGN;
  if (!sfx::up_supported(wdt, act, B)) return SFX_E_UNSUPPORTED;
  return launch_status(sfx::launch_up((hipStream_t)stream, wdt, act, B, d, f, x, Wa, Wa_scales, ba,
                                      act == SFX_REGLU ? Wl : nullptr, Wl_scales, idx, count, kmax, hact));
}

// ------------------------------------------------------------------------------ down

size_t sfx_sparse_down_ws(int wdt, int B, int d, int kmax) {
  if (wdt < SFX_F32 || wdt > SFX_Q4G32 || B < 1 || B > SFX_MAX_B || d < 1 || kmax < 1) return 0;
  return sfx::down_ws_bytes(wdt, B, d, kmax);
}

int sfx_sparse_down(void* stream, int wdt, int B, int d, int f, const void* Wd, const void* Wd_scales,
                    const int32_t* idx, const int32_t* count, int kmax, const float* hact, float* y, void* ws,
                    size_t ws_bytes) {
  if (wdt < SFX_F32 || wdt > SFX_Q4G32) return SFX_E_DTYPE;
  if (B < 1 || B > SFX_MAX_B || d < 1 || f < 1 || kmax < 1) return SFX_E_SHAPE;
  if (!Wd || !idx || !count || !hact || !y) return SFX_E_NULL;
  if (wdt == SFX_Q4G32 && !Wd_scales) return SFX_E_NULL;
  if (!row_ok(wdt, d)) return wdt == SFX_Q4G32 ? SFX_E_SHAPE : SFX_E_ALIGN;
  if (!aligned16(Wd) || !aligned16(hact) || !aligned16(y)) return SFX_E_ALIGN;
  if (!sfx::down_supported(wdt, B)) return SFX_E_UNSUPPORTED;
  const int w = check_ws(ws, ws_bytes, sfx::down_ws_bytes(wdt, B, d, kmax));
  if (w != SFX_OK) return w;
  return launch_status(sfx::launch_down((hipStream_t)stream, wdt, B, d, f, Wd, Wd_scales, idx, count, kmax,
                                        hact, y, ws));
}

int sfx_sparse_down_noalloc(void* stream, int wdt, int B, int d, int f, const void* Wd, const void* Wd_scales,
                            const int32_t* idx, const int32_t* count, int kmax, const float* hact, float* y) {
  if (wdt < SFX_F32 || wdt > SFX_Q4G32) return SFX_E_DTYPE;
  if (B < 1 || B > SFX_MAX_B || d < 1 || f < 1 || kmax < 1) return SFX_E_SHAPE;
  if (!Wd || !idx || !count || !hact || !y) return SFX_E_NULL;
  if (wdt == SFX_Q4G32 && !Wd_scales) return SFX_E_NULL;
  if (!row_ok(wdt, d)) return wdt == SFX_Q4G32 ? SFX_E_SHAPE : SFX_E_ALIGN;
  if (!aligned16(Wd) || !aligned16(hact) || !aligned16(y)) return SFX_E_ALIGN;
  if (!sfx::down_supported(wdt, B)) return SFX_E_UNSUPPORTED;
  const size_t need = sfx::down_ws_bytes(wdt, B, d, kmax);
  if (need > sfx::kDownScratchBytes) return SFX_E_SCRATCH;
  void* scratch = nullptr;
  if (sfx::down_scratch(&scratch) != hipSuccess) return SFX_E_DEVICE;
  return launch_status(sfx::launch_down((hipStream_t)stream, wdt, B, d, f, Wd, Wd_scales, idx, count, kmax,
                                        hact, y, scratch));
}

// ------------------------------------------------------------------------------ dense step

size_t sfx_dense_ffn_ws(int wdt, int B, int d, int f) {
  if (wdt < SFX_F32 || wdt > SFX_Q4G32 || B < 1 || B > SFX_MAX_B || d < 1 || f < 1) return 0;
  return sfx::dense_ws_bytes(wdt, B, d, f);
}

int sfx_dense_ffn(void* stream, int wdt, int act, int B, int d, int f, const void* x, const void* Wa,
                  const void* Wa_scales, const float* ba, const void* Wl, const void* Wl_scales, const void* Wd,
                  const void* Wd_scales, float* hact, float* y, void* ws, size_t ws_bytes) {
  if (wdt < SFX_F32 || wdt > SFX_Q4G32) return SFX_E_DTYPE;
  if (act != SFX_RELU && act != SFX_REGLU && act != SFX_RELU2) return SFX_E_DTYPE;
  if (B < 1 || B > SFX_MAX_B || d < 1 || f < 1) return SFX_E_SHAPE;
  if (!x || !Wa || !Wd || !hact || !y) return SFX_E_NULL;
  if (act == SFX_REGLU && !Wl) return SFX_E_NULL;
  if (wdt == SFX_Q4G32 && (!Wa_scales || !Wd_scales || (act == SFX_REGLU && !Wl_scales))) return SFX_E_NULL;
  if (!row_ok(wdt, d)) return wdt == SFX_Q4G32 ? SFX_E_SHAPE : SFX_E_ALIGN;
  if (!aligned16(x) || !aligned16(Wa) || !aligned16(Wd) || !aligned16(hact) || !aligned16(y) ||
      (Wl && !aligned16(Wl)))
    return SFX_E_ALIGN;
  if (!sfx::up_supported(wdt, act, B) || !sfx::down_supported(wdt, B)) return SFX_E_UNSUPPORTED;
  const int w = check_ws(ws, ws_bytes, sfx::dense_ws_bytes(wdt, B, d, f));
  if (w != SFX_OK) return w;
  return launch_status(sfx::launch_dense((hipStream_t)stream, wdt, act, B, d, f, x, Wa, Wa_scales, ba,
                                         act == SFX_REGLU ? Wl : nullptr, Wl_scales, Wd, Wd_scales, hact, y, ws));
}

// ------------------------------------------------------------------------------ TAM

size_t sfx_tam_ws(int G, int K) { return sfx::tam_ws_bytes(G, K); }

int sfx_tam_update(void* stream, int L, int G, const uint32_t* union_bits, float lambda, float eps, int K,
                   float* score, uint32_t* hot_bits, uint32_t* entered_bits, uint32_t* left_bits,
                   int32_t* topk, int32_t* topk_count, void* ws, size_t ws_bytes) {
  (void)ws;
  (void)ws_bytes;
  if (L < 1 || G < 1 || G > SFX_MAX_GROUPS || K < 0 || K > G) return SFX_E_SHAPE;
  if (!(lambda > 0.0f && lambda < 1.0f) || !(eps >= 0.0f)) return SFX_E_SHAPE;
  if (!union_bits || !score || !hot_bits || !entered_bits || !left_bits || !topk_count) return SFX_E_NULL;
  if (K > 0 && !topk) return SFX_E_NULL;
  return launch_status(sfx::launch_tam((hipStream_t)stream, L, G, union_bits, lambda, eps, K, score, hot_bits,
                                       entered_bits, left_bits, topk, topk_count));
}

int sfx_topk_now_update(void* stream, int L, int G, const uint32_t* union_bits, int K, uint32_t* hot_bits,
                        uint32_t* entered_bits, uint32_t* left_bits, int32_t* topk, int32_t* topk_count) {
  if (L < 1 || G < 1 || G > SFX_MAX_GROUPS || K < 0 || K > G) return SFX_E_SHAPE;
  if (!union_bits || !hot_bits || !entered_bits || !left_bits || !topk_count) return SFX_E_NULL;
  if (K > 0 && !topk) return SFX_E_NULL;
  return launch_status(sfx::launch_topk_now((hipStream_t)stream, L, G, union_bits, K, hot_bits, entered_bits,
                                            left_bits, topk, topk_count));
}

// ------------------------------------------------------------------------------ hot region

int sfx_hot_update(void* stream, int L, int G, int K, const uint32_t* entered_bits, const uint32_t* left_bits,
                   int32_t* slot_of, int32_t* group_of, int32_t* copies, int32_t* ncopies, int nmat,
                   const size_t* group_bytes, const void* const* src, void* const* dst) {
  if (L < 1 || G < 1 || G > SFX_MAX_GROUPS || K < 1 || K > G) return SFX_E_SHAPE;
  if (L > sfx::kHotMaxLayers) return SFX_E_SHAPE;
  if (nmat < 0 || nmat > sfx::kHotMaxMats) return SFX_E_SHAPE;
  if (!entered_bits || !left_bits || !slot_of || !group_of || !copies || !ncopies) return SFX_E_NULL;
  if (!aligned4(entered_bits) || !aligned4(left_bits) || !aligned4(slot_of) || !aligned4(group_of) ||
      !aligned4(copies) || !aligned4(ncopies))
    return SFX_E_ALIGN;
  sfx::HotMats mats{};
  mats.n = nmat;
  if (nmat > 0) {
    if (!group_bytes || !src || !dst) return SFX_E_NULL;
    if (((uintptr_t)src & 7u) || ((uintptr_t)dst & 7u)) return SFX_E_ALIGN;
    int64_t chunks = 0;
    for (int m = 0; m < nmat; ++m) {
      if (group_bytes[m] == 0 || (group_bytes[m] & 15u)) return SFX_E_SHAPE;
      mats.group_bytes[m] = group_bytes[m];
      mats.chunk_off[m] = (int)chunks;
      chunks += (int64_t)((group_bytes[m] + sfx::kHotChunk - 1) / sfx::kHotChunk);
      if (chunks > (int64_t)(1 << 20)) return SFX_E_SHAPE;      // 16 GiB per group
    }
    mats.chunk_off[nmat] = (int)chunks;
  }
  hipStream_t st = (hipStream_t)stream;
  hipError_t e = sfx::launch_hot_assign(st, L, G, K, entered_bits, left_bits, slot_of, group_of, copies, ncopies);
  if (e == hipSuccess && nmat > 0) e = sfx::launch_hot_copy(st, L, K, mats, src, dst, copies, ncopies);
  return launch_status(e);
}

// ------------------------------------------------------------------------------ calibration

int sfx_count_active(void* stream, int B, int f, const uint32_t* tok_bits, int32_t* counts) {
  if (B < 1 || B > SFX_MAX_B || f < 1) return SFX_E_SHAPE;
  if (!tok_bits || !counts) return SFX_E_NULL;
  if (!aligned4(tok_bits) || !aligned4(counts)) return SFX_E_ALIGN;
  return launch_status(sfx::launch_count_active((hipStream_t)stream, B, f, tok_bits, counts));
}

size_t sfx_select_kth_ws(void) { return sfx::select_ws_bytes(); }

int sfx_select_kth(void* stream, size_t n, const float* values, size_t k, float* out, void* ws, size_t ws_bytes) {
  if (n < 1 || n > (size_t)0xFFFFFFFFu || k >= n) return SFX_E_SHAPE;
  if (!values || !out) return SFX_E_NULL;
  if (!aligned4(values) || !aligned4(out)) return SFX_E_ALIGN;
  if (!ws || ((uintptr_t)ws & 255u) || ws_bytes < sfx::select_ws_bytes()) return SFX_E_WORKSPACE;
  return launch_status(sfx::launch_select_kth((hipStream_t)stream, n, values, k, out, ws));
}

size_t sfx_hot_first_order_ws(int f) { return f < 1 ? 0 : sfx::order_ws_bytes(f); }

int sfx_hot_first_order(void* stream, int f, const int32_t* counts, const int32_t* group, int32_t* perm, void* ws,
                        size_t ws_bytes) {
  if (f < 1 || f > (1 << 24)) return SFX_E_SHAPE;
  if (!counts || !perm) return SFX_E_NULL;
  if (!aligned4(counts) || !aligned4(perm) || (group && !aligned4(group))) return SFX_E_ALIGN;
  if (group && (!ws || ((uintptr_t)ws & 255u) || ws_bytes < sfx::order_ws_bytes(f))) return SFX_E_WORKSPACE;
  return launch_status(sfx::launch_hot_first_order((hipStream_t)stream, f, counts, group, perm, ws));
}

int sfx_gather_rows(void* stream, int n_dst, int n_src, size_t row_bytes, const void* src, const int32_t* idx,
                    void* dst) {
  if (n_dst < 1 || n_src < 1 || row_bytes == 0 || (row_bytes & 3u)) return SFX_E_SHAPE;
  if (!src || !idx || !dst) return SFX_E_NULL;
  if (!aligned4(src) || !aligned4(idx) || !aligned4(dst)) return SFX_E_ALIGN;
  return launch_status(sfx::launch_gather_rows((hipStream_t)stream, n_dst, n_src, row_bytes, src, idx, dst));
}

// ------------------------------------------------------------------------------ fused step

size_t sfx_ffn_step_ws(int wdt, int act, int B, int d, int h, int f) {
  const int P = sfx::device_cu_count();
  if (P <= 0) return 0;
  if (!sfx::step_geometry(wdt, act, B, d, h, f, P).ok) return 0;
  if (!sfx::step_resident(wdt, act, B)) return 0;
  return sfx::step_ws_bytes(B, h, f, P);
}

int sfx_ffn_step(void* stream, int wdt, int act, int B, int d, int h, int f, int L, const sfx_layer* layers,
                 void* ws, size_t ws_bytes) {
  if (wdt < SFX_F32 || wdt > SFX_Q4G32) return SFX_E_DTYPE;
  if (act == SFX_RELU2) return SFX_E_UNSUPPORTED;   // squared ReLU: the separate calls
  if (act != SFX_RELU && act != SFX_REGLU) return SFX_E_DTYPE;
  if (B < 1 || B > SFX_MAX_B || d < 1 || h < 1 || f < 1 || L < 1) return SFX_E_SHAPE;
  if (!layers) return SFX_E_NULL;
  if (!ws) return SFX_E_WORKSPACE;
  const int P = sfx::device_cu_count();
  if (P <= 0) return SFX_E_DEVICE;
  const sfx::StepGeom g = sfx::step_geometry(wdt, act, B, d, h, f, P);
  if (!g.ok) return SFX_E_UNSUPPORTED;
  if (!sfx::step_resident(wdt, act, B)) return SFX_E_UNSUPPORTED;
  const int w = check_ws(ws, ws_bytes, sfx::step_ws_bytes(B, h, f, P));
  if (w != SFX_OK) return w;
  return launch_status(sfx::launch_step((hipStream_t)stream, wdt, act, B, d, h, f, L, layers, ws, g));
}

// ------------------------------------------------------------------------------ Live Pipeline

size_t sfx_ffn_pipeline_ws(int wdt, int act, int B, int d, int h, int f) {
  const int P = sfx::device_cu_count();
  if (P <= 0) return 0;
  if (!sfx::pipe_geometry(wdt, act, B, d, h, f, P).ok) return 0;
  if (!sfx::pipe_resident(wdt, act, B)) return 0;
  return sfx::step_ws_bytes(B, h, f, P);
}

int sfx_ffn_pipeline(void* stream, int wdt, int act, int B, int d, int h, int f, int L, const sfx_layer* layers,
                     void* ws, size_t ws_bytes) {
  if (wdt < SFX_F32 || wdt > SFX_Q4G32) return SFX_E_DTYPE;
  if (act == SFX_RELU2) return SFX_E_UNSUPPORTED;   // squared ReLU: the separate calls
  if (act != SFX_RELU && act != SFX_REGLU) return SFX_E_DTYPE;
  if (B < 1 || B > SFX_MAX_B || d < 1 || h < 1 || f < 1 || L < 1) return SFX_E_SHAPE;
  if (!layers) return SFX_E_NULL;
  if (!ws) return SFX_E_WORKSPACE;
  const int P = sfx::device_cu_count();
  if (P <= 0) return SFX_E_DEVICE;
  const sfx::StepGeom g = sfx::pipe_geometry(wdt, act, B, d, h, f, P);
  if (!g.ok) return SFX_E_UNSUPPORTED;
  if (!sfx::pipe_resident(wdt, act, B)) return SFX_E_UNSUPPORTED;
  const int w = check_ws(ws, ws_bytes, sfx::step_ws_bytes(B, h, f, P));
  if (w != SFX_OK) return w;
  return launch_status(sfx::launch_pipe((hipStream_t)stream, wdt, act, B, d, h, f, L, layers, ws, g));
}

// ------------------------------------------------------------------------------ int4 projection

int sfx_linear_q4(void* stream, int xdt, int group, int B, int n, int d, const void* x, size_t ldx, const void* W,
                  const void* W_scales, const float* bias, int accumulate, float* y, size_t ldy) {
  if (xdt != SFX_F16 && xdt != SFX_BF16) return SFX_E_DTYPE;
  if (group != 32 && group != 64 && group != 128) return SFX_E_SHAPE;
  if (B < 1 || B > SFX_MAX_B || n < 1 || n > (1 << 24) || d < 1 || d > (1 << 24) || d % group != 0) return SFX_E_SHAPE;
  if (ldx < (size_t)d || ldy < (size_t)n) return SFX_E_SHAPE;
  if (!x || !W || !W_scales || !y) return SFX_E_NULL;
  if (!aligned16(x) || !aligned16(W) || ldx % 8 != 0) return SFX_E_ALIGN;
  if (((uintptr_t)W_scales & 1u) || !aligned4(y) || (bias && !aligned4(bias))) return SFX_E_ALIGN;
  const int gsh = group == 32 ? 0 : group == 64 ? 1 : 2;
  const auto f = xdt == SFX_F16 ? sfx::launch_linear_q4_f16 : sfx::launch_linear_q4_bf16;
  return launch_status(f((hipStream_t)stream, gsh, B, n, d, x, ldx * 2, W, W_scales, bias, accumulate, y, ldy));
}

// ------------------------------------------------------------------------------ int4 key/value cache

size_t sfx_kv_cache_bytes(int Hkv, int D, int page, int num_pages) {
  sfx::KvGeom g;
  if (kv_geom(1, Hkv, D, page, num_pages, 1, &g) != SFX_OK) return 0;
  return (size_t)num_pages * Hkv * (page / 8) * 9 * D;
}

int sfx_kv_append_q4(void* stream, int xdt, int qdt, int T, int Hq, int Hkv, int D, const void* q, size_t ldq,
                     const void* k, size_t ldk, const void* v, size_t ldv, const int32_t* pos, const int32_t* seq,
                     const float* cos_sin, int rot, int max_pos, int interleaved, int B, int max_pages,
                     const int32_t* table, int page, int num_pages, void* cache, void* q_out) {
  if (xdt != SFX_F32 && xdt != SFX_F16 && xdt != SFX_BF16) return SFX_E_DTYPE;
  if (q && qdt != SFX_F16 && qdt != SFX_BF16) return SFX_E_DTYPE;
  sfx::KvGeom g;
  const int st = kv_geom(B, Hkv, D, page, num_pages, max_pages, &g);
  if (st != SFX_OK) return st;
  if (T < 1 || T > sfx::kKvMaxTokens) return SFX_E_SHAPE;
  if (q && (Hq < 1 || Hq > sfx::kAttnMaxHeads || ldq < (size_t)Hq * D)) return SFX_E_SHAPE;
  if (ldk < (size_t)Hkv * D || ldv < (size_t)Hkv * D) return SFX_E_SHAPE;
  if (cos_sin && (rot < 2 || rot > D || rot % 2 != 0 || max_pos < 1)) return SFX_E_SHAPE;
  if (!k || !v || !pos || !table || !cache || (q && !q_out)) return SFX_E_NULL;
  const uintptr_t em = (uintptr_t)elem_bytes(xdt) - 1;
  if (((uintptr_t)k & em) || ((uintptr_t)v & em) || ((uintptr_t)q & em) || !aligned16(cache) || ((uintptr_t)q_out & 1u))
    return SFX_E_ALIGN;
  if (!aligned4(pos) || !aligned4(table) || (seq && !aligned4(seq)) || (cos_sin && !aligned4(cos_sin)))
    return SFX_E_ALIGN;
  return launch_status(sfx::launch_kv_append_q4((hipStream_t)stream, g, xdt, qdt, T, q ? Hq : 0, q, ldq, k, ldk, v, ldv,
                                                pos, seq, cos_sin, rot, max_pos, interleaved != 0, table, cache, q_out));
}

int sfx_kv_read_q4(void* stream, int odt, int T, int Hkv, int D, const int32_t* pos, const int32_t* seq, int B,
                   int max_pages, const int32_t* table, int page, int num_pages, const void* cache, void* k, void* v) {
  if (odt != SFX_F32 && odt != SFX_F16 && odt != SFX_BF16) return SFX_E_DTYPE;
  sfx::KvGeom g;
  const int st = kv_geom(B, Hkv, D, page, num_pages, max_pages, &g);
  if (st != SFX_OK) return st;
  if (T < 1 || T > sfx::kKvMaxTokens) return SFX_E_SHAPE;
  if (!pos || !table || !cache || !k || !v) return SFX_E_NULL;
  if (!aligned16(cache) || !aligned16(k) || !aligned16(v)) return SFX_E_ALIGN;
  if (!aligned4(pos) || !aligned4(table) || (seq && !aligned4(seq))) return SFX_E_ALIGN;
  return launch_status(sfx::launch_kv_read_q4((hipStream_t)stream, g, odt, T, pos, seq, table, cache, k, v));
}

int sfx_kv_lens_q4(void* stream, int B, const int32_t* pos, int max_pos, int window, int max_pages, const int32_t* table,
                   int page, int num_pages, int32_t* lens, int32_t* starts) {
  sfx::KvGeom g;
  const int st = kv_geom(B, 1, 32, page, num_pages, max_pages, &g);
  if (st != SFX_OK) return st;
  if (B > sfx::kKvMaxTokens || max_pos < 0 || window < 0 || (window == 0) != (starts == nullptr)) return SFX_E_SHAPE;
  if (!pos || !table || !lens) return SFX_E_NULL;
  if (!aligned4(pos) || !aligned4(table) || !aligned4(lens) || (starts && !aligned4(starts))) return SFX_E_ALIGN;
  return launch_status(sfx::launch_kv_lens_q4((hipStream_t)stream, g, pos, max_pos, window, table, lens, starts));
}

size_t sfx_attn_q4_ws(int B, int Hq, int Hkv, int D, int max_len) {
  if (B < 1 || B > SFX_MAX_B || Hkv < 1 || Hq < 1 || Hq > sfx::kAttnMaxHeads || Hq % Hkv != 0 || D < 32 || D > 256 ||
      D % 32 != 0 || max_len < 1 || max_len > (1 << 30))
    return 0;
  return sfx::attn_ws_bytes(sfx::attn_plan(B, Hq, Hkv, max_len), B, Hkv, D);
}

int sfx_attn_q4(void* stream, int qdt, int B, int Hq, int Hkv, int D, const void* q, size_t ldq, int max_pages,
                const int32_t* table, int page, int num_pages, const void* cache, const int32_t* starts,
                const int32_t* lens, float scale, void* out, float* lse, void* ws, size_t ws_bytes) {
  if (qdt != SFX_F16 && qdt != SFX_BF16) return SFX_E_DTYPE;
  sfx::KvGeom g;
  const int st = kv_geom(B, Hkv, D, page, num_pages, max_pages, &g);
  if (st != SFX_OK) return st;
  if (B > SFX_MAX_B || Hq < 1 || Hq > sfx::kAttnMaxHeads || Hq % Hkv != 0 || ldq < (size_t)Hq * D) return SFX_E_SHAPE;
  if (!(fabsf(scale) < 0x1p115f)) return SFX_E_SHAPE;           // times 2^12 log2(e) (sfx_q4.hpp) it is finite
  if (!q || !table || !cache || !lens || !out) return SFX_E_NULL;
  if (!aligned16(q) || ldq % 8 != 0 || !aligned16(cache) || !aligned16(out)) return SFX_E_ALIGN;
  if (!aligned4(table) || !aligned4(lens) || (starts && !aligned4(starts)) || (lse && !aligned4(lse))) return SFX_E_ALIGN;
  const sfx::AttnPlan p = sfx::attn_plan(B, Hq, Hkv, max_pages * page);
  const int w = check_ws(ws, ws_bytes, sfx::attn_ws_bytes(p, B, Hkv, D));
  if (w != SFX_OK) return w;
  const auto f = qdt == SFX_F16 ? sfx::launch_attn_q4_f16 : sfx::launch_attn_q4_bf16;
  return launch_status(f((hipStream_t)stream, p, g, q, ldq * 2, cache, table, starts, lens, scale * 1.44269504088896341f,
                         out, lse, ws));
}

// ------------------------------------------------------------------------------ 8-bit layer half

int sfx_norm_q8(void* stream, int xdt, int rdt, int ydt, int T, int d, int norm, float eps, const void* x, size_t ldx,
                const void* res, size_t ldr, void* res_out, size_t ldro, const float* weight, int8_t* q, float* s, void* y,
                size_t ldy) {
  if (!dt16_or_32(xdt) || (res && !dt16_or_32(rdt)) || (y && !dt16_or_32(ydt))) return SFX_E_DTYPE;
  if (T < 1 || T > sfx::kQ8MaxTokens || d < 1 || d > (1 << 24)) return SFX_E_SHAPE;
  if (norm && !(eps > 0.f && eps < INFINITY)) return SFX_E_SHAPE;
  if ((!norm && weight) || (!res && res_out) || (q == nullptr) != (s == nullptr)) return SFX_E_SHAPE;
  if (ldx < (size_t)d || (res && ldr < (size_t)d) || (res_out && ldro < (size_t)d) || (y && ldy < (size_t)d)) return SFX_E_SHAPE;
  if (!x || (!q && !y && !res_out)) return SFX_E_NULL;
  if (!aligned_elem(x, xdt) || (res && (!aligned_elem(res, rdt) || !aligned_elem(res_out, rdt))) || (y && !aligned_elem(y, ydt)))
    return SFX_E_ALIGN;
  if ((weight && !aligned4(weight)) || (q && !aligned16(q)) || (s && !aligned4(s))) return SFX_E_ALIGN;
  return launch_status(sfx::launch_norm_q8((hipStream_t)stream, xdt, rdt, ydt, T, d, norm != 0, eps, x, ldx, res, ldr, res_out,
                                           ldro, weight, q, s, y, ldy));
}

int sfx_linear_q8(void* stream, int ydt, int T, int n, int d, const int8_t* x, size_t ldx, const float* x_scales,
                  const int8_t* W, const float* W_scales, const float* bias, int accumulate, void* y, size_t ldy) {
  if (!dt16_or_32(ydt)) return SFX_E_DTYPE;
  if (T < 1 || T > sfx::kQ8MaxTokens || n < 1 || n > (1 << 24) || d < 16 || d > 131056 || d % 16 != 0) return SFX_E_SHAPE;
  if (ldx < (size_t)d || ldy < (size_t)n) return SFX_E_SHAPE;
  if (!x || !x_scales || !W || !W_scales || !y) return SFX_E_NULL;
  if (!aligned16(x) || !aligned16(W) || ldx % 16 != 0 || !aligned_elem(y, ydt)) return SFX_E_ALIGN;
  if (!aligned4(x_scales) || !aligned4(W_scales) || (bias && !aligned4(bias))) return SFX_E_ALIGN;
  return launch_status(sfx::launch_linear_q8((hipStream_t)stream, ydt, T, n, d, x, ldx, x_scales, W, W_scales, bias,
                                             accumulate != 0, y, ldy));
}

size_t sfx_kv_cache_q8_bytes(int Hkv, int D, int page, int num_pages) {
  sfx::KvGeom g;
  if (kv_geom8(1, Hkv, D, page, num_pages, 1, &g) != SFX_OK) return 0;
  return (size_t)num_pages * Hkv * (page / 16) * (32 * (size_t)D + 16);
}

int sfx_kv_append_q8(void* stream, int xdt, int qdt, int T, int Hq, int Hkv, int D, const void* q, size_t ldq,
                     const void* k, size_t ldk, const void* v, size_t ldv, const int32_t* q_start, const int32_t* lens,
                     const float* cos_sin, int rot, int max_pos, int interleaved, int B, int max_pages,
                     const int32_t* table, int page, int num_pages, void* cache, void* q_out) {
  if (!dt16_or_32(xdt)) return SFX_E_DTYPE;
  if (q && qdt != SFX_F16 && qdt != SFX_BF16) return SFX_E_DTYPE;
  sfx::KvGeom g;
  const int st = kv_geom8(B, Hkv, D, page, num_pages, max_pages, &g);
  if (st != SFX_OK) return st;
  if (T < 1 || T > sfx::kQ8MaxTokens || (!q_start && T != B)) return SFX_E_SHAPE;
  if (q && (Hq < 1 || Hq > sfx::kAttnMaxHeads || ldq < (size_t)Hq * D)) return SFX_E_SHAPE;
  if (ldk < (size_t)Hkv * D || ldv < (size_t)Hkv * D) return SFX_E_SHAPE;
  if (cos_sin && (rot < 2 || rot > D || rot % 2 != 0 || max_pos < 1)) return SFX_E_SHAPE;
  // workgroups of 256 threads, and a launch holds fewer than 2^32 threads
  if (sfx::kv_append_q8_groups(g, T, q != nullptr) >= (1 << 24)) return SFX_E_SHAPE;
  if (!k || !v || !lens || !table || !cache || (q && !q_out)) return SFX_E_NULL;
  if (!aligned_elem(k, xdt) || !aligned_elem(v, xdt) || !aligned_elem(q, xdt) || !aligned16(cache) || ((uintptr_t)q_out & 1u))
    return SFX_E_ALIGN;
  if (!aligned4(lens) || !aligned4(table) || (q_start && !aligned4(q_start)) || (cos_sin && !aligned4(cos_sin)))
    return SFX_E_ALIGN;
  return launch_status(sfx::launch_kv_append_q8((hipStream_t)stream, g, xdt, qdt, T, q ? Hq : 0, q, ldq, k, ldk, v, ldv,
                                                q_start, lens, cos_sin, rot, max_pos, interleaved != 0, table, cache, q_out));
}

int sfx_kv_blank_q8(void* stream, int T, int n, const int32_t* q_start, const int32_t* lens, int max_pos, int max_q, int B,
                    int max_pages, const int32_t* table, int page, int num_pages, void* x) {
  sfx::KvGeom g;
  const int st = kv_geom8(B, 1, 32, page, num_pages, max_pages, &g);
  if (st != SFX_OK) return st;
  if (T < 1 || T > sfx::kQ8MaxTokens || (!q_start && T != B) || max_q < 1 || max_pos < 0) return SFX_E_SHAPE;
  if (n < 8 || n > (1 << 24) || n % 8 != 0) return SFX_E_SHAPE;
  if (!lens || !table || !x) return SFX_E_NULL;
  if (!aligned16(x) || !aligned4(lens) || !aligned4(table) || (q_start && !aligned4(q_start))) return SFX_E_ALIGN;
  return launch_status(sfx::launch_kv_blank_q8((hipStream_t)stream, g, T, n, x, q_start, lens, max_pos, max_q, table));
}

int sfx_kv_read_q8(void* stream, int odt, int T, int Hkv, int D, const int32_t* pos, const int32_t* seq, int B,
                   int max_pages, const int32_t* table, int page, int num_pages, const void* cache, void* k, void* v) {
  if (!dt16_or_32(odt)) return SFX_E_DTYPE;
  sfx::KvGeom g;
  const int st = kv_geom8(B, Hkv, D, page, num_pages, max_pages, &g);
  if (st != SFX_OK) return st;
  if (T < 1 || T > sfx::kQ8MaxTokens) return SFX_E_SHAPE;
  if (!pos || !table || !cache || !k || !v) return SFX_E_NULL;
  if (!aligned16(cache) || !aligned16(k) || !aligned16(v)) return SFX_E_ALIGN;
  if (!aligned4(pos) || !aligned4(table) || (seq && !aligned4(seq))) return SFX_E_ALIGN;
  return launch_status(sfx::launch_kv_read_q8((hipStream_t)stream, g, odt, T, pos, seq, table, cache, k, v));
}

static bool attn8_shape(int B, int max_q, int Hq, int Hkv) {
  return B >= 1 && B <= sfx::kQ8MaxSeqs && max_q >= 1 && max_q <= sfx::kQ8MaxTokens && Hkv >= 1 && Hq >= 1 &&
         Hq <= sfx::kAttnMaxHeads && Hq % Hkv == 0 && (long long)max_q * (Hq / Hkv) <= (1 << 26);
}

size_t sfx_attn_q8_ws(int B, int max_q, int Hq, int Hkv, int D, int max_len) {
  if (!attn8_shape(B, max_q, Hq, Hkv) || D < 32 || D > 256 || D % 32 != 0 || max_len < 1 || max_len > (1 << 30)) return 0;
  const sfx::Attn8Plan p = sfx::attn8_plan(B, max_q, Hq, Hkv, D, max_len);
  return sfx::attn8_fits(p, B, Hkv) ? sfx::attn8_ws_bytes(p, B, Hkv, D) : 0;
}

int sfx_attn_q8(void* stream, int qdt, int T, int B, int max_q, int Hq, int Hkv, int D, const void* q, size_t ldq,
                const int32_t* q_start, int max_pages, const int32_t* table, int page, int num_pages, const void* cache,
                const int32_t* starts, const int32_t* lens, int window, float scale, void* out, float* lse, void* ws,
                size_t ws_bytes) {
  if (qdt != SFX_F16 && qdt != SFX_BF16) return SFX_E_DTYPE;
  sfx::KvGeom g;
  const int st = kv_geom8(B, Hkv, D, page, num_pages, max_pages, &g);
  if (st != SFX_OK) return st;
  if (!attn8_shape(B, max_q, Hq, Hkv) || T < 1 || T > sfx::kQ8MaxTokens || ldq < (size_t)Hq * D) return SFX_E_SHAPE;
  if (!q_start && (T != B || max_q != 1)) return SFX_E_SHAPE;
  if (window < 0 || !(fabsf(scale) < 0x1p115f)) return SFX_E_SHAPE;
  if (!q || !table || !cache || !lens || !out) return SFX_E_NULL;
  if (!aligned16(q) || ldq % 8 != 0 || !aligned16(cache) || !aligned16(out)) return SFX_E_ALIGN;
  if (!aligned4(table) || !aligned4(lens) || (starts && !aligned4(starts)) || (q_start && !aligned4(q_start)) ||
      (lse && !aligned4(lse)))
    return SFX_E_ALIGN;
  const sfx::Attn8Plan p = sfx::attn8_plan(B, max_q, Hq, Hkv, D, max_pages * page);
  if (!sfx::attn8_fits(p, B, Hkv)) return SFX_E_SHAPE;
  const int w = check_ws(ws, ws_bytes, sfx::attn8_ws_bytes(p, B, Hkv, D));
  if (w != SFX_OK) return w;
  const auto f = qdt == SFX_F16 ? sfx::launch_attn_q8_f16 : sfx::launch_attn_q8_bf16;
  return launch_status(f((hipStream_t)stream, p, g, T, max_q, q, ldq * 2, q_start, cache, table, starts, lens, window,
                         scale * 1.44269504088896341f, out, lse, ws));
}

// ------------------------------------------------------------------------------ measurement helper

int sfx_stream_read(void* stream, const void* buf, size_t nbytes, uint32_t* out) {
  if (nbytes < 16 || nbytes % 16 != 0) return SFX_E_SHAPE;
  if (!buf || !out) return SFX_E_NULL;
  if (!aligned16(buf) || !aligned4(out)) return SFX_E_ALIGN;
  return launch_status(sfx::launch_stream_read((hipStream_t)stream, buf, nbytes, out));
}

}  // extern "C"
