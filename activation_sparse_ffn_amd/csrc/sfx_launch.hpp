// Internal launchers, one per kernel family.  Arguments are already validated by
// the C ABI layer; each launcher only picks an instantiation and enqueues it.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/sfx.h"

namespace sfx {

int device_cu_count();  // cached per device; 0 if no device

size_t predict_ws_bytes(int wdt, int B, int d, int h, int f);
hipError_t launch_predict(hipStream_t s, int wdt, int B, int d, int h, int f, const void* x,
                          const void* W1, const void* W2, float* scores, void* ws);

hipError_t launch_predict_q4(hipStream_t s, int B, int d, int h, int f, const void* x, const void* W1,
                             const void* W1_s, const void* W2, const void* W2_s, float* scores, void* ws);

size_t compact_ws_bytes(int B, int f);
hipError_t launch_compact(hipStream_t s, int B, int f, const float* scores, float t,
                          uint32_t* tok_bits, uint32_t* union_bits, int32_t* idx, int kmax,
                          int32_t* count, void* ws);

hipError_t launch_up(hipStream_t s, int wdt, int act, int B, int d, int f, const void* x,
                     const void* Wa, const void* Wa_s, const float* ba, const void* Wl,
                     const void* Wl_s, const int32_t* idx, const int32_t* count, int kmax,
                     float* hact);
bool up_supported(int wdt, int act, int B);

size_t down_ws_bytes(int wdt, int B, int d, int kmax);
hipError_t launch_down(hipStream_t s, int wdt, int B, int d, int f, const void* Wd,
                       const void* Wd_s, const int32_t* idx, const int32_t* count, int kmax,
                       const float* hact, float* y, void* ws);
bool down_supported(int wdt, int B);
size_t dense_ws_bytes(int wdt, int B, int d, int f);
hipError_t launch_dense(hipStream_t s, int wdt, int act, int B, int d, int f, const void* x, const void* Wa,
                        const void* Wa_s, const float* ba, const void* Wl, const void* Wl_s, const void* Wd,
                        const void* Wd_s, float* hact, float* y, void* ws);
// Static scratch of the down kernel for callers that cannot allocate: its size, and
// its device address on the current device (looked up on the first call per device).
constexpr size_t kDownScratchBytes = SFX_DOWN_SCRATCH_BYTES;
hipError_t down_scratch(void** ptr);

size_t stream_read_out_words();
hipError_t launch_stream_read(hipStream_t s, const void* buf, size_t nbytes, uint32_t* out);

size_t tam_ws_bytes(int G, int K);
hipError_t launch_tam(hipStream_t s, int L, int G, const uint32_t* union_bits, float lambda,
                      float eps, int K, float* score, uint32_t* hot_bits, uint32_t* entered,
                      uint32_t* left, int32_t* topk, int32_t* topk_count);
hipError_t launch_topk_now(hipStream_t s, int L, int G, const uint32_t* union_bits, int K, uint32_t* hot_bits,
                           uint32_t* entered, uint32_t* left, int32_t* topk, int32_t* topk_count);

hipError_t launch_count_active(hipStream_t s, int B, int f, const uint32_t* tok_bits, int32_t* counts);
size_t select_ws_bytes();
hipError_t launch_select_kth(hipStream_t s, size_t n, const float* v, size_t k, float* out, void* ws);
size_t order_ws_bytes(int f);
hipError_t launch_hot_first_order(hipStream_t s, int f, const int32_t* counts, const int32_t* group, int32_t* perm,
                                  void* ws);
hipError_t launch_gather_rows(hipStream_t s, int n_dst, int n_src, size_t row_bytes, const void* src,
                              const int32_t* idx, void* dst);

constexpr int kHotMaxMats = 8;
constexpr int kHotMaxLayers = 1024;
constexpr int kHotChunk = 16384;         // bytes per work item of the copy kernel
struct HotMats {
  int n;                                 // matrices per layer, 0..kHotMaxMats
  size_t group_bytes[kHotMaxMats];       // bytes of one group's rows in matrix m
  int chunk_off[kHotMaxMats + 1];        // first chunk of matrix m; chunk_off[n] = chunks per group
};
hipError_t launch_hot_assign(hipStream_t s, int L, int G, int K, const uint32_t* entered, const uint32_t* left,
                             int32_t* slot_of, int32_t* group_of, int32_t* copies, int32_t* ncopies);
hipError_t launch_hot_copy(hipStream_t s, int L, int K, const HotMats& mats, const void* const* src,
                           void* const* dst, const int32_t* copies, const int32_t* ncopies);

// Int4 projection (gsh = log2(group / 32)).
hipError_t launch_linear_q4_f16(hipStream_t s, int gsh, int B, int n, int d, const void* x, size_t ldx_bytes,
                                const void* W, const void* Ws, const float* bias, int accumulate, float* y, size_t ldy);
hipError_t launch_linear_q4_bf16(hipStream_t s, int gsh, int B, int n, int d, const void* x, size_t ldx_bytes,
                                 const void* W, const void* Ws, const float* bias, int accumulate, float* y,
                                 size_t ldy);

// Paged int4 key/value cache.  Tokens of a call: one workgroup column of 256 threads per token,
// and a launch holds fewer than 2^32 threads in x.
constexpr int kKvMaxTokens = (1 << 24) - 1;
struct KvGeom {
  int B, Hkv, D, page_shift, num_pages, max_pages;
};
hipError_t launch_kv_append_q4(hipStream_t s, const KvGeom& g, int xdt, int qdt, int T, int Hq, const void* q, size_t ldq,
                               const void* k, size_t ldk, const void* v, size_t ldv, const int32_t* pos,
                               const int32_t* seq, const float* cos_sin, int rot, int max_pos, int pairs,
                               const int32_t* table, void* cache, void* q_out);
hipError_t launch_kv_read_q4(hipStream_t s, const KvGeom& g, int odt, int T, const int32_t* pos, const int32_t* seq,
                             const int32_t* table, const void* cache, void* k, void* v);
hipError_t launch_kv_lens_q4(hipStream_t s, const KvGeom& g, const int32_t* pos, int max_pos, int window,
                             const int32_t* table, int32_t* lens, int32_t* starts);

// Decode attention: heads per workgroup and the number of runs a sequence is split into.
struct AttnPlan {
  int Hq, G, HT, HG, S;      // query heads, per kv head, tiles of 16 of those, heads of a full tile, runs
};
constexpr int kAttnMaxHeads = 256;
AttnPlan attn_plan(int B, int Hq, int Hkv, int max_len);
size_t attn_ws_bytes(const AttnPlan& p, int B, int Hkv, int D);
hipError_t launch_attn_q4_f16(hipStream_t s, const AttnPlan& p, const KvGeom& g, const void* q, size_t ldq_bytes,
                              const void* cache, const int32_t* table, const int32_t* starts, const int32_t* lens,
                              float k2, void* out, float* lse, void* ws);
hipError_t launch_attn_q4_bf16(hipStream_t s, const AttnPlan& p, const KvGeom& g, const void* q, size_t ldq_bytes,
                               const void* cache, const int32_t* table, const int32_t* starts, const int32_t* lens,
                               float k2, void* out, float* lse, void* ws);

// The 8-bit layer half: rows (tokens) and sequences of a call.
constexpr int kQ8MaxTokens = 1 << 20;
constexpr int kQ8MaxSeqs = 4096;
hipError_t launch_norm_q8(hipStream_t s, int xdt, int rdt, int ydt, int T, int d, int norm, float eps, const void* x,
                          size_t ldx, const void* r, size_t ldr, void* r_out, size_t ldro, const float* w, int8_t* q,
                          float* sc, void* y, size_t ldy);
hipError_t launch_linear_q8(hipStream_t s, int ydt, int T, int n, int d, const int8_t* x, size_t ldx, const float* sx,
                            const int8_t* W, const float* sw, const float* bias, int accumulate, void* y, size_t ldy);
long long kv_append_q8_groups(const KvGeom& g, int T, bool queries);      // workgroups of the append
hipError_t launch_kv_append_q8(hipStream_t s, const KvGeom& g, int xdt, int qdt, int T, int Hq, const void* q, size_t ldq,
                               const void* k, size_t ldk, const void* v, size_t ldv, const int32_t* q_start,
                               const int32_t* lens, const float* cos_sin, int rot, int max_pos, int pairs,
                               const int32_t* table, void* cache, void* q_out);
hipError_t launch_kv_blank_q8(hipStream_t s, const KvGeom& g, int T, int n, void* x, const int32_t* q_start,
                              const int32_t* lens, int max_pos, int max_q, const int32_t* table);
hipError_t launch_kv_read_q8(hipStream_t s, const KvGeom& g, int odt, int T, const int32_t* pos, const int32_t* seq,
                             const int32_t* table, const void* cache, void* k, void* v);

// Rows of a workgroup of the kernel for many of them, D = 32 NG.  256 share the decoding (8192 tokens
// of 32/8 heads of 128: 581 us and 621 by 128 when both were there, 566 now).  Where that is little, at heads of 32 and 64, three workgroups of 128
// fit a compute unit and do not hold each other up (heads of 64, 4096 tokens: 201 us, 217 by 256).  From heads of 160 on a
// wave needs the registers of a SIMD for itself and the two buffers most of the LDS: one workgroup of four waves
// (heads of 256, 4096 tokens: 249 us, 323 by 256).
constexpr int attn8_rows(int NG) { return NG == 3 || NG == 4 ? 256 : 128; }
// Attention over the int8 cache: query heads, per kv head, rows of a tile (16, 32 or attn8_rows), tiles
// of rows, runs of positions that a tile is cut into.
struct Attn8Plan {
  int Hq, G, R, RT, S;
};
Attn8Plan attn8_plan(int B, int max_q, int Hq, int Hkv, int D, int max_len);
size_t attn8_ws_bytes(const Attn8Plan& p, int B, int Hkv, int D);
hipError_t launch_attn_q8_f16(hipStream_t s, const Attn8Plan& p, const KvGeom& g, int T, int max_q, const void* q,
                              size_t ldq_bytes, const int32_t* q_start, const void* cache, const int32_t* table,
                              const int32_t* starts, const int32_t* lens, int window, float k2, void* out, float* lse,
                              void* ws);
hipError_t launch_attn_q8_bf16(hipStream_t s, const Attn8Plan& p, const KvGeom& g, int T, int max_q, const void* q,
                               size_t ldq_bytes, const int32_t* q_start, const void* cache, const int32_t* table,
                               const int32_t* starts, const int32_t* lens, int window, float k2, void* out, float* lse,
                               void* ws);

}  // namespace sfx
