// Paged int8 key/value cache: layout shared by the append, read and attention kernels, and
// which rows of a call belong to which sequence.
//
// One layer's cache is [pages][Hkv][page / 16][32 D + 16] bytes.  A block holds 16 consecutive
// positions of one kv head.  A code is stored as u = q + 128, a value is q * scale:
//   K codes  16 D bytes  [16 positions][D]: 16 bytes of a position are what a lane feeds to the
//            product of 32 dims, twice;
//   V codes  16 D bytes  [4][D][4]: byte i of dim d in quarter c is position 4 c + i, so a
//            word is four neighbouring positions of one dim, as the second product wants them;
//   scales   fp32 of K, fp32 of V, 8 bytes unused.
#pragma once
#include "sfx_kv.hpp"

namespace sfx {

constexpr int kBlk8 = 16;
__host__ __device__ constexpr int kv8_block_bytes(int D) { return 32 * D + 16; }

// Block `o` of page `id`, head h.
__device__ __forceinline__ size_t kv8_block(const KvCache& kv, int id, int h, int o) {
  return ((((size_t)id * kv.Hkv + h) << (kv.page_shift - 4)) + o) * (size_t)kv8_block_bytes(kv.D);
}

// Rows of a call: sequence b has rows first .. first + n - 1, the last n of its `len` positions.
// Without offsets row b is sequence b's last position.  A sequence with n > len has rows in front
// of position 0: they have no position.  Of a sequence with more than `most` rows the first ones are taken, at
// the positions that they have among all.
struct Rows8 {
  const int32_t *start, *lens;   // [B + 1] or null; [B]
  int T, most;                   // rows of the call, at most `most` of a sequence
};
struct Seq8 {
  int first, n, len;
  int pos;                       // position of row `first`
};
__device__ __forceinline__ Seq8 rows8_seq(const Rows8& r, int b) {
  Seq8 s;
  s.len = max(r.lens[b], 0);                 // may pass the table: positions without a page
  if (!r.start) {
    s.first = b;
    s.n = 1;
    s.pos = s.len - 1;
  } else {
    s.first = min(max(r.start[b], 0), r.T);
    const int all = min(max(r.start[b + 1] - s.first, 0), r.T - s.first);
    s.n = min(all, r.most);
    s.pos = s.len - all;
  }
  return s;
}

}  // namespace sfx
