// Paged int4 key/value cache: layout shared by the append, read and attention kernels.
//
// One layer's cache is [pages][Hkv][page / 8][9 D] bytes.  A block of 9 D bytes holds 8
// consecutive positions of one kv head (NG = D / 32 groups):
//   K codes  4 D bytes  per position D / 2 bytes = words [c = 0..3][g < NG]; word (c, g)
//            holds dims 32 g + 8 c + 2 j and + 2 j + 1 in nibbles j and j + 4: the eight
//            numbers a lane of quarter c feeds to the product of group g;
//   V codes  4 D bytes  [n = 0..15][g][8 bytes]; the byte of position i is number
//            kv_byte(i), dims 32 g + n (low nibble) and 32 g + 16 + n: a register of
//            two bytes two apart is two neighbouring positions of one dim;
//   scales   fp16 [g][8 positions] of K, then of V.
// Codes are q + 8.  Everything a wave reads for 32 positions is four such blocks.
#pragma once
#include "sfx_common.hpp"

namespace sfx {

__host__ __device__ constexpr int kv_block_bytes(int D) { return 9 * D; }
__device__ __forceinline__ int kv_byte(int i) { return (i & 4) | ((i & 1) << 1) | ((i >> 1) & 1); }

struct KvCache {
  uint8_t* base;
  const int32_t* table;     // [B][max_pages]
  int Hkv, D, page_shift, num_pages, max_pages, B;
};

// Page id of position p (>= 0) of sequence b, or -1 where there is none.
__device__ __forceinline__ int kv_page(const KvCache& kv, int b, int p) {
  const int j = p >> kv.page_shift;
  if (j >= kv.max_pages) return -1;
  const int id = kv.table[(size_t)b * kv.max_pages + j];
  return (unsigned)id < (unsigned)kv.num_pages ? id : -1;
}
// Block of octet `o` of page `id`, head h.
__device__ __forceinline__ size_t kv_block(const KvCache& kv, int id, int h, int o) {
  return ((((size_t)id * kv.Hkv + h) << (kv.page_shift - 3)) + o) * (size_t)kv_block_bytes(kv.D);
}

}  // namespace sfx
