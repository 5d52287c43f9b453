// Decode attention over the int4 cache, f16 queries.
#include "k_attn_q4.hpp"

namespace sfx {

hipError_t launch_attn_q4_f16(hipStream_t s, const AttnPlan& p, const KvGeom& g, const void* q, size_t ldq_bytes,
                            const void* cache, const int32_t* table, const int32_t* starts, const int32_t* lens,
                            float k2, void* out, float* lse, void* ws) {
  const KvCache kv{(uint8_t*)cache, table, g.Hkv, g.D, g.page_shift, g.num_pages, g.max_pages, g.B};
  const AttnArgs a{kv, (const uint8_t*)q, ldq_bytes, starts, lens, (uint8_t*)out, lse, (float*)ws, k2,
                   p.Hq, p.G, p.HT, p.HG, p.S};
  return attn_launch<TF16>(s, a);
}

}  // namespace sfx
