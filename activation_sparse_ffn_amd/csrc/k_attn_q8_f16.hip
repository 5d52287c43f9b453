// Attention over the int8 cache, f16 queries.
#include "k_attn_q8.hpp"

namespace sfx {

hipError_t launch_attn_q8_f16(hipStream_t s, const Attn8Plan& p, const KvGeom& g, int T, int max_q, const void* q,
                            size_t ldq_bytes, const int32_t* q_start, const void* cache, const int32_t* table,
                            const int32_t* starts, const int32_t* lens, int window, float k2, void* out, float* lse,
                            void* ws) {
  const KvCache kv{(uint8_t*)cache, table, g.Hkv, g.D, g.page_shift, g.num_pages, g.max_pages, g.B};
  const Attn8Args a{kv, {q_start, lens, T, max_q}, (const uint8_t*)q, ldq_bytes, starts, (uint8_t*)out, lse, (float*)ws,
                    k2, p.Hq, p.G, window, p.RT, p.S};
  return attn8_launch<TF16>(s, a, p.R);
}

}  // namespace sfx
