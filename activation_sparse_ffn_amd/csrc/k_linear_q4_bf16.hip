// Int4 projection, bf16 inputs.
#include "k_linear_q4.hpp"

namespace sfx {

hipError_t launch_linear_q4_bf16(hipStream_t s, int gsh, int B, int n, int d, const void* x, size_t ldx_bytes,
                              const void* W, const void* Ws, const float* bias, int accumulate, float* y, size_t ldy) {
  const LinearArgs a{(const uint8_t*)x, ldx_bytes, (const uint8_t*)W, (const uint16_t*)Ws, bias, y, ldy, B, n, d,
                     accumulate};
  return lin_launch<TBF16>(s, a, gsh);
}

}  // namespace sfx
