// As attn_shared_prefix.cu, for quantised pages of fp16 caches.
#include "attn_decode.cuh"

namespace rssm {

cudaError_t attn_shared_prefix_quant(const DecodeParams* p, const void* maps, int D, int dt, int rows,
                                   int sms, cudaStream_t st) {
  if (dt != DT_F16) return cudaErrorInvalidValue;  // attn_shared_tc.cu
  return decode_any<__half, true, DEC_PREFIX>(p, maps, D, rows, sms, st);
}

}  // namespace rssm
