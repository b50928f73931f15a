// As attn_shared_own.cu, for quantised pages.
#include "attn_decode.cuh"

namespace rssm {

cudaError_t attn_shared_own_quant(const DecodeParams* p, const void* maps, int D, int dt, int rows,
                                   int sms, cudaStream_t st) {
  return dt == DT_BF16 ? decode_any<__nv_bfloat16, true, DEC_OWN>(p, maps, D, rows, sms, st)
                       : decode_any<__half, true, DEC_OWN>(p, maps, D, rows, sms, st);
}

}  // namespace rssm
