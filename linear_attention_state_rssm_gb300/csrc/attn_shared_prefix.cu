// The kernels of the first launch of attention over shared prefixes: the prefixes
// (attn_decode.cuh), fp32 pages.
#include "attn_decode.cuh"

namespace rssm {

cudaError_t attn_shared_prefix(const DecodeParams* p, const void* maps, int D, int dt, int rows,
                               int sms, cudaStream_t st) {
  if (dt != DT_F32) return cudaErrorInvalidValue;  // attn_shared_tc.cu
  return decode_any<float, false, DEC_PREFIX>(p, maps, D, rows, sms, st);
}

}  // namespace rssm
