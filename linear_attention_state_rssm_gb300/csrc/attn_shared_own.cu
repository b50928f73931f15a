// The kernels of the second launch of attention over shared prefixes: the rows' own keys
// (attn_decode.cuh), unquantised pages.
#include "attn_decode.cuh"

namespace rssm {

cudaError_t attn_shared_own(const DecodeParams* p, const void* maps, int D, int dt, int rows,
                            int sms, cudaStream_t st) {
  if (dt == DT_F32) return decode_any<float, false, DEC_OWN>(p, maps, D, rows, sms, st);
  if (dt == DT_BF16) return decode_any<__nv_bfloat16, false, DEC_OWN>(p, maps, D, rows, sms, st);
  return decode_any<__half, false, DEC_OWN>(p, maps, D, rows, sms, st);
}

}  // namespace rssm
