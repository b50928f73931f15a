// Attention over shared prefixes on the 5th-generation tensor cores: tensor maps
// of the pool and launches (attn_shared_tc.cuh).
#include "attn_shared_tc.cuh"

namespace rssm {

// Boxes of one column of up to 128 tokens: 64 16-bit values under the 128-byte
// swizzle that the products read, or up to 128 codes as they are.
cudaError_t attn_shared_tc_maps(void* maps, const void* k, const void* v, long long rows, int D,
                                int dt, bool quant, int page_size) {
  static_assert(sizeof(SharedTcMaps) == kKvMapBytes, "two tensor maps");
  if (tma_encoder() == nullptr) return cudaErrorNotSupported;
  const cuuint64_t bytes = quant ? D : 2 * D, column = bytes < 128 ? bytes : 128;
  const cuuint64_t inner = quant ? column : 64;
  const cuuint64_t dims[3] = {inner, (cuuint64_t)rows, bytes / column};
  const cuuint64_t strides[2] = {bytes, column};
  const cuuint32_t box[3] = {(cuuint32_t)inner, (cuuint32_t)(page_size < 128 ? page_size : 128), 1};
  const cuuint32_t ones[3] = {1, 1, 1};
  SharedTcMaps* m = static_cast<SharedTcMaps*>(maps);
  for (int i = 0; i < 2; ++i) {
    if (tma_encoder()(i == 0 ? &m->k : &m->v,
                      quant           ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                      : dt == DT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                      : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                      3, const_cast<void*>(i == 0 ? k : v), dims, strides, box, ones,
                      CU_TENSOR_MAP_INTERLEAVE_NONE,
                      quant ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
                      CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  return cudaSuccess;
}

cudaError_t attn_shared_tc_prefix(const DecodeParams* p, const void* maps, int D, int dt,
                                  bool quant, cudaStream_t st) {
  // every block of a group has a part behind the last of an even split
  long long ctas = 0;
  if (p != nullptr) {
    ctas = share_segments(p->B, p->T, p->G, p->HKV);
    if (ctas > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  }
  const int n = (int)ctas;
  if (dt == DT_BF16)
    return quant ? shared_tc_any<__nv_bfloat16, true>(p, maps, D, n, st)
                 : shared_tc_any<__nv_bfloat16, false>(p, maps, D, n, st);
  return quant ? shared_tc_any<__half, true>(p, maps, D, n, st)
               : shared_tc_any<__half, false>(p, maps, D, n, st);
}

}  // namespace rssm
