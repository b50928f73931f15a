// Attention of new tokens over the pages: choice of the kernel, tensor maps of
// the pool, launches; the kernels of unquantised pages (attn_decode.cuh).
#include "attn_decode.cuh"

namespace rssm {

namespace {

cudaError_t plain(const DecodeParams* p, const void* maps, int D, int dt, int rows, int sms,
                  cudaStream_t st) {
  if (dt == DT_F32) return decode_any<float, false, DEC_PLAIN>(p, maps, D, rows, sms, st);
  if (dt == DT_BF16) return decode_any<__nv_bfloat16, false, DEC_PLAIN>(p, maps, D, rows, sms, st);
  return decode_any<__half, false, DEC_PLAIN>(p, maps, D, rows, sms, st);
}

}  // namespace

// Rows of a block for `rows` query rows of a row of the batch and a key head.
int attn_decode_block_rows(int D, int dt, bool quant, int rows) {
  if (dt == DT_F32 || rows <= 16) return quant && rows <= 8 ? 8 : 16;
  return rows <= 32 ? 32 : D == 256 ? 48 : 64;
}

cudaError_t attn_decode_prepare(int D, int dt, bool quant) {
  return quant ? attn_decode_quant(nullptr, nullptr, D, dt, 0, 0, nullptr)
               : plain(nullptr, nullptr, D, dt, 0, 0, nullptr);
}

// The pool as rows of 128-byte columns: a box is sixteen tokens of one head. Of
// quantised pages it is 32 where a page has them, else one column of sixteen;
// heads of 64 have rows of 64 bytes there.
cudaError_t attn_decode_maps(void* maps, const void* k, const void* v, long long rows, int D,
                             int dt, bool quant, int page_size) {
  static_assert(sizeof(KvMaps) == kKvMapBytes, "two tensor maps");
  if (tma_encoder() == nullptr) return cudaErrorNotSupported;
  const cuuint64_t es = quant ? 1 : dtype_bytes(dt), bytes = D * es;
  const cuuint64_t column = bytes < 128 ? bytes : 128, inner = column / es;
  const cuuint64_t dims[3] = {inner, (cuuint64_t)rows, bytes / column};
  const cuuint64_t strides[2] = {bytes, column};
  const bool wide = quant && page_size >= kQuantBox;
  const cuuint32_t box[3] = {(cuuint32_t)inner, (cuuint32_t)(wide ? kQuantBox : kBox),
                             quant && !wide ? 1 : (cuuint32_t)(bytes / column)};
  const cuuint32_t ones[3] = {1, 1, 1};
  KvMaps* m = static_cast<KvMaps*>(maps);
  for (int i = 0; i < 2; ++i) {
    if (tma_encoder()(i == 0 ? &m->k : &m->v,
                      quant           ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                      : dt == DT_F32  ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                      : dt == DT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                      : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                      3, const_cast<void*>(i == 0 ? k : v), dims, strides, box, ones,
                      CU_TENSOR_MAP_INTERLEAVE_NONE,
                      column == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                      CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  return cudaSuccess;
}

cudaError_t attn_decode_launch(const DecodeParams& p, const void* maps, int D, int dt, int num_sms,
                               cudaStream_t st) {
  const int sms = num_sms < kMaxSms ? num_sms : kMaxSms;
  const int rows = attn_decode_block_rows(D, dt, p.scales != nullptr, p.T * p.G);
  return p.scales != nullptr ? attn_decode_quant(&p, maps, D, dt, rows, sms, st)
                             : plain(&p, maps, D, dt, rows, sms, st);
}

// Shared prefixes: on the 5th-generation tensor cores, fp32 ones by the kernel of
// single rows with a group's query rows in its blocks.
cudaError_t attn_shared_prepare(int D, int dt, bool quant) {
  const cudaError_t e = dt == DT_F32
                            ? attn_shared_prefix(nullptr, nullptr, D, dt, 0, 0, nullptr)
                            : attn_shared_tc_prefix(nullptr, nullptr, D, dt, quant, nullptr);
  if (e != cudaSuccess) return e;
  return quant ? attn_shared_own_quant(nullptr, nullptr, D, dt, 0, 0, nullptr)
               : attn_shared_own(nullptr, nullptr, D, dt, 0, 0, nullptr);
}

cudaError_t attn_shared_launch(DecodeParams p, const void* maps, const void* tc_maps, int D,
                               int dt, int num_sms, cudaStream_t st) {
  const int sms = num_sms < kMaxSms ? num_sms : kMaxSms;
  const bool quant = p.scales != nullptr;
  p.cut = dt != DT_F32;
  const cudaError_t e = dt == DT_F32 ? attn_shared_prefix(&p, maps, D, dt, 16, sms, st)
                                     : attn_shared_tc_prefix(&p, tc_maps, D, dt, quant, st);
  if (e != cudaSuccess) return e;
  // OWN has no blocks of 32 rows over unquantised pages (decode_of_size)
  int own = attn_decode_block_rows(D, dt, quant, p.T * p.G);
  if (own == 32 && !quant) own = D == 256 ? 48 : 64;
  p.nmb = (p.T * p.G + own - 1) / own;
  return quant ? attn_shared_own_quant(&p, maps, D, dt, own, sms, st)
               : attn_shared_own(&p, maps, D, dt, own, sms, st);
}

}  // namespace rssm
