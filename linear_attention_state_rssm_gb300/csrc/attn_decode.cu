// Attention of new tokens over the pages: choice of the kernel, tensor maps of
// the pool, launches; the kernels of unquantised pages (attn_decode.cuh).
#include "attn_decode.cuh"

namespace rssm {

namespace {

// warps that share a stream's keys, sixteen rows each
int warps_for(int D, int dt, int rows) {
  if (dt == DT_F32 || rows <= 16) return 1;
  return rows <= 32 ? 2 : D == 256 ? 3 : 4;
}

cudaError_t plain(const DecodeParams* p, const void* maps, int D, int dt, int mw, int sms,
                  cudaStream_t st) {
  if (dt == DT_F32) return decode_any<float, false, DEC_PLAIN>(p, maps, D, mw, sms, st);
  if (dt == DT_BF16) return decode_any<__nv_bfloat16, false, DEC_PLAIN>(p, maps, D, mw, sms, st);
  return decode_any<__half, false, DEC_PLAIN>(p, maps, D, mw, sms, st);
}

}  // namespace

int attn_decode_block_rows(int D, int dt, int rows) { return 16 * warps_for(D, dt, rows); }

cudaError_t attn_decode_prepare(int D, int dt, bool quant) {
  return quant ? attn_decode_quant(nullptr, nullptr, D, dt, 0, 0, nullptr)
               : plain(nullptr, nullptr, D, dt, 0, 0, nullptr);
}

// The pool as rows of 128-byte columns: a box is sixteen tokens of one head.
// Quantised heads of 64 have rows of 64 bytes.
cudaError_t attn_decode_maps(void* maps, const void* k, const void* v, long long rows, int D,
                             int dt, bool quant) {
  static_assert(sizeof(KvMaps) == kKvMapBytes, "two tensor maps");
  if (tma_encoder() == nullptr) return cudaErrorNotSupported;
  const cuuint64_t es = quant ? 1 : dtype_bytes(dt), bytes = D * es;
  const cuuint64_t column = bytes < 128 ? bytes : 128, inner = column / es;
  const cuuint64_t dims[3] = {inner, (cuuint64_t)rows, bytes / column};
  const cuuint64_t strides[2] = {bytes, column};
  const cuuint32_t box[3] = {(cuuint32_t)inner, kBox, (cuuint32_t)(bytes / column)};
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
  const int mw = warps_for(D, dt, p.T * p.G);
  return p.scales != nullptr ? attn_decode_quant(&p, maps, D, dt, mw, sms, st)
                             : plain(&p, maps, D, dt, mw, sms, st);
}

// Shared prefixes: a stream of one warp where all the batch's query rows of a key
// head are sixteen at most, else of as many as there are.
cudaError_t attn_shared_prepare(int D, int dt, bool quant) {
  const cudaError_t e = quant ? attn_shared_prefix_quant(nullptr, nullptr, D, dt, 0, 0, nullptr)
                              : attn_shared_prefix(nullptr, nullptr, D, dt, 0, 0, nullptr);
  if (e != cudaSuccess) return e;
  return quant ? attn_shared_own_quant(nullptr, nullptr, D, dt, 0, 0, nullptr)
               : attn_shared_own(nullptr, nullptr, D, dt, 0, 0, nullptr);
}

cudaError_t attn_shared_launch(DecodeParams p, const void* maps, int D, int dt, int num_sms,
                               cudaStream_t st) {
  const int sms = num_sms < kMaxSms ? num_sms : kMaxSms;
  const bool quant = p.scales != nullptr;
  const int most = dt == DT_F32 ? 1 : D == 256 ? 3 : 4;
  const int all = (long long)p.B * p.T * p.G <= 16 ? 1 : most;
  const int own = p.T * p.G <= 16 ? 1 : most;
  const cudaError_t e = quant ? attn_shared_prefix_quant(&p, maps, D, dt, all, sms, st)
                              : attn_shared_prefix(&p, maps, D, dt, all, sms, st);
  if (e != cudaSuccess) return e;
  p.nmb = (p.T * p.G + 16 * own - 1) / (16 * own);
  return quant ? attn_shared_own_quant(&p, maps, D, dt, own, sms, st)
               : attn_shared_own(&p, maps, D, dt, own, sms, st);
}

}  // namespace rssm
