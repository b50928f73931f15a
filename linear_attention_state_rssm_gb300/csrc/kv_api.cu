// C ABI of the full-attention layers' operators: host-side validation and
// launches. See include/rssm.h for the contract of every entry point.
#include <cmath>
#include <new>

#include "../../include/rssm.h"
#include "kv_common.cuh"

using namespace rssm;

struct rssm_kv_handle {
  rssm_kv_config cfg;
  rssm_kv_buffers buf;
  int num_sms;
  int shift;            // log2(page_size)
  size_t layer_bytes;   // one layer's keys (or values)
  size_t page_bytes;    // one page of one layer's keys (or values)
  int hook_cta, hook_unit;  // test hook of the bounded waits; -1: off
  alignas(64) unsigned char maps[kKvMapBytes];  // the pool's tensor maps
};

namespace {

constexpr int kMaxRows = 65535;
constexpr int kMaxWindow = 1 << 20;

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

rssm_status from_cuda(cudaError_t e) { return e == cudaSuccess ? RSSM_OK : RSSM_ERR_CUDA; }

rssm_status check_config(const rssm_kv_config* c) {
  if (c == nullptr) return RSSM_ERR_INVALID_ARG;
  if (c->n_layers < 1 || c->n_slots < 1 || c->HQ < 1 || c->HKV < 1 || c->D < 1 ||
      c->n_pages < 1 || c->page_size < 1 || c->max_pages < 1)
    return RSSM_ERR_INVALID_ARG;
  if (c->HQ % c->HKV != 0) return RSSM_ERR_INVALID_ARG;
  if (c->dtype != RSSM_F32 && c->dtype != RSSM_BF16 && c->dtype != RSSM_F16)
    return RSSM_ERR_INVALID_ARG;
  if (!std::isfinite(c->scale) || !(c->scale > 0.f)) return RSSM_ERR_INVALID_ARG;
  if (c->D != 64 && c->D != 128 && c->D != 256) return RSSM_ERR_UNSUPPORTED;
  if (c->HQ / c->HKV > 64 || c->HQ > 4096) return RSSM_ERR_UNSUPPORTED;
  if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1)) != 0)
    return RSSM_ERR_UNSUPPORTED;
  // token positions are 32-bit, and a plan's sums over rows too
  // and the pool's rows (one token of one head) are addressed in 31 bits
  if ((long long)c->n_layers * c->n_pages * c->HKV > 0x7fffffffll / c->page_size)
    return RSSM_ERR_UNSUPPORTED;
  if (c->n_pages > (1 << 28) || c->max_pages > (1 << 20)) return RSSM_ERR_UNSUPPORTED;
  return RSSM_OK;
}

size_t page_bytes(const rssm_kv_config& c) {
  return (size_t)c.HKV * c.page_size * c.D * dtype_bytes(c.dtype);
}

rssm_status check_rows(const rssm_kv_handle* h, const int32_t* slot, int32_t B) {
  if (h == nullptr || B < 0 || B > kMaxRows) return RSSM_ERR_INVALID_ARG;
  if (B > 0 && (slot == nullptr || !aligned4(slot))) return RSSM_ERR_INVALID_ARG;
  return RSSM_OK;
}

// A view of tokens: 16-byte aligned rows of `heads` heads, `stride` elements apart.
bool tokens_ok(const rssm_kv_config& c, const void* p, int64_t stride, int heads) {
  return p != nullptr && aligned16(p) && stride >= (int64_t)heads * c.D &&
         (stride * dtype_bytes(c.dtype)) % 16 == 0 && stride <= ((int64_t)1 << 31);
}

PageParams page_params(const rssm_kv_handle* h) {
  const KvWork w(h->cfg.n_pages);
  char* work = static_cast<char*>(h->buf.work);
  PageParams p{};
  p.table = h->buf.table;
  p.held = h->buf.held;
  p.length = h->buf.length;
  p.refs = h->buf.refs;
  p.err = h->buf.err_word;
  p.moves = reinterpret_cast<int32_t*>(work + w.moves);
  p.src = reinterpret_cast<int32_t*>(work + w.src);
  p.dst = reinterpret_cast<int32_t*>(work + w.dst);
  p.map = reinterpret_cast<int32_t*>(work + w.map);
  p.rows = reinterpret_cast<int32_t*>(work + w.rows);
  p.n_slots = h->cfg.n_slots;
  p.n_pages = h->cfg.n_pages;
  p.max_pages = h->cfg.max_pages;
  p.shift = h->shift;
  return p;
}

rssm_status copy_pages(const rssm_kv_handle* h, const PageParams& p, bool remap,
                       cudaStream_t st) {
  CopyParams c{};
  c.k = static_cast<unsigned char*>(h->buf.k_pages);
  c.v = static_cast<unsigned char*>(h->buf.v_pages);
  c.moves = p.moves;
  c.src = p.src;
  c.dst = p.dst;
  c.map = remap ? p.map : nullptr;
  c.table = p.table;
  c.page_bytes = h->page_bytes;
  c.layer_bytes = h->layer_bytes;
  c.table_size = (size_t)h->cfg.n_slots * h->cfg.max_pages;
  c.n_layers = h->cfg.n_layers;
  c.n_pages = h->cfg.n_pages;
  return from_cuda(kv_copy_launch(c, h->num_sms, st));
}

}  // namespace

extern "C" {

rssm_status rssm_kv_required_bytes(const rssm_kv_config* cfg, rssm_kv_sizes* out) {
  const rssm_status st = check_config(cfg);
  if (st != RSSM_OK) return st;
  if (out == nullptr) return RSSM_ERR_INVALID_ARG;
  out->k_pages = out->v_pages = (size_t)cfg->n_layers * cfg->n_pages * page_bytes(*cfg);
  out->table = (size_t)cfg->n_slots * cfg->max_pages * 4;
  out->held = out->length = (size_t)cfg->n_slots * 4;
  out->refs = (size_t)cfg->n_pages * 4;
  out->work = KvWork(cfg->n_pages).total;
  out->err_word = 4;
  return RSSM_OK;
}

rssm_status rssm_kv_alloc(const rssm_kv_config* cfg, const rssm_kv_buffers* buf,
                          rssm_kv_handle** out) {
  const rssm_status st = check_config(cfg);
  if (st != RSSM_OK) return st;
  if (buf == nullptr || out == nullptr) return RSSM_ERR_INVALID_ARG;
  if (!buf->k_pages || !buf->v_pages || !buf->table || !buf->held || !buf->length || !buf->refs ||
      !buf->work || !buf->err_word)
    return RSSM_ERR_INVALID_ARG;
  if (!aligned16(buf->k_pages) || !aligned16(buf->v_pages) || !aligned16(buf->work) ||
      !aligned4(buf->table) || !aligned4(buf->held) || !aligned4(buf->length) ||
      !aligned4(buf->refs) || !aligned4(buf->err_word))
    return RSSM_ERR_INVALID_ARG;
  rssm_kv_handle* h = new (std::nothrow) rssm_kv_handle;
  if (h == nullptr) return RSSM_ERR_CUDA;
  h->cfg = *cfg;
  h->buf = *buf;
  h->shift = 0;
  while ((1 << h->shift) < cfg->page_size) ++h->shift;
  h->page_bytes = page_bytes(*cfg);
  h->layer_bytes = (size_t)cfg->n_pages * h->page_bytes;
  h->hook_cta = h->hook_unit = -1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess)
    e = cudaDeviceGetAttribute(&h->num_sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = attn_decode_prepare(cfg->D, cfg->dtype);
  if (e == cudaSuccess) e = attn_prompt_prepare(cfg->D, cfg->dtype);
  if (e == cudaSuccess)
    e = attn_decode_maps(h->maps, buf->k_pages, buf->v_pages,
                         (long long)cfg->n_layers * cfg->n_pages * cfg->HKV * cfg->page_size,
                         cfg->D, cfg->dtype);
  if (e != cudaSuccess) {
    delete h;
    return RSSM_ERR_CUDA;
  }
  *out = h;
  return RSSM_OK;
}

void rssm_kv_free(rssm_kv_handle* h) { delete h; }

rssm_status rssm_kv_reserve(rssm_kv_handle* h, const int32_t* slot, const int32_t* cu_seqlens,
                            int32_t B, int32_t T, void* stream) {
  const rssm_status st = check_rows(h, slot, B);
  if (st != RSSM_OK) return st;
  if (!aligned4(cu_seqlens)) return RSSM_ERR_INVALID_ARG;
  if (cu_seqlens == nullptr && (T < 1 || T > kMaxWindow)) return RSSM_ERR_INVALID_ARG;
  if (B == 0) return RSSM_OK;
  PageParams p = page_params(h);
  p.slot = slot;
  p.cu = cu_seqlens;
  p.B = B;
  p.T = T;
  return from_cuda(kv_plan_launch(PLAN_RESERVE, p, static_cast<cudaStream_t>(stream)));
}

rssm_status rssm_kv_commit(rssm_kv_handle* h, const int32_t* slot, const int32_t* accept_len,
                           const int32_t* cu_seqlens, int32_t B, int32_t T, void* stream) {
  const rssm_status st = check_rows(h, slot, B);
  if (st != RSSM_OK) return st;
  if (!aligned4(cu_seqlens) || !aligned4(accept_len)) return RSSM_ERR_INVALID_ARG;
  if (cu_seqlens == nullptr && (T < 1 || T > kMaxWindow)) return RSSM_ERR_INVALID_ARG;
  if (B == 0) return RSSM_OK;
  LengthParams p{};
  p.slot = slot;
  p.accept = accept_len;
  p.cu = cu_seqlens;
  p.held = h->buf.held;
  p.length = h->buf.length;
  p.err = h->buf.err_word;
  p.B = B;
  p.T = T;
  p.n_slots = h->cfg.n_slots;
  p.shift = h->shift;
  return from_cuda(kv_length_launch(p, static_cast<cudaStream_t>(stream)));
}

rssm_status rssm_kv_fork(rssm_kv_handle* h, const int32_t* src, const int32_t* dst, int32_t B,
                         int32_t deep, void* stream) {
  rssm_status st = check_rows(h, src, B);
  if (st == RSSM_OK) st = check_rows(h, dst, B);
  if (st != RSSM_OK || B == 0) return st;
  PageParams p = page_params(h);
  p.slot = dst;
  p.parent = src;
  p.B = B;
  p.deep = deep != 0;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = kv_plan_launch(PLAN_FORK, p, s);
  if (e != cudaSuccess) return from_cuda(e);
  return copy_pages(h, p, false, s);
}

rssm_status rssm_kv_release(rssm_kv_handle* h, const int32_t* slot, int32_t B, void* stream) {
  const rssm_status st = check_rows(h, slot, B);
  if (st != RSSM_OK || B == 0) return st;
  PageParams p = page_params(h);
  p.slot = slot;
  p.B = B;
  return from_cuda(kv_plan_launch(PLAN_RELEASE, p, static_cast<cudaStream_t>(stream)));
}

rssm_status rssm_kv_compact(rssm_kv_handle* h, void* stream) {
  if (h == nullptr) return RSSM_ERR_INVALID_ARG;
  const PageParams p = page_params(h);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = kv_plan_launch(PLAN_COMPACT, p, s);
  if (e != cudaSuccess) return from_cuda(e);
  return copy_pages(h, p, true, s);
}

rssm_status rssm_kv_append(rssm_kv_handle* h, int32_t layer, const void* q, const void* k,
                           const void* v, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                           const rssm_rope* rope, const int32_t* positions,
                           const int32_t* cu_seqlens, const int32_t* slot, int32_t B, int32_t T,
                           int32_t N, void* q_out, void* k_out, void* stream) {
  const rssm_status st = check_rows(h, slot, B);
  if (st != RSSM_OK) return st;
  const rssm_kv_config& c = h->cfg;
  if (layer < 0 || layer >= c.n_layers) return RSSM_ERR_INVALID_ARG;
  if (N < 0 || !aligned4(cu_seqlens) || !aligned4(positions)) return RSSM_ERR_INVALID_ARG;
  if (cu_seqlens == nullptr && (T < 1 || T > kMaxWindow || (int64_t)B * T != N))
    return RSSM_ERR_INVALID_ARG;
  if ((q == nullptr) != (q_out == nullptr)) return RSSM_ERR_INVALID_ARG;
  AppendParams p{};
  if (rope != nullptr) {
    if (rope->table == nullptr || !aligned16(rope->table) || rope->max_pos < 1)
      return RSSM_ERR_INVALID_ARG;
    if (rope->axes < 1 || rope->axes > kMaxRopeAxes) return RSSM_ERR_UNSUPPORTED;
    if (rope->pairs < 1 || 2 * (int64_t)rope->pairs > c.D) return RSSM_ERR_INVALID_ARG;
    if (rope->pairs % 8 != 0) return RSSM_ERR_UNSUPPORTED;  // whole 16-byte vectors
    int64_t sum = 0;
    for (int a = 0; a < rope->axes; ++a) {
      if (rope->sections[a] < 0) return RSSM_ERR_INVALID_ARG;
      sum += rope->sections[a];
      p.sec[a] = rope->sections[a];
    }
    if (sum != rope->pairs) return RSSM_ERR_INVALID_ARG;
    p.rope = rope->table;
    p.positions = positions;
    p.P = rope->pairs;
    p.axes = rope->axes;
    p.max_pos = rope->max_pos;
    p.interleaved = rope->interleaved != 0;
  }
  if (B == 0 || N == 0) return RSSM_OK;
  if (!tokens_ok(c, k, k_stride, c.HKV) || !tokens_ok(c, v, v_stride, c.HKV))
    return RSSM_ERR_INVALID_ARG;
  if (q != nullptr && (!tokens_ok(c, q, q_stride, c.HQ) || !aligned16(q_out)))
    return RSSM_ERR_INVALID_ARG;
  if (!aligned16(k_out)) return RSSM_ERR_INVALID_ARG;
  p.q = q;
  p.k = k;
  p.v = v;
  p.q_out = q_out;
  p.k_out = k_out;
  p.kp = static_cast<unsigned char*>(h->buf.k_pages) + (size_t)layer * h->layer_bytes;
  p.vp = static_cast<unsigned char*>(h->buf.v_pages) + (size_t)layer * h->layer_bytes;
  p.cu = cu_seqlens;
  p.slot = slot;
  p.table = h->buf.table;
  p.held = h->buf.held;
  p.length = h->buf.length;
  p.err = h->buf.err_word;
  p.qs = q_stride;
  p.ks = k_stride;
  p.vs = v_stride;
  p.B = B;
  p.T = T;
  p.N = N;
  p.HQ = c.HQ;
  p.HKV = c.HKV;
  p.D = c.D;
  p.n_slots = c.n_slots;
  p.n_pages = c.n_pages;
  p.max_pages = c.max_pages;
  p.shift = h->shift;
  p.dt = c.dtype;
  return from_cuda(kv_append_launch(p, static_cast<cudaStream_t>(stream)));
}

rssm_status rssm_attn_decode(rssm_kv_handle* h, int32_t layer, const void* q, int64_t q_stride,
                             const int32_t* slot, int32_t B, int32_t T, void* o, float* lse,
                             void* stream) {
  const rssm_status st = check_rows(h, slot, B);
  if (st != RSSM_OK) return st;
  const rssm_kv_config& c = h->cfg;
  if (layer < 0 || layer >= c.n_layers || T < 1) return RSSM_ERR_INVALID_ARG;
  if (T > 64) return RSSM_ERR_UNSUPPORTED;
  if (B == 0) return RSSM_OK;
  if (!tokens_ok(c, q, q_stride, c.HQ) || o == nullptr || !aligned16(o) || !aligned4(lse))
    return RSSM_ERR_INVALID_ARG;
  const KvWork w(c.n_pages);
  char* work = static_cast<char*>(h->buf.work);
  DecodeParams p{};
  p.q = q;
  p.slot = slot;
  p.table = h->buf.table;
  p.held = h->buf.held;
  p.length = h->buf.length;
  p.o = o;
  p.lse = lse;
  p.page0 = (long long)layer * c.n_pages;
  p.part = reinterpret_cast<float*>(work + w.part);
  p.count = reinterpret_cast<int32_t*>(work + w.count);
  p.err = h->buf.err_word;
  p.qs = q_stride;
  p.B = B;
  p.T = T;
  p.HQ = c.HQ;
  p.HKV = c.HKV;
  p.G = c.HQ / c.HKV;
  p.n_slots = c.n_slots;
  p.n_pages = c.n_pages;
  p.max_pages = c.max_pages;
  p.shift = h->shift;
  const int rows = attn_decode_block_rows(c.D, c.dtype, T * p.G);
  p.nmb = (T * p.G + rows - 1) / rows;
  p.hook_cta = h->hook_cta;
  p.hook_unit = h->hook_unit;
  p.c = (float)((double)c.scale * 1.4426950408889634);
  return from_cuda(
      attn_decode_launch(p, h->maps, c.D, c.dtype, h->num_sms,
                                     static_cast<cudaStream_t>(stream)));
}

rssm_status rssm_attn_prefill(rssm_kv_handle* h, const void* q, const void* k, const void* v,
                              int64_t q_stride, int64_t k_stride, int64_t v_stride,
                              const int32_t* cu_seqlens, const int32_t* cu_keys,
                              const int32_t* slot, int32_t B, int32_t N, int32_t M, void* o,
                              float* lse, void* stream) {
  if (h == nullptr || B < 0 || B > kMaxRows || N < 0 || M < 0) return RSSM_ERR_INVALID_ARG;
  if (B == 0 || N == 0) return RSSM_OK;
  const rssm_kv_config& c = h->cfg;
  if (cu_seqlens == nullptr || !aligned4(cu_seqlens) || !aligned4(cu_keys) || !aligned4(slot))
    return RSSM_ERR_INVALID_ARG;
  if (cu_keys == nullptr && M != N) return RSSM_ERR_INVALID_ARG;
  if (!tokens_ok(c, q, q_stride, c.HQ) || o == nullptr || !aligned16(o) || !aligned4(lse))
    return RSSM_ERR_INVALID_ARG;
  if (M > 0 && (!tokens_ok(c, k, k_stride, c.HKV) || !tokens_ok(c, v, v_stride, c.HKV)))
    return RSSM_ERR_INVALID_ARG;
  PromptParams p{};
  p.q = q;
  p.k = k;
  p.v = v;
  p.o = o;
  p.lse = lse;
  p.cu = cu_seqlens;
  p.cuk = cu_keys;
  p.slot = slot;
  p.err = h->buf.err_word;
  p.qs = q_stride;
  p.ks = k_stride;
  p.vs = v_stride;
  p.B = B;
  p.N = N;
  p.M = M;
  p.HQ = c.HQ;
  p.HKV = c.HKV;
  p.G = c.HQ / c.HKV;
  p.D = c.D;
  p.n_slots = c.n_slots;
  p.dt = c.dtype;
  p.hook_cta = h->hook_cta;
  p.hook_unit = h->hook_unit;
  p.c = (float)((double)c.scale * 1.4426950408889634);
  return from_cuda(attn_prompt_launch(p, static_cast<cudaStream_t>(stream)));
}

rssm_status rssm_kv_debug_withhold(rssm_kv_handle* h, int32_t cta, int32_t unit) {
  if (h == nullptr || cta < -1 || (cta >= 0 && unit < 0)) return RSSM_ERR_INVALID_ARG;
  h->hook_cta = cta;
  h->hook_unit = cta < 0 ? -1 : unit;
  return RSSM_OK;
}

rssm_status rssm_kv_get_device_error(rssm_kv_handle* h, uint32_t* out, int32_t clear,
                                     void* stream) {
  if (h == nullptr || out == nullptr) return RSSM_ERR_INVALID_ARG;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint32_t word = 0;
  if (cudaMemcpyAsync(&word, h->buf.err_word, sizeof(word), cudaMemcpyDeviceToHost, st) !=
      cudaSuccess)
    return RSSM_ERR_CUDA;
  if (cudaStreamSynchronize(st) != cudaSuccess) return RSSM_ERR_CUDA;
  if (clear) {
    if (cudaMemsetAsync(h->buf.err_word, 0, sizeof(uint32_t), st) != cudaSuccess)
      return RSSM_ERR_CUDA;
    if (cudaStreamSynchronize(st) != cudaSuccess) return RSSM_ERR_CUDA;
  }
  *out = word;
  return word == 0 ? RSSM_OK : RSSM_ERR_DEVICE;
}

}  // extern "C"
