// Parameters and launches of the full-attention layers' operators: the paged
// key-value cache (kv_pages.cu), the rotary append (kv_append.cu), attention of
// new tokens over the pages (attn_decode.cu) and of whole prompts
// (attn_prompt.cu, attn_prompt_tc.cu). Internal to librssm.
#pragma once

#include "rssm_common.cuh"

namespace rssm {

enum : uint32_t {
  DEVERR_PAGES = 32u,     // pool empty, table row full, window past its pages, bad page id
  DEVERR_POSITION = 64u,  // rotary position outside the table
};

constexpr int kMaxSms = 152;        // SMs that a decode launch uses at most
constexpr int kMaxParts = 3 * kMaxSms;  // its CTAs: parts a row can be cut into
// fp32 values of two parts per CTA: outputs, running maxima and sums. Heads of
// 128 have the most: two CTAs per SM and 64 rows (D = 256: one CTA and 48 rows;
// D = 64: three CTAs). 20 MB, whatever the cache's D.
constexpr size_t kPartFloats = (size_t)2 * 2 * kMaxSms * 64 * (128 + 2);
constexpr int kMaxRopeAxes = 3;

// Regions of the caller's work buffer (bytes); `count` is zero between calls.
struct KvWork {
  size_t count;   // [kMaxParts] arrivals of the parts of a split row
  size_t part;    // [kPartFloats]
  size_t moves;   // [1] number of page copies of the last plan
  size_t src;     // [n_pages] pages to copy from
  size_t dst;     // [n_pages] pages to copy to; free pages of a reservation
  size_t map;     // [n_pages] new place of each moved page
  size_t rows;    // [65535 + 1] first free page of each row of a plan
  size_t total;
  __host__ __device__ static size_t up(size_t x) { return (x + 255) & ~(size_t)255; }
  __host__ __device__ explicit KvWork(int n_pages) {
    const size_t n = up((size_t)n_pages * 4);
    count = 0;
    part = up(kMaxParts * 4);
    moves = part + up(kPartFloats * 4);
    src = moves + 256;
    dst = src + n;
    map = dst + n;
    rows = map + n;
    total = rows + up(65536 * 4);
  }
};

enum : int { PLAN_RESERVE = 0, PLAN_FORK = 1, PLAN_RELEASE = 2, PLAN_COMPACT = 3 };

struct PageParams {
  int32_t* table;   // [n_slots][max_pages], -1 where no page is held
  int32_t* held;    // [n_slots]
  int32_t* length;  // [n_slots]
  int32_t* refs;    // [n_pages]
  uint32_t* err;
  int32_t* moves;
  int32_t* src;
  int32_t* dst;
  int32_t* map;
  int32_t* rows;
  const int32_t* slot;    // reserve, release: rows; fork: destination slots
  const int32_t* parent;  // fork: source slots
  const int32_t* cu;      // reserve: ragged lengths, or null
  int B, T, n_slots, n_pages, max_pages, shift, deep;
};

struct CopyParams {
  unsigned char* k;
  unsigned char* v;
  const int32_t* moves;
  const int32_t* src;
  const int32_t* dst;
  const int32_t* map;     // compaction: renames the tables' pages (else null)
  int32_t* table;
  size_t page_bytes, layer_bytes, table_size;
  int n_layers, n_pages;
};

struct LengthParams {
  const int32_t* slot;
  const int32_t* accept;  // or null: the whole window
  const int32_t* cu;      // or null: T tokens a row
  const int32_t* held;
  int32_t* length;
  uint32_t* err;
  int B, T, n_slots, shift;
};

struct AppendParams {
  const void* q;
  const void* k;
  const void* v;
  void* q_out;
  void* k_out;        // or null
  unsigned char* kp;  // this layer's pages
  unsigned char* vp;
  const float* rope;         // [max_pos][2][P] cosines, sines; null: no rotation
  const int32_t* positions;  // [axes][N]; null: the token's place in its cache
  const int32_t* cu;
  const int32_t* slot;
  const int32_t* table;
  const int32_t* held;
  const int32_t* length;
  uint32_t* err;
  long long qs, ks, vs;  // token strides, elements
  int B, T, N, HQ, HKV, D, P, axes, max_pos, interleaved;
  int sec[kMaxRopeAxes];
  int n_slots, n_pages, max_pages, shift, dt;
};

struct DecodeParams {
  const void* q;
  const int32_t* slot;
  const int32_t* table;
  const int32_t* held;
  const int32_t* length;
  void* o;
  float* lse;
  float* part;
  int32_t* count;
  uint32_t* err;
  long long qs;
  long long page0;  // the layer's first page among all layers'
  int B, T, HQ, HKV, G, n_slots, n_pages, max_pages, shift;
  int nmb;      // row blocks of a (row, key head): ceil(T G / rows of a block)
  int hook_cta, hook_unit;  // test hook of the bounded waits; -1: off
  float c;      // scale * log2(e)
};

struct PromptParams {
  const void* q;
  const void* k;
  const void* v;
  void* o;
  float* lse;
  const int32_t* cu;
  const int32_t* cuk;
  const int32_t* slot;  // or null
  uint32_t* err;
  long long qs, ks, vs;
  int B, N, M, HQ, HKV, G, D, n_slots, dt;
  int hook_cta, hook_unit;  // test hook of the bounded waits; -1: off
  float c;
};

cudaError_t kv_plan_launch(int mode, const PageParams& p, cudaStream_t st);
cudaError_t kv_copy_launch(const CopyParams& p, int num_sms, cudaStream_t st);
cudaError_t kv_length_launch(const LengthParams& p, cudaStream_t st);
cudaError_t kv_append_launch(const AppendParams& p, cudaStream_t st);
cudaError_t attn_decode_prepare(int D, int dt);
// tensor maps of the pool (kKvMapBytes, 64-byte aligned) and the launch with them
constexpr int kKvMapBytes = 256;
cudaError_t attn_decode_maps(void* maps, const void* k, const void* v, long long rows, int D,
                             int dt);
cudaError_t attn_decode_launch(const DecodeParams& p, const void* maps, int D, int dt, int num_sms,
                               cudaStream_t st);
int attn_decode_block_rows(int D, int dt, int rows);  // rows of a block for T G rows
cudaError_t attn_prompt_prepare(int D, int dt);
cudaError_t attn_prompt_launch(const PromptParams& p, cudaStream_t st);
cudaError_t attn_prompt_tc_prepare(int D, int dt);  // 16-bit types
cudaError_t attn_prompt_tc_launch(const PromptParams& p, cudaStream_t st);
cudaError_t attn_prompt_tc_wide_prepare(int dt);    // and D = 256
cudaError_t attn_prompt_tc_wide_launch(const PromptParams& p, cudaStream_t st);

}  // namespace rssm
