// Parameters and launches of the full-attention layers' operators: the paged
// key-value cache (kv_pages.cu), the rotary append (kv_append.cu,
// kv_append_norm.cu), pages read back in a row (kv_gather.cu), attention of new
// tokens over the pages (attn_decode.cu), with prefixes that rows share
// (kv_share.cu, attn_shared_tc.cu), and of whole prompts (attn_prompt.cu,
// attn_prompt_tc.cu). Internal to librssm.
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
  unsigned char* scales;  // e4m3 pages (else null)
  const int32_t* moves;
  const int32_t* src;
  const int32_t* dst;
  const int32_t* map;     // compaction: renames the tables' pages (else null)
  int32_t* table;
  size_t page_bytes, layer_bytes, table_size;
  size_t scale_page_bytes, scale_layer_bytes;
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
  void* v_out;        // or null
  unsigned char* kp;  // this layer's pages
  unsigned char* vp;
  unsigned char* scales;  // this layer's, of e4m3 pages (else null)
  const float* q_weight;  // [D] norms of q and k, or null
  const float* k_weight;
  float eps;
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

struct GatherParams {
  const unsigned char* kp;  // this layer's pages
  const unsigned char* vp;
  const unsigned char* scales;  // this layer's, of e4m3 pages (else null)
  void* k_out;              // [N][HKV][D], or null
  void* v_out;
  const int32_t* cu;        // or null: T tokens a row
  const int32_t* first;     // [B] cache position of each row's first token; null: 0
  const int32_t* slot;
  const int32_t* table;
  const int32_t* held;
  uint32_t* err;
  int B, T, N, HKV, D;
  int n_slots, n_pages, max_pages, shift, dt;
};

constexpr int kShareSplit = kMaxSms;  // stretches that prefixes are cut into, about

// Stretches that a call can have: an even split over the SMs, and one more for
// every block of 128 rows of a group (of two members at least) and key head.
inline long long share_segments(int B, int T, int G, int HKV) {
  return kShareSplit + (long long)HKV * ((long long)B * T * G / 128 + B / 2 + 1);
}
struct ShareSeg {  // a stretch of a prefix, for 128 query rows of a key head
  int32_t begin;  // of its group's rows in order
  int32_t lead;   // the first of them
  int32_t group;
  int32_t keys;   // of the whole prefix
  int32_t rows;   // query rows of a key head of the group
  int32_t at;     // key head * blocks + block of 128 rows
  int32_t part;   // which stretch
  int32_t out;    // its place among the parts; -1: the only one
};
struct ShareRow {  // of a row with a prefix
  int32_t group;
  int32_t lead;    // the group's first row
  int32_t first;   // the row's first query row of a key head, among the group's
  int32_t parts;   // stretches of each of the group's blocks of 128 query rows
  int32_t part0;   // the first of them among the parts, where there are several
  int32_t blocks;  // of a key head
  int32_t pad[2];
};
// What rows of a batch share (kv_share.cu), in the caller's buffer: the groups,
// and what the first of the two launches leaves for the second.
struct ShareView {
  int32_t* of;          // [2] B and T of the plan
  int32_t* groups;      // [1] their number
  int32_t* lost;        // [1] a wait ran out: the prefixes' outputs are not all there
  int32_t* prefix;      // [B] keys of each row's shared prefix (0: none)
  int32_t* group;       // [B] each row's group (where it has a prefix)
  int32_t* order;       // [B] rows, group by group
  int32_t* begin;       // [B + 1] first place of a group in order
  int32_t* group_keys;  // [B] keys of a group's prefix
  ShareRow* rows;       // [B]
  int32_t* made_for;    // [1] the stamp of its cache
  int32_t* steps;       // [1] of 128 keys: a stretch of a prefix (attn_shared_tc.cuh)
  int32_t* segments;    // [1] stretches of all groups
  int32_t* direct;      // [1] each row's own keys, of one key head, are one CTA's
  int32_t* seg;         // [B + 1] first stretch of a group
  int32_t* parts;       // [B] stretches of a group's block of 128 rows and a key head
  int32_t* part0;       // [B] its first place among the parts, where there are several
  ShareSeg* segs;       // the stretches
  int32_t* scratch;     // [2 B] of the plan
  float2* ml;           // [B T][HQ] running maxima and sums of the prefixes
  float* o;             // [B T][HQ][D] and outputs
  float* part;          // [2 kShareSplit] of the stretches of prefixes that are cut:
                        // outputs [part_rows][D], maxima and sums [part_rows][2]
  int part_rows;        // query rows of a key head in a stretch, at most 128
  int32_t stamp;        // of the cache of this call
  __host__ __device__ static size_t up(size_t x) { return (x + 255) & ~(size_t)255; }
  // the view of a buffer (null: only its size)
  static size_t lay(void* base, int B, int T, int HQ, int HKV, int D, int shift, ShareView* v) {
    char* at = static_cast<char*>(base);
    size_t n = 0;
    auto take = [&](size_t bytes) {
      const size_t from = n;
      n += up(bytes);
      return at + from;
    };
    const size_t b = (size_t)B * 4, rows = (size_t)B * T * HQ;
    ShareView s{};
    char* head = take(32);
    char* prefix = take(b);
    char* group = take(b);
    char* order = take(b);
    char* begin = take(b + 4);
    char* keys = take(b);
    char* rec = take((size_t)B * sizeof(ShareRow));
    char* seg = take(b + 4);
    char* parts = take(b);
    char* part0 = take(b);
    char* scratch = take(2 * b);
    char* segs = take((size_t)share_segments(B, T, HQ / HKV, HKV) * sizeof(ShareSeg));
    char* ml = take(rows * 8);
    char* o = take(rows * (size_t)D * 4);
    // whole fours: parts begin on 16 bytes
    const size_t part_rows = rows / HKV < 125 ? (rows / HKV + 3) / 4 * 4 : 128;
    char* part = take(2 * kShareSplit * part_rows * (size_t)(D + 2) * 4);
    if (v != nullptr) {
      s.of = reinterpret_cast<int32_t*>(head);
      s.groups = s.of + 2;
      s.lost = s.of + 3;
      s.steps = s.of + 4;
      s.segments = s.of + 5;
      s.direct = s.of + 6;
      s.made_for = s.of + 7;
      s.segs = reinterpret_cast<ShareSeg*>(segs);
      s.rows = reinterpret_cast<ShareRow*>(rec);
      s.seg = reinterpret_cast<int32_t*>(seg);
      s.parts = reinterpret_cast<int32_t*>(parts);
      s.part0 = reinterpret_cast<int32_t*>(part0);
      s.prefix = reinterpret_cast<int32_t*>(prefix);
      s.group = reinterpret_cast<int32_t*>(group);
      s.order = reinterpret_cast<int32_t*>(order);
      s.begin = reinterpret_cast<int32_t*>(begin);
      s.group_keys = reinterpret_cast<int32_t*>(keys);
      s.scratch = reinterpret_cast<int32_t*>(scratch);
      s.ml = reinterpret_cast<float2*>(ml);
      s.o = reinterpret_cast<float*>(o);
      s.part = reinterpret_cast<float*>(part);
      s.part_rows = (int)part_rows;
      // what places and records depend on: HQ <= 4096, HQ / HKV <= 64, D in 64s, page size
      s.stamp = HQ | HQ / HKV << 13 | D / 64 << 20 | shift << 23 | 1 << 30;
      *v = s;
    }
    return n;
  }
};
// Whether the plan is one of B rows of T tokens, of a cache like this call's.
__device__ __forceinline__ bool share_is_of(const ShareView& s, int B, int T) {
  return s.of[0] == B && s.of[1] == T && *s.made_for == s.stamp;
}

struct DecodeParams {
  const void* q;
  const unsigned char* scales;  // all layers', of e4m3 pages (else null)
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
  int line_ctas;  // DEC_OWN: CTAs that the line is split over
  int cut;        // DEC_OWN: prefixes may be in parts (attn_shared_tc.cuh)
  int nmb;      // row blocks of a (row, key head): ceil(T G / rows of a block)
  int hook_cta, hook_unit;  // test hook of the bounded waits; -1: off
  float c;      // scale * log2(e)
  ShareView share;
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
cudaError_t kv_share_launch(const ShareView& v, const PageParams& p, int HKV, int G, bool quant,
                            cudaStream_t st);
cudaError_t kv_copy_launch(const CopyParams& p, int num_sms, cudaStream_t st);
cudaError_t kv_length_launch(const LengthParams& p, cudaStream_t st);
cudaError_t kv_append_launch(const AppendParams& p, cudaStream_t st);
cudaError_t kv_append_norm_launch(const AppendParams& p, cudaStream_t st);
cudaError_t kv_gather_launch(const GatherParams& p, int num_sms, cudaStream_t st);
cudaError_t attn_decode_prepare(int D, int dt, bool quant);
// tensor maps of the pool (kKvMapBytes, 64-byte aligned) and the launch with them
constexpr int kKvMapBytes = 256;
cudaError_t attn_decode_maps(void* maps, const void* k, const void* v, long long rows, int D,
                             int dt, bool quant, int page_size);
// kernels of quantised pages, blocks of `rows`; p null: prepares them all
cudaError_t attn_decode_quant(const DecodeParams* p, const void* maps, int D, int dt, int rows,
                              int sms, cudaStream_t st);
cudaError_t attn_decode_launch(const DecodeParams& p, const void* maps, int D, int dt, int num_sms,
                               cudaStream_t st);
int attn_decode_block_rows(int D, int dt, bool quant, int rows);  // rows of a block for T G rows
// the two launches of attention over shared prefixes, and their preparation
cudaError_t attn_shared_prepare(int D, int dt, bool quant);
cudaError_t attn_shared_launch(DecodeParams p, const void* maps, const void* tc_maps, int D,
                               int dt, int num_sms, cudaStream_t st);
cudaError_t attn_shared_tc_maps(void* maps, const void* k, const void* v, long long rows, int D,
                                int dt, bool quant, int page_size);
cudaError_t attn_shared_tc_prefix(const DecodeParams* p, const void* maps, int D, int dt,
                                  bool quant, cudaStream_t st);
cudaError_t attn_shared_prefix(const DecodeParams* p, const void* maps, int D, int dt, int rows,
                               int sms, cudaStream_t st);
cudaError_t attn_shared_own(const DecodeParams* p, const void* maps, int D, int dt, int rows,
                            int sms, cudaStream_t st);
cudaError_t attn_shared_own_quant(const DecodeParams* p, const void* maps, int D, int dt, int rows,
                                  int sms, cudaStream_t st);
cudaError_t attn_prompt_prepare(int D, int dt);
cudaError_t attn_prompt_launch(const PromptParams& p, cudaStream_t st);
cudaError_t attn_prompt_tc_prepare(int D, int dt);  // 16-bit types
cudaError_t attn_prompt_tc_launch(const PromptParams& p, cudaStream_t st);
cudaError_t attn_prompt_tc_wide_prepare(int dt);    // and D = 256
cudaError_t attn_prompt_tc_wide_launch(const PromptParams& p, cudaStream_t st);

}  // namespace rssm
