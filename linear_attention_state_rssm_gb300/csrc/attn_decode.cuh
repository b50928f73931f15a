// Attention of a window of T new tokens per request over its paged cache.
//
// For row r with slot s: query token t (its key and value already appended at
// cache position length[s] + t) sees the cache positions 0 .. length[s] + t.
// The T G query rows of one key head (G query heads share it) form blocks of
// 16, 32 or 64 rows (48 for D = 256); a block reads the keys and values of its head once.
//
// Bytes bound it: 2 D values per key and head, 2 T G D products with them. So
// the loads have to be wide, many, and never pause, and the work has to be even
// whatever the lengths. The chunks (16 or 32 keys) of every (row, key head,
// block) are laid on one line, each row's behind a gap that stands for what it
// costs to begin and end one, and each CTA of one wave takes an equal
// stretch of the line. A stretch that begins or ends inside a row leaves a part
// (running maximum, sum and unnormalised output) in the work buffer; the last
// CTA to leave one for a row joins them, in the order of the keys whoever it
// is, so results do not depend on the order of arrival.
//
// In a CTA one producer warp walks the stretch ahead of the others, over the
// ends of rows too: it looks the pages up and has one thread issue one TMA box
// per 16 keys and one per 16 values into a ring. Each stream (one
// warp per 16 rows of the block) takes every NG-th chunk of the CTA; streams meet
// only where a row ends, while the ring fills with the next row's chunks.
//
// Measured (GB300, back to back): 56 rows of 1 to 8 k tokens, 16/4 heads of 256:
// 133 us, 6.2 TB/s (92% of the copy rate); two rows of 109 to 131 k tokens, 32/8
// heads of 128, fp16: 157 us, 6.3 TB/s; 125 windows of 8 tokens over 0.3 to 3 k
// tokens, 16/4 heads of 128: 67 us, 4.4 TB/s, held back by the ends of its 2.5
// stretches a CTA (11 k cycles each, of 128 k) and by steps of two warps to a
// stream. Steps: private rings of cp.async per warp and whole CTAs to a row 142,
// 160, 113 us; the gap on the line 93 for the windows; this ring 86; rows of a
// join loaded side by side and 32 keys a step 68.
//
// Quantised pages (Q): the same with e4m3 boxes and, beside each, two bytes a key
// with its powers of two (attn_quant.cuh); blocks of 8 rows too. Measured: 56 rows
// of 1 to 8 k tokens, 16/4 heads of 256: 79 us, 5.6 TB/s (83% of the copy rate);
// two rows of 109 to 131 k tokens, 32/8 heads of 128: 88 us, 5.9 TB/s (87%). What a
// step costs besides its bytes holds them back: half the bytes, as many keys.
// Windows of 8 tokens (32 rows to a head): 77 us, 2.0 TB/s, bound by two warps'
// steps per stream, one instruction after the other (16-bit pages: 69 us).
//
// Prefixes that rows share (kv_share.cu) come in two launches. PREFIX, here for
// fp32 alone (else attn_shared_tc.cuh): a line of groups instead of rows; the query
// rows of all of a group's members are the rows of its blocks, all of the prefix is
// seen by all, and what is left is the running maximum, sum and output of every
// query row, in fp32. OWN: each row from the end of its prefix on, its first stream
// beginning with what the prefix left. Rows without a group begin at their
// first key. Behind the tensor cores' launch OWN's CTAs start as its own leave: lengths,
// tables, queries and a ring of keys are looked up and on their way when it ends, which
// they wait for (20 groups of 4 rows, four layers: 191 us, so 179).
#pragma once

#include "attn_core.cuh"
#include "attn_quant.cuh"
#include "attn_tma.h"
#include "kv_common.cuh"

namespace rssm {

namespace {

enum : int { DEC_PLAIN = 0, DEC_PREFIX = 1, DEC_OWN = 2 };

constexpr int kBox = 16;        // keys of a TMA box: within one page (pages of 16 k keys)
constexpr int kQuantBox = 32;   // rows of a column of quantised keys: a box's, or two of kBox's
constexpr int kGapKeys = 256;   // what beginning and ending a row costs, as keys
constexpr int kLeastKeys = 512; // keys that a CTA takes at least (of longer rows)
constexpr int kRowParts = 96;   // parts of the longest row, about: one CTA joins them
constexpr int kLostPart = 1 << 16;  // in a row's arrivals, beside their number: a part that is not there

// Streams of MW warps; quantised pages: of 8 NQ rows a warp, else of 16 (NQ 0).
template <typename T, int D, int MW, int NQ>
struct DecCfg {
  static constexpr bool Q = NQ > 0;
  using Warp = std::conditional_t<Q, WarpAttnQuant<D, NQ, 8 * NQ * MW, kQuantBox>,
                                  WarpAttn<T, D, 1, 16 * MW, kBox>>;
  static constexpr bool F32 = std::is_same<T, float>::value;
  // Outputs live in registers, D / 2 a lane: seven warps of 255 registers for
  // D = 256, ten of 168 for 128, fifteen of 128 for 64 (eight of 255 for fp32,
  // whose FMAs want more). A quarter of the registers belongs to each quarter
  // of the SM. Where they suffice a step takes 32 keys: what a step costs
  // whatever its size (waits, maxima over lanes) is most of it.
  // Quantised pages, eight rows a warp: half the outputs, and more warps. More
  // than five in a CTA leave too little of the ring on its way (128: seven 92 us
  // for two rows of 109 to 131 k tokens instead of 89; one CTA of nine 104).
  // Sixteen rows a warp of heads of 128: as many warps as 168 registers leave room
  // for, in two CTAs, or in one where a stream is several warps, whose steps then wait
  // less for one another (125 windows of 8 tokens over 3300 tokens, 16/4 heads: two
  // CTAs of four warps 166 us, one of ten 153, of twelve 202; of 16 tokens, four warps
  // to a stream: two of four 485, one of eight 315).
  static constexpr bool WIDE = NQ == 2 && D == 128 && MW > 1;
  static constexpr int CPS = NQ == 1              ? (D == 64 ? 3 : 2)
                             : D == 256 || WIDE   ? 1
                             : F32 || D == 128    ? 2
                                                  : 3;  // CTAs per SM
  static constexpr int NW = F32                    ? (D == 256 ? 4 : 3)
                            : NQ == 1              ? 5
                            : WIDE                 ? (MW == 2 ? 10 : 8)
                            : NQ == 2 && D == 128  ? 5
                            : D == 256             ? 6
                                                   : 4;  // warps of the streams
  static constexpr int CH = F32 || (D == 256 && !Q) ? 16 : 32;  // keys of a chunk
  static constexpr int GRP = D == 256 ? 2 : 4;         // chunks that are sent for together
  static constexpr int CT = NW * 32;                   // threads of the streams
  static constexpr int NT = CT + 32;                   // and the producer warp
  static constexpr int NG = NW / MW;                   // streams of a CTA
  static constexpr int WROWS = Warp::WROWS;            // rows of a warp
  static constexpr int ROWS = WROWS * MW;
  static constexpr int UNIT = CH * D * (Q ? 1 : (int)sizeof(T));
  static constexpr int SCALES = Q ? CH * 2 : 0;        // of a chunk
  static constexpr int QBYTES = ROWS * D * (int)sizeof(T);
  static constexpr int OP = 72;                        // row pitch of 64 columns of outputs
  static constexpr int OBYTES = NG > 1 ? NG * ROWS * OP * 4 : 0;
  // the joined parts of a prefix fit in the room of the streams' outputs
  static constexpr bool JOIN_HERE = OBYTES >= ROWS * D * 4;
  static constexpr int REST = 1024 + 2 * QBYTES + OBYTES + 2 * NG * ROWS * 4 + ROWS * 8 + 1024 +
                              (Q ? 2 * ROWS * 4 : 0);
  static constexpr int MOST = (228 / CPS - 1) * 1024;  // a CTA's share of the SM
  static_assert(NW % MW == 0, "whole streams");
  static constexpr int FIT = (MOST - REST) / (UNIT + SCALES);
  static constexpr int NU = FIT < 32 ? FIT : 32;       // units in the ring
  static constexpr int SMEM = NU * (UNIT + SCALES) + REST;
  static constexpr int PART = ROWS * (D + 2);          // floats of a part
  static_assert(NU >= 2 * NG && NU >= 2 * GRP, "a chunk for each stream, and a group of them");
  static_assert(CPS * kMaxSms * 2 * PART <= kPartFloats, "work buffer");
  static_assert(CPS * kMaxSms <= kMaxParts, "arrivals");
};

// Slot whose table stands for those of all of a group's members: the first that
// is still in use; -1 where none is.
__device__ __forceinline__ int lead_slot(const DecodeParams& p, int group) {
  for (int i = p.share.begin[group]; i < p.share.begin[group + 1]; ++i) {
    const int s = p.slot[p.share.order[i]];
    if (s >= 0 && s < p.n_slots) return s;
  }
  return -1;
}

// keys of row r (committed and new), 0 for a null or refused row; for PREFIX the
// shared keys of group r. start: the first key that the row reads here.
template <int MODE>
__device__ __forceinline__ int row_keys(const DecodeParams& p, int r, bool tell, int& s,
                                        int& start) {
  start = 0;
  if constexpr (MODE == DEC_PREFIX) {
    s = -1;
    if (!share_is_of(p.share, p.B, p.T) || r >= *p.share.groups) return 0;
    s = lead_slot(p, r);
    if (s < 0) return 0;
    const int keys = p.share.group_keys[r], most = p.max_pages << p.shift;
    return keys < most ? keys : most;
  } else {
    s = p.slot[r];
    if (s < 0) return 0;
    uint32_t bad = 0;
    int n = 0;
    if (s >= p.n_slots) {
      bad = DEVERR_SLOT;
    } else {
      const int len = p.length[s], held = p.held[s];
      if (len < 0) {
        bad = DEVERR_CURSOR;
      } else if (held < 0 || held > p.max_pages ||
                 (long long)len + p.T > ((long long)held << p.shift)) {
        bad = DEVERR_PAGES;
      } else {
        n = len + p.T;
        if constexpr (MODE == DEC_OWN) {
          start = p.share.prefix[r];
          // a plan of another call's windows, or of a slot that has got shorter
          if (!share_is_of(p.share, p.B, p.T) || start < 0 || start > len) {
            bad = DEVERR_PAGES;
            n = start = 0;
          }
        }
      }
    }
    if (bad && tell) atomicOr(p.err, bad);
    return n;
  }
}

// blocks of query rows of a row (or group)
template <int MODE, int ROWS>
__device__ __forceinline__ int row_blocks(const DecodeParams& p, int r) {
  if constexpr (MODE == DEC_PREFIX) {
    if (!share_is_of(p.share, p.B, p.T) || r >= *p.share.groups) return 1;
    const long long rows = (long long)(p.share.begin[r + 1] - p.share.begin[r]) * p.T * p.G;
    return (int)((rows + ROWS - 1) / ROWS);
  } else {
    return p.nmb;
  }
}

// places of a row's chunks of CH keys on the line, with the gap before them
template <int CH, int GAP>
__device__ __forceinline__ long long places(int keys) {
  return keys > 0 ? ((long long)keys + CH - 1) / CH + GAP : 0;
}

__device__ __forceinline__ long long warp_scan(long long x, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long y = __shfl_up_sync(kFull, x, d);
    if (lane >= d) x += y;
  }
  return x;
}

// A stretch of one (row, key head, block): chunks [c0, c1).
struct Seg {
  int row, slot, keys, h, mb, c0, c1, chunks;
  long long item0;  // place of its first chunk on the line
  int more, start;  // more 0: the stretch is done; start: the row's first key
};

// The CTA's stretch of the line, one Seg after the other.
template <int CH, int MODE, int ROWS>
struct Line {
  static constexpr int kGap = kGapKeys / CH;
  long long pos, end, row0;
  int row;
  __device__ __forceinline__ bool next(const DecodeParams& p, Seg& g) {
    while (pos < end) {
      g.keys = row_keys<MODE>(p, row, false, g.slot, g.start);
      const int nmb = row_blocks<MODE, ROWS>(p, row), items = p.HKV * nmb;
      const int cost = (int)places<CH, kGap>(g.keys - g.start);
      if (pos >= row0 + (long long)cost * items) {
        row0 += (long long)cost * items;
        ++row;
        continue;
      }
      const int item = (int)((pos - row0) / cost);
      const int off = (int)((pos - row0) % cost);
      const int len = (long long)cost - off <= end - pos ? cost - off : (int)(end - pos);
      g.row = row;
      g.h = item / nmb;
      g.mb = item % nmb;
      g.chunks = cost - kGap;
      g.c0 = max(0, off - kGap);
      g.c1 = max(0, off + len - kGap);
      g.item0 = row0 + (long long)item * cost + kGap;
      pos += len;
      if (g.c1 > g.c0) return true;
    }
    return false;
  }
};

// Counts a CTA's part of a split row in (one thread). Every part is counted,
// there or not, so the last one clears the count for the next call whatever
// happened, and joins the row (true) only if none is missing.
__device__ __forceinline__ bool count_part(int32_t* count, long long item0, int chunks,
                                           long long share, bool lost) {
  const int cta0 = (int)(item0 / share);
  const int parts = (int)((item0 + chunks - 1) / share) - cta0 + 1;
  const int add = lost ? kLostPart + 1 : 1;
  const int n = atomicAdd(count + cta0, add) + add;
  if ((n & (kLostPart - 1)) != parts) return false;
  count[cta0] = 0;
  return n < kLostPart;
}

// Counts in what a CTA that gave up in its ns-th segment leaves undone.
template <int CH, int MODE, int ROWS>
__device__ __noinline__ void give_up(const DecodeParams& p, Line<CH, MODE, ROWS> line, int ns,
                                     long long share) {
  Seg g;
  for (int i = 0; line.next(p, g); ++i) {
    if (i >= ns && (g.c0 > 0 || g.c1 < g.chunks))
      count_part(p.count, g.item0, g.chunks, share, true);
  }
}

struct KvMaps {
  CUtensorMap k, v;
};

// query rows of a row (or group) for one key head
template <int MODE>
__device__ __forceinline__ int query_rows(const DecodeParams& p, int r) {
  if constexpr (MODE == DEC_PREFIX) {
    return (p.share.begin[r + 1] - p.share.begin[r]) * p.T * p.G;
  } else {
    return p.T * p.G;
  }
}

// token of query row tr of a row (or group)
template <int MODE>
__device__ __forceinline__ long long query_token(const DecodeParams& p, int r, int tr) {
  if constexpr (MODE == DEC_PREFIX) {
    const int member = tr / (p.T * p.G), rest = tr % (p.T * p.G);
    return (long long)p.share.order[p.share.begin[r] + member] * p.T + rest / p.G;
  } else {
    return (long long)r * p.T + tr / p.G;
  }
}

// Whether the row's pages up to its prefix's end are those that the group's keys
// are read from (the plan may be older than the tables).
template <int THREADS>
__device__ __forceinline__ bool prefix_holds(const DecodeParams& p, const Seg& sg,
                                             const ShareRow& rec, int tid) {
  int lead = p.slot[rec.lead];
  if (lead < 0 || lead >= p.n_slots) lead = lead_slot(p, rec.group);
  bool same = lead >= 0;
  if (!same || sg.slot == lead) return same;
  const int32_t* a = p.table + (size_t)sg.slot * p.max_pages;
  const int32_t* b = p.table + (size_t)lead * p.max_pages;
  const int n = sg.start >> p.shift;
  for (int i = tid; i < n; i += THREADS) same = same && a[i] == b[i];
  return same;
}

// The end of the launch before this one, whose memory is then there to be read
// (at once where the launch does not overlap it).
__device__ __forceinline__ void launch_before_ended() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Whether any of the `count` threads of a named barrier says so (a barrier too).
__device__ __forceinline__ bool named_any(int id, int count, bool x) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %3, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"(id), "r"(count), "r"((uint32_t)x)
      : "memory");
  return any != 0;
}

// l 2^d for d <= 0. Over quantised pages l is up to 2^78 times the number of keys, and 2^d
// alone may be below fp32's range where the product counts (attn_quant.cuh).
template <bool Q>
__device__ __forceinline__ float brought(float l, float d) {
  if constexpr (!Q) return l * exp2_fast(d);
  const float half = exp2_fast(0.5f * d);
  return l * half * half;
}

// The parts of a prefix that was cut, joined for a block's rows: outputs [R][D]
// to where `to` says, maxima and sums into row_m and row_l. All threads of the
// streams; a barrier has to follow. A thread has four dimensions of a row, so
// that all its loads are one trip to memory.
template <typename C, int D, typename F>
__device__ __forceinline__ void join_parts(const DecodeParams& p, const Seg& sg,
                                           const ShareRow& rec, int base, int R, F to,
                                           float* row_m, float* row_l, int tid) {
  const ShareView& s = p.share;
  const size_t part = (size_t)s.part_rows * (D + 2);
  for (int i = tid; i < R * (D / 4); i += C::CT) {
    const int rr = i / (D / 4), d = i % (D / 4) * 4;
    const int row = rec.first + base + rr, block = row / 128, r = row % 128;
    const float* from =
        s.part + (rec.part0 + ((size_t)sg.h * rec.blocks + block) * rec.parts) * part;
    const float* at_o = from + (size_t)r * D + d;
    const float* at_ml = from + (size_t)s.part_rows * D + 2 * r;
    float m = kNegInf, l = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int k = 0; k < rec.parts; ++k) {
      const float4 y = __ldcg(reinterpret_cast<const float4*>(at_o + k * part));
      const float2 ml = __ldcg(reinterpret_cast<const float2*>(at_ml + k * part));
      const float top = fmaxf(m, ml.x), mu = top == kNegInf ? 0.f : top;
      const float fa = exp2_fast(m - mu), fb = exp2_fast(ml.x - mu);
      l = brought<C::Q>(l, m - mu) + brought<C::Q>(ml.y, ml.x - mu);
      a.x = a.x * fa + y.x * fb;
      a.y = a.y * fa + y.y * fb;
      a.z = a.z * fa + y.z * fb;
      a.w = a.w * fa + y.w * fb;
      m = top;
    }
    *reinterpret_cast<float4*>(to(rr) + d) = a;
    if (d == 0) row_m[rr] = m, row_l[rr] = l;
  }
}

template <typename T, int D, int MW, int NQ, int MODE>
__global__ void __launch_bounds__(DecCfg<T, D, MW, NQ>::NT, DecCfg<T, D, MW, NQ>::CPS)
    attn_decode_kernel(const __grid_constant__ DecodeParams p,
                       const __grid_constant__ KvMaps maps) {
  using C = DecCfg<T, D, MW, NQ>;
  using W = typename C::Warp;
  constexpr bool Q = NQ > 0;
  using Stretch = Line<C::CH, MODE, C::ROWS>;
  constexpr int NG = C::NG, NW = C::NW;
  static_assert(MODE != DEC_PREFIX || (C::F32 && NG > 1), "else on the tensor cores");
  extern __shared__ unsigned char sm_raw[];
  unsigned char* ring = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(sm_raw) + 1023) & ~(uintptr_t)1023);
  unsigned char* qs = ring + C::NU * C::UNIT;                  // [2][QBYTES]
  float* os = reinterpret_cast<float*>(qs + 2 * C::QBYTES);    // [NG][ROWS][OP]
  float* sm_m = os + C::OBYTES / 4;                            // [NG][ROWS]
  float* sm_l = sm_m + NG * C::ROWS;
  float* row_m = sm_l + NG * C::ROWS;                          // [ROWS]
  float* row_l = row_m + C::ROWS;
  uint64_t* full = reinterpret_cast<uint64_t*>(row_l + C::ROWS);  // [NU] a unit has landed
  uint64_t* empty = full + C::NU;                              // [NU] its stream has read it
  uint64_t* qfull = empty + C::NU;                             // [2] a segment is described
  uint64_t* qempty = qfull + 2;                                // [2] and done
  long long* scan = reinterpret_cast<long long*>(qempty + 2);  // [3 (NW + 1) + 2]
  Seg* segs = reinterpret_cast<Seg*>(scan + 3 * (NW + 1) + 3); // [2]
  volatile int* issued = reinterpret_cast<volatile int*>(segs + 2);  // units on their way
  int* flag = const_cast<int*>(issued) + 1;  // [4] no output; joins; a wait ran out (by turns)
  // the unit that was not sent for because a wait ran out (in a register it would
  // cost the producer's loop 1.5% of 56 rows of 1 to 8 k tokens)
  volatile int* stop = issued + 5;
  // quantised pages: a chunk's powers of two beside each place of the ring, and
  // c 2^a of the rows of both halves
  unsigned char* ring_scales =
      Q ? reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(stop + 1) + 15) &
                                           ~(uintptr_t)15)
        : nullptr;
  float* row_f = reinterpret_cast<float*>(ring_scales + C::NU * C::SCALES);  // [2][ROWS]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int u = 0; u < C::NU; ++u) mbar_init(&full[u], 1), mbar_init(&empty[u], MW);
    for (int i = 0; i < 2; ++i) mbar_init(&qfull[i], 33), mbar_init(&qempty[i], NW);
    *issued = 0;
    *stop = -1;
    for (int i = 0; i < 4; ++i) flag[i] = 0;
    if (p.hook_cta == (int)blockIdx.x) mbar_promise(&full[p.hook_unit % C::NU], 16);
    fence_mbar_init();
  }
  // A CTA of OWN does not leave before the prefixes' launch has ended, or the launch
  // after them could begin while it runs.
  auto nothing_to_do = [] {
    if constexpr (MODE == DEC_OWN) launch_before_ended();
  };
  Stretch line;
  long long share = 0;  // places of a CTA's stretch
  bool direct = false;
  if constexpr (MODE == DEC_OWN) {
    // Rows with few keys of their own: an item to a CTA, without a look at the
    // others' lengths and never two beginnings one behind the other.
    const int items = p.HKV * p.nmb;
    direct = (long long)p.B * items <= gridDim.x && *p.share.direct != 0;
    if (!direct && (int)blockIdx.x >= p.line_ctas) return nothing_to_do();
    if (direct) {
      line.row = blockIdx.x / items;
      if (line.row >= p.B) return nothing_to_do();
      int s, start;
      const int keys = row_keys<MODE>(p, line.row, blockIdx.x % items == 0 && tid == 0, s, start);
      const long long cost = places<C::CH, Stretch::kGap>(keys - start);
      if (cost == 0) return nothing_to_do();
      line.row0 = 0;
      line.pos = blockIdx.x % items * cost;
      line.end = line.pos + cost;
      share = cost;
      __syncthreads();  // barriers are set up
    }
  }
  if (!direct) {
    const int ctas = MODE == DEC_OWN ? p.line_ctas : (int)gridDim.x;
    // ---- the line's length and its longest row, and the row that holds this
    // CTA's first place: one look at the lengths for up to NT rows, else two
    long long mine = 0, most = 0, first_w = 0;
    for (int r = tid; r < p.B; r += C::NT) {
      int s, start;
      const int keys = row_keys<MODE>(p, r, blockIdx.x == 0, s, start);
      const long long cost = places<C::CH, Stretch::kGap>(keys - start);
      const long long w = cost * p.HKV * row_blocks<MODE, C::ROWS>(p, r);
      if (r < C::NT) first_w = w;
      mine += w;
      most = cost > most ? cost : most;
    }
    const long long first_incl = warp_scan(first_w, lane);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      mine += __shfl_xor_sync(kFull, mine, d);
      const long long y = __shfl_xor_sync(kFull, most, d);
      most = y > most ? y : most;
    }
    if (lane == 31) {
      scan[warp] = mine;
      scan[NW + 1 + warp] = most;
      scan[2 * (NW + 1) + warp] = first_incl;
    }
    __syncthreads();
    long long total = 0, longest = 0, at = 0, firsts = 0;
    for (int w = 0; w <= NW; ++w) {
      total += scan[w];
      longest = scan[NW + 1 + w] > longest ? scan[NW + 1 + w] : longest;
      if (w < warp) at += scan[2 * (NW + 1) + w];
      firsts += scan[2 * (NW + 1) + w];
    }
    share = (total + ctas - 1) / ctas;
    const long long few = longest / kRowParts + 1;
    share = share > few ? share : few;
    // not less than kLeastKeys, or a whole row where the longest has fewer
    const long long least =
        longest < Stretch::kGap + kLeastKeys / C::CH ? longest : Stretch::kGap + kLeastKeys / C::CH;
    share = share > least ? share : least;
    line.pos = share * blockIdx.x;
    line.end = line.pos + share < total ? line.pos + share : total;
    if (line.pos >= line.end) return nothing_to_do();
    at += first_incl - first_w;
    long long* found = scan + 3 * (NW + 1);  // row, its first place
    if (at <= line.pos && line.pos < at + first_w) {
      found[0] = tid;
      found[1] = at;
    }
    long long before = firsts;
    for (int r0 = C::NT; r0 < p.B && before <= line.pos; r0 += C::NT) {
      long long w = 0;
      if (r0 + tid < p.B) {
        int s, start;
        const int keys = row_keys<MODE>(p, r0 + tid, false, s, start);
        w = places<C::CH, Stretch::kGap>(keys - start) * p.HKV *
            row_blocks<MODE, C::ROWS>(p, r0 + tid);
      }
      const long long incl = warp_scan(w, lane);
      __syncthreads();  // the last sums have been read
      if (lane == 31) scan[warp] = incl;
      __syncthreads();
      long long first = before + incl - w;
      for (int i = 0; i <= NW; ++i) {
        if (i < warp) first += scan[i];
        before += scan[i];
      }
      if (first <= line.pos && line.pos < first + w) {
        found[0] = r0 + tid;
        found[1] = first;
      }
    }
    __syncthreads();
    line.row = (int)found[0];
    line.row0 = found[1];
  }

  const long long begin = line.pos;
  // for a CTA that gives up; the sums that stood there have been read
  Stretch* from_start = reinterpret_cast<Stretch*>(scan);
  static_assert(sizeof(Stretch) <= 3 * 8 * (NW + 1), "behind the barriers");
  if (tid == 0) *from_start = line;
  bool dead = false;  // a bounded wait ran out
  if (warp == NW) {
    // ---- producer
    Seg sg;
    int n = 0, ns = 0;  // chunks and segments issued
    while (!dead) {
      sg.more = line.next(p, sg);
      // the segment's description and its query rows (zeros after the last),
      // into the half that the segment before the last has left
      const int half = ns & 1;
      if (MODE == DEC_OWN && ns == 2) launch_before_ended();  // as where the ring is full
      if (ns >= 2) dead = !mbar_wait_bounded(&qempty[half], (uint32_t)((ns / 2 - 1) & 1));
      dead = __any_sync(kFull, dead);
      if (dead) break;
      // a lane without bulk copies on their way, which a release would wait for
      if (lane == (MODE != DEC_PLAIN || Q ? 31 : 1)) {
        segs[half] = sg;
        mbar_arrive(&qfull[half]);
      }
      if (sg.more) {
        constexpr int QU = D * (int)sizeof(T) / 16;  // units per row
        const int base = sg.mb * C::ROWS, R = min(C::ROWS, query_rows<MODE>(p, sg.row) - base);
        const uint32_t qd = smem_addr(qs + half * C::QBYTES);
#pragma unroll 4
        for (int i = lane; i < C::ROWS * QU; i += 32) {
          const int rr = i / QU, u = i % QU;
          const int tr = base + (rr < R ? rr : 0);
          const T* q = static_cast<const T*>(p.q) +
                       query_token<MODE>(p, sg.row, tr) * p.qs +
                       (long long)(sg.h * p.G + tr % p.G) * D;
          cp_async16_or_zero(qd + unit_off<C::ROWS>(rr, u), reinterpret_cast<const uint4*>(q) + u,
                             rr < R);
        }
      }
      __syncwarp();
      cp_async_arrive(&qfull[half]);
      ++ns;
      if (!sg.more) break;
      const int32_t* tab = p.table + (size_t)sg.slot * p.max_pages;
      // the boxes of the segment's chunks, 32 looked up at a time
      constexpr int BPC = C::CH / kBox;  // boxes of a chunk
      const int b_end = min(sg.c1 * BPC, (sg.keys - sg.start + kBox - 1) / kBox);
      for (int cb = sg.c0; cb < sg.c1 && !dead; cb += 32 / BPC) {
        const int box = cb * BPC + lane;
        int row = -1;  // of the pool: ((layer pages + page) HKV + head) page_size + token
        if (box < b_end) {
          const long long tok = sg.start + (long long)box * kBox;
          int page = tab[tok >> p.shift];
          if (page < 0 || page >= p.n_pages) {
            page = 0;  // the row's output is undefined; nothing outside the pool is read
            atomicOr(p.err, DEVERR_PAGES);
          }
          row = (int)((((p.page0 + page) * p.HKV + sg.h) << p.shift) +
                      (tok & ((1 << p.shift) - 1)));
        }
        const int cnt = min(32 / BPC, sg.c1 - cb);
        // Copies go out from lanes side by side, a group of chunks at a time: lane u
        // sees to it that the group's u-th place in the ring is free and says what
        // will land there, then each sends for one copy. From one lane, chunk by
        // chunk, the six copies of a quantised chunk in boxes of sixteen took 1300
        // cycles, twice what their bytes take; from several, with boxes of 32, 865;
        // in groups of four chunks 430 (two rows of 109 to 131 k tokens: 143, 107,
        // 89 us).
        constexpr int GRP = C::GRP;
        for (int i = 0; i < cnt && (MODE != DEC_PLAIN || Q); i += GRP) {
          const int units = 2 * min(GRP, cnt - i);
          const int u = 2 * n + lane, at_u = u % C::NU;
          // The streams, who empty the ring, begin when the prefixes' launch has ended: a
          // wait that could be for that would count it in its limit.
          if (MODE == DEC_OWN && 2 * n <= C::NU && 2 * n + units > C::NU) launch_before_ended();
          if (lane < units && u >= C::NU)
            dead = !mbar_wait_bounded(&empty[at_u], (uint32_t)((u / C::NU - 1) & 1));
          dead = __any_sync(kFull, dead);
          if (dead) {
            if (lane == 0) *stop = 2 * n;
            break;
          }
          if (lane < units)
            mbar_expect_tx(&full[at_u], C::UNIT + (lane % 2 == 0 ? C::SCALES : 0));
          __syncwarp();
          if (lane == 0) *issued = 2 * n + units;
          // boxes of the chunk of this lane's unit; one behind the last key is not
          // loaded: the one before it stands in its place, and no row sees it
          const int c = i + lane / 2;  // its chunk
          int at_row[BPC];
#pragma unroll
          for (int b = 0; b < BPC; ++b) at_row[b] = __shfl_sync(kFull, row, (c * BPC + b) & 31);
#pragma unroll
          for (int b = 1; b < BPC; ++b) at_row[b] = at_row[b] >= 0 ? at_row[b] : at_row[0];
          unsigned char* to = ring + at_u * C::UNIT;
          const CUtensorMap* map = lane % 2 == 0 ? &maps.k : &maps.v;
          if constexpr (Q) {
            static_assert(C::CH == kQuantBox, "one box of a page of 32 tokens or more");
            if (p.shift >= 5) {
              if (lane < units) tma_load3(smem_addr(to), map, 0, at_row[0], 0, &full[at_u]);
              if (lane < units && lane % 2 == 0)
                bulk_g2s(ring_scales + at_u * C::SCALES, p.scales + 2 * (size_t)at_row[0],
                         C::SCALES, &full[at_u]);
            } else if (lane < units) {
              constexpr int COLS = D == 256 ? 2 : 1;  // columns of 128 bytes (64: of 64)
#pragma unroll
              for (int b = 0; b < BPC; ++b) {
#pragma unroll
                for (int col = 0; col < COLS; ++col)
                  tma_load3(smem_addr(to + col * (kQuantBox * 128) + b * (C::UNIT / COLS / 2)), map,
                            0, at_row[b], col, &full[at_u]);
                if (lane % 2 == 0)
                  bulk_g2s(ring_scales + at_u * C::SCALES + b * (2 * kBox),
                           p.scales + 2 * (size_t)at_row[b], 2 * kBox, &full[at_u]);
              }
            }
          } else if (lane < units) {
#pragma unroll
            for (int b = 0; b < BPC; ++b)
              tma_load3(smem_addr(to + b * (C::UNIT / BPC)), map, 0, at_row[b], 0, &full[at_u]);
          }
          __syncwarp();
          n += units / 2;
        }
        for (int i = 0; i < cnt && MODE == DEC_PLAIN && !Q; ++i) {
          int at_row[BPC];
#pragma unroll
          for (int b = 0; b < BPC; ++b) at_row[b] = __shfl_sync(kFull, row, i * BPC + b);
          if (lane == 0) {
            // a box behind the last key is not loaded: the one before it stands
            // in its place, and no row sees it
            int boxes = 0;
#pragma unroll
            for (int b = 0; b < BPC; ++b) boxes += at_row[b] >= 0;
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
              const int u = 2 * n + kv, at_u = u % C::NU;
              if (!dead && u >= C::NU &&
                  !mbar_wait_bounded(&empty[at_u], (uint32_t)((u / C::NU - 1) & 1)))
                dead = true, *stop = u;
              if (!dead) {
                mbar_expect_tx(&full[at_u], C::UNIT);
#pragma unroll
                for (int b = 0; b < BPC; ++b)
                  tma_load3(smem_addr(ring + at_u * C::UNIT + b * (C::UNIT / BPC)),
                            kv == 0 ? &maps.k : &maps.v, 0, at_row[b < boxes ? b : 0], 0,
                            &full[at_u]);
              }
            }
            if (!dead) *issued = 2 * n + 2;
          }
          ++n;
        }
        dead = __any_sync(kFull, dead);
      }
    }
    // Every copy has landed before the CTA leaves. Once a wait ran out the copies
    // on their way get one more limit between them (a slot's earlier units were
    // read, or it would not have been filled again).
    if (lane == 0) {
      bool late = false;
      const int sent = *stop >= 0 ? *stop : 2 * n;
      for (int u = max(0, sent - C::NU); u < sent; ++u)
        late |= !mbar_wait_bounded(&full[u % C::NU], (uint32_t)((u / C::NU) & 1),
                                   late ? 0 : kWaitLimitNs);
      if (dead || late) atomicOr(p.err, DEVERR_TIMEOUT);
    }
    if (dead) cp_async_wait_all();  // the queries'
    return;
  }

  // ---- streams
  // where the CTA has one row, what its prefix left is got ready while the queries
  // and the first keys are on their way
  [[maybe_unused]] ShareRow rec{};
  [[maybe_unused]] bool early = false, early_bad = false;
  if constexpr (MODE == DEC_OWN) {
    Seg sg;
    Stretch ahead = line;
    if (direct && ahead.next(p, sg) && sg.start > 0) {
      early = true;
      rec = p.share.rows[sg.row];
      const int base = sg.mb * C::ROWS, R = min(C::ROWS, p.T * p.G - base);
      early_bad = !prefix_holds<C::CT>(p, sg, rec, tid);
      launch_before_ended();
      if (p.cut && rec.parts > 1) {
        auto joined = [&](int rr) {
          const int tr = base + rr;
          return C::JOIN_HERE ? os + rr * D
                              : p.share.o + ((size_t)query_token<MODE>(p, sg.row, tr) * p.HQ +
                                             sg.h * p.G + tr % p.G) * D;
        };
        join_parts<C, D>(p, sg, rec, base, R, joined, row_m, row_l, tid);
      }
    } else {
      launch_before_ended();
    }
    // the streams' waits begin here: none counts the prefixes' time in its limit
  }
  const int grp = warp / MW, wr = C::WROWS * (warp % MW);  // the warp's stream, its first row
  int n0 = 0;    // the segment's first chunk among the CTA's
  int seen = 0;  // units known to be on their way
  for (int ns = 0;; ++ns) {
    const int half = ns & 1;
    // The streams meet at barriers, so they stop together: a wait that ran out
    // is told here, by turns in two places (the next turn's word is written
    // only once every stream has read this one's).
    dead = dead || !mbar_wait_bounded(&qfull[half], (uint32_t)((ns >> 1) & 1));
    if (dead) flag[2 + half] = 1;
    named_sync(1, C::CT);
    const Seg sg = segs[half];
    if (flag[2 + half] != 0) {
      if (tid == 0) give_up(p, *from_start, ns, share);
      break;
    }
    if (!sg.more) break;
    const int base = sg.mb * C::ROWS;                  // first of the block's T G rows
    const int R = min(C::ROWS, query_rows<MODE>(p, sg.row) - base);  // rows in use
    // how many keys the lane's rows see
    const int first = sg.keys - p.T;  // committed keys
    int lim[W::RL];
#pragma unroll
    for (int e = 0; e < W::RL; ++e)
      lim[e] = MODE == DEC_PREFIX ? sg.keys
                                  : first + (base + min(wr + W::row(e, lane), R - 1)) / p.G + 1;
    const int fewest =
        MODE == DEC_PREFIX ? sg.keys : first + (base + min(wr, R - 1)) / p.G + 1;
    W w;
    w.clear();
    const unsigned char* qw = qs + half * C::QBYTES + wr * 128;
    [[maybe_unused]] float rf[W::RL];
    if constexpr (Q) {
      // the block's queries as fp16, each row by a power of two of its own
      constexpr int L = D / 16;
      for (int i = tid; i < C::ROWS * L; i += C::CT) {
        const float f = scale_query<T, D, C::ROWS>(qs + half * C::QBYTES, i / L, i % L);
        if (i % L == 0) row_f[half * C::ROWS + i / L] = f * p.c;
      }
      named_sync(1, C::CT);
#pragma unroll
      for (int e = 0; e < W::RL; ++e) rf[e] = row_f[half * C::ROWS + wr + W::row(e, lane)];
    }
    auto out_row = [&](int rr) {
      const int tr = base + rr;
      return (size_t)query_token<MODE>(p, sg.row, tr) * p.HQ + sg.h * p.G + tr % p.G;
    };
    bool skip = false;  // no output of this segment
    if constexpr (MODE == DEC_OWN) {
      if (sg.start > 0 && sg.c0 == 0) {
        // The first stream goes on from where the prefix ended; from the parts of a
        // prefix that was cut, joined by all streams where their outputs will be.
        if (!early) rec = p.share.rows[sg.row];
        const int parts = p.cut ? rec.parts : 1;
        auto joined = [&](int rr) {
          return C::JOIN_HERE && parts > 1 ? os + rr * D : p.share.o + out_row(rr) * D;
        };
        if (!early) {
          early_bad = !prefix_holds<C::CT>(p, sg, rec, tid);
          if (parts > 1) join_parts<C, D>(p, sg, rec, base, R, joined, row_m, row_l, tid);
        }
        const bool lost = __ldcg(p.share.lost) != 0;
        skip = named_any(1, C::CT, early_bad || lost);
        if (skip && tid == 0)
          atomicOr(p.err, lost ? (uint32_t)DEVERR_TIMEOUT : (uint32_t)DEVERR_PAGES);
        if (!skip && grp == 0) {
#pragma unroll
          for (int e = 0; e < W::RL; ++e) {
            const int rr = wr + W::row(e, lane);
            if (rr >= R) continue;
            const float2 ml =
                parts > 1 ? make_float2(row_m[rr], row_l[rr]) : p.share.ml[out_row(rr)];
            const float* from = joined(rr);
            w.top(e) = ml.x;
            w.sum(e) = W::tells(lane) ? ml.y : 0.f;
#pragma unroll
            for (int i = 0; i < W::PAIRS; ++i)
              w.set_pair(i, e, *reinterpret_cast<const float2*>(from + W::dim(i, lane)));
          }
        }
        if (parts > 1) named_sync(1, C::CT);  // before the streams' outputs take the room
      }
    }

    // A slot serves one stream's unit after another's, and copies may land out
    // of order. A parity tells a phase only from its neighbours: so a stream
    // first sees that its unit is on its way, which the producer says after
    // the slot's last unit was read, then that it has landed.
    auto landed = [&](int u) {
      if (u >= seen && (seen = *issued) <= u) {
        const unsigned long long t0 = global_ns();
        while ((seen = *issued) <= u) {
          if (global_ns() - t0 > kWaitLimitNs) return false;
        }
      }
      return mbar_wait_bounded(&full[u % C::NU], (uint32_t)((u / C::NU) & 1));
    };
    const int nc = sg.c1 - sg.c0;
    for (int i = (grp + NG - n0 % NG) % NG; i < nc && !dead; i += NG) {
      const int key0 = sg.start + (sg.c0 + i) * C::CH, u = 2 * (n0 + i);
      const int uk = u % C::NU, uv = (u + 1) % C::NU;
      dead = !landed(u);
      std::conditional_t<Q, float[C::CH / 16][Q ? NQ : 1][4], float[1][C::CH / 8][4]> x;
      [[maybe_unused]] int lim1[1][2] = {{lim[0], lim[1]}};
      if constexpr (Q) {
        w.template weights<C::CH / 16>(x, qw, ring + uk * C::UNIT, ring_scales + uk * C::SCALES,
                                       key0, lim, fewest, rf, lane);
      } else {
        w.template weights<C::CH / 8>(x, qw, ring + uk * C::UNIT, key0, lim1, fewest, p.c, lane);
      }
      __syncwarp();
      // A unit that was not seen to land is not given back: the producer would
      // fill a slot, and arm a barrier, whose last copy is still on its way.
      if (lane == 0 && !dead) mbar_arrive(&empty[uk]);
      dead |= !landed(u + 1);
      if constexpr (Q) {
        w.template add<C::CH / 16>(x, ring + uv * C::UNIT, key0, lim, fewest, lane);
      } else {
        w.template add<C::CH / 8>(x, ring + uv * C::UNIT, key0, lim1, fewest, lane);
      }
      dead = __any_sync(kFull, dead);
      if (lane == 0 && !dead) mbar_arrive(&empty[uv]);
    }
    n0 += nc;
    w.finish();

    if (dead) flag[0] = 1;  // no output from here on

    // ---- join the streams
    const bool whole = sg.c0 == 0 && sg.c1 == sg.chunks;
    const bool head = sg.item0 < begin;  // the row began in an earlier CTA
    float* part = p.part + (size_t)(2 * blockIdx.x + (head ? 0 : 1)) * C::PART;
    float f[W::RL], inv[W::RL];
    if constexpr (NG > 1) {
      if (W::tells(lane)) {
#pragma unroll
        for (int e = 0; e < W::RL; ++e) {
          sm_m[grp * C::ROWS + wr + W::row(e, lane)] = w.top(e);
          sm_l[grp * C::ROWS + wr + W::row(e, lane)] = w.sum(e);
        }
      }
      named_sync(1, C::CT);
    }
#pragma unroll
    for (int e = 0; e < W::RL; ++e) {
      const int rr = wr + W::row(e, lane);
      float mx = w.top(e), sum = w.sum(e);
      f[e] = 1.f;
      if constexpr (NG > 1) {
#pragma unroll
        for (int k = 0; k < NG; ++k) mx = fmaxf(mx, sm_m[k * C::ROWS + rr]);
        const float mu = mx == kNegInf ? 0.f : mx;
        f[e] = exp2_fast(w.top(e) - mu);
        sum = 0.f;
#pragma unroll
        for (int k = 0; k < NG; ++k)
          sum += brought<Q>(sm_l[k * C::ROWS + rr], sm_m[k * C::ROWS + rr] - mu);
      }
      inv[e] = 1.f / sum;
      if (grp == 0 && W::tells(lane) && rr < R) {
        row_l[rr] = inv[e];
        if (!whole) {
          part[C::ROWS * D + rr] = mx;
          part[C::ROWS * (D + 1) + rr] = sum;
        } else if constexpr (MODE == DEC_PREFIX) {
          if (flag[0] == 0) p.share.ml[out_row(rr)] = make_float2(mx, sum);
        } else if (p.lse != nullptr && (NG > 1 ? flag[0] == 0 : !dead) && !skip) {
          p.lse[out_row(rr)] = lse_of(mx, sum);
        }
      }
    }
    if constexpr (NG == 1) {
#pragma unroll
      for (int e = 0; e < W::RL; ++e) {
        const int rr = wr + W::row(e, lane);
        if (rr < R && !dead && !(skip && whole)) {
          const size_t at = out_row(rr) * D;
#pragma unroll
          for (int i = 0; i < W::PAIRS; ++i) {
            const auto [a, b] = w.pair(i, e);
            const int d = W::dim(i, lane);
            if (whole) {
              store2(static_cast<T*>(p.o) + at + d, a * inv[e], b * inv[e]);
            } else {
              *reinterpret_cast<float2*>(part + rr * D + d) = make_float2(a, b);
            }
          }
        }
      }
    } else {
#pragma unroll
      for (int s = 0; s < D / 64; ++s) {
#pragma unroll
        for (int e = 0; e < W::RL; ++e) {
          const int rr = wr + W::row(e, lane);
          if (rr < R) {
#pragma unroll
            for (int i = 0; i < W::PAIRS * 64 / D; ++i) {
              const float2 y = w.pair(W::PAIRS * 64 / D * s + i, e);
              *reinterpret_cast<float2*>(os + (grp * C::ROWS + rr) * C::OP + W::dim(i, lane)) =
                  make_float2(y.x * f[e], y.y * f[e]);
            }
          }
        }
        named_sync(1, C::CT);
        const bool ok = flag[0] == 0 && !skip;
#pragma unroll 2
        for (int i = tid; i < R * 16; i += C::CT) {
          const int rr = i / 16, d = 4 * (i % 16);
          float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int k = 0; k < NG; ++k) {
            const float4 y =
                *reinterpret_cast<const float4*>(os + (k * C::ROWS + rr) * C::OP + d);
            a.x += y.x;
            a.y += y.y;
            a.z += y.z;
            a.w += y.w;
          }
          if (!whole) {
            *reinterpret_cast<float4*>(part + rr * D + 64 * s + d) = a;
          } else if (ok) {
            const size_t at = out_row(rr) * D + 64 * s + d;
            if constexpr (MODE == DEC_PREFIX) {
              *reinterpret_cast<float4*>(p.share.o + at) = a;
            } else {
              const float r = row_l[rr];
              T* o = static_cast<T*>(p.o) + at;
              store2(o, a.x * r, a.y * r);
              store2(o + 2, a.z * r, a.w * r);
            }
          }
        }
        if (s + 1 < D / 64) named_sync(1, C::CT);
      }
    }

    if (!whole) {
      // ---- the last part to arrive joins the row's parts
      const int cta0 = (int)(sg.item0 / share);
      const int parts = (int)((sg.item0 + sg.chunks - 1) / share) - cta0 + 1;
      named_sync(1, C::CT);
      if (tid == 0) {
        __threadfence();  // the CTA's part, and after the count the others'
        flag[1] = count_part(p.count, sg.item0, sg.chunks, share, flag[0] != 0 || skip);
        __threadfence();
      }
      named_sync(1, C::CT);
      if (flag[1]) {
        const size_t stride = C::PART;
        // part k of the row: the first CTA's second slot, then first slots
        const float* parts0 = p.part + (size_t)(2 * cta0 + 1) * stride;
        const float* partsn = p.part + (size_t)(2 * cta0) * stride;
        auto at_part = [&](int k) { return k == 0 ? parts0 : partsn + (size_t)2 * k * stride; };
        {
          // all rows' statistics at once, LPR lanes to a row
          constexpr int LPR = C::ROWS <= 16 ? 8 : C::ROWS <= 48 ? 4 : 2;
          static_assert(C::ROWS * LPR <= C::CT || C::F32, "a lane group for each row");
          const int sub = tid % LPR;
          for (int rr = tid / LPR; rr < C::ROWS; rr += C::CT / LPR) {
            float mx = kNegInf, sum = 0.f;
            if (rr < R) {
#pragma unroll 4
              for (int k = sub; k < parts; k += LPR) {
                const float mk = __ldcg(at_part(k) + C::ROWS * D + rr);
                const float lk = __ldcg(at_part(k) + C::ROWS * (D + 1) + rr);
                const float to = fmaxf(mx, mk), mu = to == kNegInf ? 0.f : to;
                sum = brought<Q>(sum, mx - mu) + brought<Q>(lk, mk - mu);
                mx = to;
              }
            }
#pragma unroll
            for (int d = 1; d < LPR; d <<= 1) {
              const float mk = __shfl_xor_sync(kFull, mx, d), lk = __shfl_xor_sync(kFull, sum, d);
              const float to = fmaxf(mx, mk), mu = to == kNegInf ? 0.f : to;
              // the same order on both sides, so that every lane has the same sum
              const float a = brought<Q>(sum, mx - mu), b = brought<Q>(lk, mk - mu);
              sum = (sub & d) ? b + a : a + b;
              mx = to;
            }
            if (sub == 0 && rr < R) {
              row_m[rr] = mx == kNegInf ? 0.f : mx;
              row_l[rr] = 1.f / sum;
              if constexpr (MODE == DEC_PREFIX) {
                p.share.ml[out_row(rr)] = make_float2(mx, sum);
              } else if (p.lse != nullptr) {
                p.lse[out_row(rr)] = lse_of(mx, sum);
              }
            }
          }
        }
        named_sync(1, C::CT);
        // kJoin values of four a thread at a time, so that a part's loads go out
        // together: the loop over the parts is one trip to L2 each
        constexpr int kJoin = C::ROWS >= 32 ? 8 : 4;
        for (int i0 = tid; i0 < R * (D / 4); i0 += C::CT * kJoin) {
          float4 a[kJoin];
#pragma unroll
          for (int j = 0; j < kJoin; ++j) a[j] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
          for (int k = 0; k < parts; ++k) {
            const float* pk = at_part(k);
            float4 y[kJoin];
            float fk[kJoin];
#pragma unroll
            for (int j = 0; j < kJoin; ++j) {
              const int i = i0 + j * C::CT;
              if (i < R * (D / 4)) {
                y[j] = __ldcg(reinterpret_cast<const float4*>(pk) + i);
                fk[j] = __ldcg(pk + C::ROWS * D + i / (D / 4));
              }
            }
#pragma unroll
            for (int j = 0; j < kJoin; ++j) {
              const int i = i0 + j * C::CT;
              if (i < R * (D / 4)) {
                const float e = exp2_fast(fk[j] - row_m[i / (D / 4)]);
                a[j].x = fmaf(e, y[j].x, a[j].x);
                a[j].y = fmaf(e, y[j].y, a[j].y);
                a[j].z = fmaf(e, y[j].z, a[j].z);
                a[j].w = fmaf(e, y[j].w, a[j].w);
              }
            }
          }
#pragma unroll
          for (int j = 0; j < kJoin; ++j) {
            const int i = i0 + j * C::CT;
            if (i < R * (D / 4)) {
              const int rr = i / (D / 4), d = 4 * (i % (D / 4));
              if constexpr (MODE == DEC_PREFIX) {
                *reinterpret_cast<float4*>(p.share.o + out_row(rr) * D + d) = a[j];
              } else {
                const float r = row_l[rr];
                T* o = static_cast<T*>(p.o) + out_row(rr) * D + d;
                store2(o, a[j].x * r, a[j].y * r);
                store2(o + 2, a[j].z * r, a[j].w * r);
              }
            }
          }
        }
      }
    }
    // shared memory, and this half of the segments, are free for the next
    if (NG > 1 || !whole) named_sync(1, C::CT);
    __syncwarp();
    if (lane == 0) mbar_arrive(&qempty[half]);
  }
  if (dead && lane == 0) {
    atomicOr(p.err, DEVERR_TIMEOUT);
    if constexpr (MODE == DEC_PREFIX) atomicExch(p.share.lost, 1);
  }
}

// The kernels of one page type, by head size and warps of a stream: launches, or,
// with p null, only asks for their shared memory.
template <typename T, int NQ, int MODE, int D, int MW>
cudaError_t decode_one(const DecodeParams* p, const void* maps, int sms, cudaStream_t st) {
  using C = DecCfg<T, D, MW, NQ>;
  const auto kernel = attn_decode_kernel<T, D, MW, NQ, MODE>;
  if (p == nullptr)
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if constexpr (MODE == DEC_OWN) {
    // Up to two turns of CTAs for rows with few keys, an item each: 20 groups of 4
    // rows with four heads, 320 items for 304 places, 179 us of four layers, by the
    // line 191.
    DecodeParams own = *p;
    own.line_ctas = C::CPS * sms;
    const long long items = (long long)p->B * p->HKV * p->nmb;
    const bool turns = items > own.line_ctas && items <= 2 * own.line_ctas;
    const int grid = turns ? (int)items : own.line_ctas;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(C::NT);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = st;
    // Its CTAs may start while the prefixes' launch runs, but not beside PREFIX, which
    // has its parts in the same work buffer.
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = p->cut;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, own, *static_cast<const KvMaps*>(maps));
  } else {
    kernel<<<C::CPS * sms, C::NT, C::SMEM, st>>>(*p, *static_cast<const KvMaps*>(maps));
  }
  return cudaGetLastError();
}

// The kernel for blocks of `rows` query rows (attn_decode_block_rows).
template <typename T, bool Q, int MODE, int D>
cudaError_t decode_of_size(const DecodeParams* p, const void* maps, int rows, int sms,
                           cudaStream_t st) {
  const bool all = p == nullptr;
  cudaError_t e = all ? cudaSuccess : cudaErrorInvalidValue;
#define RSSM_ROWS(NQ, MW)                                                    \
  if (e == cudaSuccess || !all) {                                           \
    if (all || rows == DecCfg<T, D, MW, NQ>::ROWS) {                         \
      e = decode_one<T, NQ, MODE, D, MW>(p, maps, sms, st);                  \
      if (!all) return e;                                                    \
    }                                                                        \
  }
  if constexpr (Q) {
    RSSM_ROWS(1, 1)
    RSSM_ROWS(2, 1)
    RSSM_ROWS(2, 2)
    if constexpr (D == 256) { RSSM_ROWS(2, 3) } else { RSSM_ROWS(2, 4) }
  } else {
    RSSM_ROWS(0, 1)
    if constexpr (!std::is_same<T, float>::value) {
      if constexpr (MODE == DEC_PLAIN) { RSSM_ROWS(0, 2) }
      if constexpr (D == 256) { RSSM_ROWS(0, 3) } else { RSSM_ROWS(0, 4) }
    }
  }
#undef RSSM_ROWS
  return e;
}

template <typename T, bool Q, int MODE>
cudaError_t decode_any(const DecodeParams* p, const void* maps, int D, int rows, int sms,
                       cudaStream_t st) {
  if (D == 64) return decode_of_size<T, Q, MODE, 64>(p, maps, rows, sms, st);
  if (D == 128) return decode_of_size<T, Q, MODE, 128>(p, maps, rows, sms, st);
  if (D == 256) return decode_of_size<T, Q, MODE, 256>(p, maps, rows, sms, st);
  return cudaErrorInvalidValue;
}

}  // namespace

}  // namespace rssm
