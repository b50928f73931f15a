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
#include "attn_core.cuh"
#include "attn_tma.h"
#include "kv_common.cuh"

namespace rssm {

namespace {

constexpr int kBox = 16;        // keys of a TMA box: within one page (pages of 16 k keys)
constexpr int kGapKeys = 256;   // what beginning and ending a row costs, as keys
constexpr int kLeastKeys = 512; // keys that a CTA takes at least (of longer rows)
constexpr int kRowParts = 96;   // parts of the longest row, about: one CTA joins them
constexpr int kLostPart = 1 << 16;  // in a row's arrivals, beside their number: a part that is not there

template <typename T, int D, int MW>
struct DecCfg {
  static constexpr bool F32 = std::is_same<T, float>::value;
  // Outputs live in registers, D / 2 a lane: seven warps of 255 registers for
  // D = 256, ten of 168 for 128, fifteen of 128 for 64 (eight of 255 for fp32,
  // whose FMAs want more). A quarter of the registers belongs to each quarter
  // of the SM. Where they suffice a step takes 32 keys: what a step costs
  // whatever its size (waits, maxima over lanes) is most of it.
  static constexpr int CPS = D == 256 ? 1 : F32 || D == 128 ? 2 : 3;  // CTAs per SM
  static constexpr int NW = F32 ? (D == 256 ? 4 : 3) : D == 256 ? 6 : 4;
  static constexpr int CH = F32 || D == 256 ? 16 : 32;  // keys of a chunk
  static constexpr int GAP = kGapKeys / CH;
  static constexpr int CT = NW * 32;                   // threads of the streams
  static constexpr int NT = CT + 32;                   // and the producer warp
  static constexpr int NG = NW / MW;                   // streams of a CTA
  static constexpr int ROWS = 16 * MW;
  static constexpr int UNIT = CH * D * (int)sizeof(T);
  static constexpr int QBYTES = ROWS * D * (int)sizeof(T);
  static constexpr int OP = 72;                        // row pitch of 64 columns of outputs
  static constexpr int OBYTES = NG > 1 ? NG * ROWS * OP * 4 : 0;
  static constexpr int REST = 1024 + 2 * QBYTES + OBYTES + 2 * NG * ROWS * 4 + ROWS * 8 + 1024;
  static constexpr int MOST = (228 / CPS - 1) * 1024;  // a CTA's share of the SM
  static_assert(NW % MW == 0, "whole streams");
  static constexpr int FIT = (MOST - REST) / UNIT;
  static constexpr int NU = FIT < 32 ? FIT : 32;       // units in the ring
  static constexpr int SMEM = NU * UNIT + REST;
  static constexpr int PART = ROWS * (D + 2);          // floats of a part
  static_assert(NU >= 2 * NG, "a chunk for each stream");
  static_assert(CPS * kMaxSms * 2 * PART <= kPartFloats, "work buffer");
};

// keys of row r (committed and new), 0 for a null or refused row
__device__ __forceinline__ int row_keys(const DecodeParams& p, int r, bool tell, int& s) {
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
    }
  }
  if (bad && tell) atomicOr(p.err, bad);
  return n;
}

// places of a row's chunks of CH keys on the line, with the gap before them
template <int CH>
__device__ __forceinline__ long long places(int keys) {
  return keys > 0 ? ((long long)keys + CH - 1) / CH + kGapKeys / CH : 0;
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
  int more, pad;    // 0: the stretch is done
};

// The CTA's stretch of the line, one Seg after the other.
template <int CH>
struct Line {
  static constexpr int kGap = kGapKeys / CH;
  long long pos, end, row0;
  int row;
  __device__ __forceinline__ bool next(const DecodeParams& p, Seg& g) {
    const int items = p.HKV * p.nmb;
    while (pos < end) {
      g.keys = row_keys(p, row, false, g.slot);
      const int cost = (int)places<CH>(g.keys);
      if (pos >= row0 + (long long)cost * items) {
        row0 += (long long)cost * items;
        ++row;
        continue;
      }
      const int item = (int)((pos - row0) / cost);
      const int off = (int)((pos - row0) % cost);
      const int len = (long long)cost - off <= end - pos ? cost - off : (int)(end - pos);
      g.row = row;
      g.h = item / p.nmb;
      g.mb = item % p.nmb;
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
template <int CH>
__device__ __noinline__ void give_up(const DecodeParams& p, Line<CH> line, int ns,
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

template <typename T, int D, int MW>
__global__ void __launch_bounds__(DecCfg<T, D, MW>::NT, DecCfg<T, D, MW>::CPS)
    attn_decode_kernel(const __grid_constant__ DecodeParams p,
                       const __grid_constant__ KvMaps maps) {
  using C = DecCfg<T, D, MW>;
  constexpr int NG = C::NG, NW = C::NW;
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
  // ---- the line's length and its longest row, and the row that holds this
  // CTA's first place: one look at the lengths for up to NT rows, else two
  const int items = p.HKV * p.nmb;
  long long mine = 0, most = 0, first_w = 0;
  for (int r = tid; r < p.B; r += C::NT) {
    int s;
    const long long w = places<C::CH>(row_keys(p, r, blockIdx.x == 0, s)) * items;
    if (r < C::NT) first_w = w;
    mine += w;
    most = w > most ? w : most;
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
  long long share = (total + gridDim.x - 1) / gridDim.x;
  const long long few = longest / items / kRowParts + 1;
  share = share > few ? share : few;
  // not less than kLeastKeys, or a whole row where the longest has fewer
  const long long row_cost = longest / items;
  const long long least =
      row_cost < C::GAP + kLeastKeys / C::CH ? row_cost : C::GAP + kLeastKeys / C::CH;
  share = share > least ? share : least;
  Line<C::CH> line;
  line.pos = share * blockIdx.x;
  line.end = line.pos + share < total ? line.pos + share : total;
  if (line.pos >= line.end) return;
  at += first_incl - first_w;
  long long* found = scan + 3 * (NW + 1);  // row, its first place
  if (at <= line.pos && line.pos < at + first_w) {
    found[0] = tid;
    found[1] = at;
  }
  long long before = firsts;
  for (int r0 = C::NT; r0 < p.B && before <= line.pos; r0 += C::NT) {
    int s;
    const long long w =
        r0 + tid < p.B ? places<C::CH>(row_keys(p, r0 + tid, false, s)) * items : 0;
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

  const long long begin = line.pos;
  // for a CTA that gives up; the sums that stood there have been read
  Line<C::CH>* from_start = reinterpret_cast<Line<C::CH>*>(scan);
  static_assert(sizeof(Line<C::CH>) <= 3 * 8 * (NW + 1), "behind the barriers");
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
      if (ns >= 2) dead = !mbar_wait_bounded(&qempty[half], (uint32_t)((ns / 2 - 1) & 1));
      dead = __any_sync(kFull, dead);
      if (dead) break;
      if (lane == 1) {  // lane 0 has bulk copies on their way, which a release would wait for
        segs[half] = sg;
        mbar_arrive(&qfull[half]);
      }
      if (sg.more) {
        constexpr int QU = D * (int)sizeof(T) / 16;  // units per row
        const int base = sg.mb * C::ROWS, R = min(C::ROWS, p.T * p.G - base);
        const uint32_t qd = smem_addr(qs + half * C::QBYTES);
#pragma unroll 4
        for (int i = lane; i < C::ROWS * QU; i += 32) {
          const int rr = i / QU, u = i % QU;
          const int tr = base + (rr < R ? rr : 0);
          const T* q = static_cast<const T*>(p.q) + ((long long)sg.row * p.T + tr / p.G) * p.qs +
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
      const int b_end = min(sg.c1 * BPC, (sg.keys + kBox - 1) / kBox);
      for (int cb = sg.c0; cb < sg.c1 && !dead; cb += 32 / BPC) {
        const int box = cb * BPC + lane;
        int row = -1;  // of the pool: ((layer pages + page) HKV + head) page_size + token
        if (box < b_end) {
          const long long tok = (long long)box * kBox;
          int page = tab[tok >> p.shift];
          if (page < 0 || page >= p.n_pages) {
            page = 0;  // the row's output is undefined; nothing outside the pool is read
            atomicOr(p.err, DEVERR_PAGES);
          }
          row = (int)((((p.page0 + page) * p.HKV + sg.h) << p.shift) +
                      (tok & ((1 << p.shift) - 1)));
        }
        const int cnt = min(32 / BPC, sg.c1 - cb);
        for (int i = 0; i < cnt; ++i) {
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
  const int grp = warp / MW, wr = 16 * (warp % MW);  // the warp's stream, its first row
  const int g = lane >> 2, tq = lane & 3;
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
    const int R = min(C::ROWS, p.T * p.G - base);      // rows in use
    // how many keys the lane's rows see
    const int first = sg.keys - p.T;  // committed keys
    int lim[1][2];
#pragma unroll
    for (int e = 0; e < 2; ++e)
      lim[0][e] = first + (base + min(wr + 8 * e + g, R - 1)) / p.G + 1;
    const int fewest = first + (base + min(wr, R - 1)) / p.G + 1;
    WarpAttn<T, D, 1, C::ROWS, kBox> w;
    w.clear();
    const unsigned char* qw = qs + half * C::QBYTES + wr * 128;

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
      const int key0 = (sg.c0 + i) * C::CH, u = 2 * (n0 + i);
      const int uk = u % C::NU, uv = (u + 1) % C::NU;
      float x[1][C::CH / 8][4];
      dead = !landed(u);
      w.template weights<C::CH / 8>(x, qw, ring + uk * C::UNIT, key0, lim, fewest, p.c, lane);
      __syncwarp();
      // A unit that was not seen to land is not given back: the producer would
      // fill a slot, and arm a barrier, whose last copy is still on its way.
      if (lane == 0 && !dead) mbar_arrive(&empty[uk]);
      dead |= !landed(u + 1);
      w.template add<C::CH / 8>(x, ring + uv * C::UNIT, key0, lim, fewest, lane);
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
    auto out_row = [&](int rr) {
      const int tr = base + rr;
      return ((size_t)sg.row * p.T + tr / p.G) * p.HQ + sg.h * p.G + tr % p.G;
    };
    float f[2], inv[2];
    if constexpr (NG > 1) {
      if (tq == 0) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          sm_m[grp * C::ROWS + wr + 8 * e + g] = w.m[0][e];
          sm_l[grp * C::ROWS + wr + 8 * e + g] = w.l[0][e];
        }
      }
      named_sync(1, C::CT);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int rr = wr + 8 * e + g;
      float mx = w.m[0][e], sum = w.l[0][e];
      f[e] = 1.f;
      if constexpr (NG > 1) {
#pragma unroll
        for (int k = 0; k < NG; ++k) mx = fmaxf(mx, sm_m[k * C::ROWS + rr]);
        const float mu = mx == kNegInf ? 0.f : mx;
        f[e] = exp2_fast(w.m[0][e] - mu);
        sum = 0.f;
#pragma unroll
        for (int k = 0; k < NG; ++k)
          sum += sm_l[k * C::ROWS + rr] * exp2_fast(sm_m[k * C::ROWS + rr] - mu);
      }
      inv[e] = 1.f / sum;
      if (grp == 0 && tq == 0 && rr < R) {
        row_l[rr] = inv[e];
        if (!whole) {
          part[C::ROWS * D + rr] = mx;
          part[C::ROWS * (D + 1) + rr] = sum;
        } else if (p.lse != nullptr && (NG > 1 ? flag[0] == 0 : !dead)) {
          p.lse[out_row(rr)] = lse_of(mx, sum);
        }
      }
    }
    if constexpr (NG == 1) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int rr = wr + 8 * e + g;
        if (rr < R && !dead) {
          T* o = static_cast<T*>(p.o) + out_row(rr) * D;
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            const float a = w.o[0][i][2 * e], b = w.o[0][i][2 * e + 1];
            if (whole) {
              store2(o + w.col(i, tq), a * inv[e], b * inv[e]);
            } else {
              *reinterpret_cast<float2*>(part + rr * D + w.col(i, tq)) = make_float2(a, b);
            }
          }
        }
      }
    } else {
#pragma unroll
      for (int s = 0; s < D / 64; ++s) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int rr = wr + 8 * e + g;
          if (rr < R) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<float2*>(os + (grp * C::ROWS + rr) * C::OP + w.col(i, tq)) =
                  make_float2(w.o[0][8 * s + i][2 * e] * f[e],
                              w.o[0][8 * s + i][2 * e + 1] * f[e]);
          }
        }
        named_sync(1, C::CT);
        const bool ok = flag[0] == 0;
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
            const float r = row_l[rr];
            T* o = static_cast<T*>(p.o) + out_row(rr) * D + 64 * s + d;
            store2(o, a.x * r, a.y * r);
            store2(o + 2, a.z * r, a.w * r);
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
        flag[1] = count_part(p.count, sg.item0, sg.chunks, share, flag[0] != 0);
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
                sum = sum * exp2_fast(mx - mu) + lk * exp2_fast(mk - mu);
                mx = to;
              }
            }
#pragma unroll
            for (int d = 1; d < LPR; d <<= 1) {
              const float mk = __shfl_xor_sync(kFull, mx, d), lk = __shfl_xor_sync(kFull, sum, d);
              const float to = fmaxf(mx, mk), mu = to == kNegInf ? 0.f : to;
              // the same order on both sides, so that every lane has the same sum
              const float a = sum * exp2_fast(mx - mu), b = lk * exp2_fast(mk - mu);
              sum = (sub & d) ? b + a : a + b;
              mx = to;
            }
            if (sub == 0 && rr < R) {
              row_m[rr] = mx == kNegInf ? 0.f : mx;
              row_l[rr] = 1.f / sum;
              if (p.lse != nullptr) p.lse[out_row(rr)] = lse_of(mx, sum);
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
              const float r = row_l[rr];
              T* o = static_cast<T*>(p.o) + out_row(rr) * D + d;
              store2(o, a[j].x * r, a[j].y * r);
              store2(o + 2, a[j].z * r, a[j].w * r);
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
  if (dead && lane == 0) atomicOr(p.err, DEVERR_TIMEOUT);
}

// warps that share a stream's keys, sixteen rows each
int warps_for(int D, int dt, int rows) {
  if (dt == DT_F32 || rows <= 16) return 1;
  return rows <= 32 ? 2 : D == 256 ? 3 : 4;
}

template <typename F>
cudaError_t pick(int D, int dt, int mw, F f) {
#define RSSM_CASE(TT, DD, MM)                                                      \
  if (D == DD && mw == MM)                                                         \
    return f(attn_decode_kernel<TT, DD, MM>, DecCfg<TT, DD, MM>::NT, DecCfg<TT, DD, MM>::SMEM, \
             DecCfg<TT, DD, MM>::CPS);
#define RSSM_CASES(TT, MM) RSSM_CASE(TT, 64, MM) RSSM_CASE(TT, 128, MM) RSSM_CASE(TT, 256, MM)
#define RSSM_CASES16(TT)                                                           \
  RSSM_CASES(TT, 1) RSSM_CASES(TT, 2) RSSM_CASE(TT, 64, 4) RSSM_CASE(TT, 128, 4)   \
  RSSM_CASE(TT, 256, 3)
  if (dt == DT_F32) {
    RSSM_CASES(float, 1)
  } else if (dt == DT_BF16) {
    RSSM_CASES16(__nv_bfloat16)
  } else {
    RSSM_CASES16(__half)
  }
#undef RSSM_CASES16
#undef RSSM_CASES
#undef RSSM_CASE
  return cudaErrorInvalidValue;
}

}  // namespace

int attn_decode_block_rows(int D, int dt, int rows) { return 16 * warps_for(D, dt, rows); }

cudaError_t attn_decode_prepare(int D, int dt) {
  for (int rows = 16; rows <= 64; rows *= 2) {
    const cudaError_t e = pick(D, dt, warps_for(D, dt, rows), [](auto kernel, int, int smem, int) {
      return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    });
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

// The pool as rows of 128-byte columns: a box is one chunk of one head.
cudaError_t attn_decode_maps(void* maps, const void* k, const void* v, long long rows, int D,
                             int dt) {
  static_assert(sizeof(KvMaps) == kKvMapBytes, "two tensor maps");
  if (tma_encoder() == nullptr) return cudaErrorNotSupported;
  const cuuint64_t es = dtype_bytes(dt), inner = 128 / es;
  const cuuint64_t dims[3] = {inner, (cuuint64_t)rows, D * es / 128};
  const cuuint64_t strides[2] = {D * es, 128};
  const cuuint32_t box[3] = {(cuuint32_t)inner, kBox, (cuuint32_t)(D * es / 128)};
  const cuuint32_t ones[3] = {1, 1, 1};
  KvMaps* m = static_cast<KvMaps*>(maps);
  for (int i = 0; i < 2; ++i) {
    if (tma_encoder()(i == 0 ? &m->k : &m->v,
                      dt == DT_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                      : dt == DT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                      : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                      3, const_cast<void*>(i == 0 ? k : v), dims, strides, box, ones,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                      CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  return cudaSuccess;
}

cudaError_t attn_decode_launch(const DecodeParams& p, const void* maps, int D, int dt, int num_sms,
                               cudaStream_t st) {
  const int sms = num_sms < kMaxSms ? num_sms : kMaxSms;
  const KvMaps& m = *static_cast<const KvMaps*>(maps);
  return pick(D, dt, warps_for(D, dt, p.T * p.G), [&](auto kernel, int nt, int smem, int cps) {
    kernel<<<cps * sms, nt, smem, st>>>(p, m);
    return cudaGetLastError();
  });
}

}  // namespace rssm
