// Attention of a group's query rows over the prefix that they share, on the
// 5th-generation tensor cores: the first launch of attention over shared
// prefixes (kv_share.cu) for all but fp32 pages.
//
// All rows see all of the prefix, so it is a matrix product with a softmax in
// it. A CTA takes 128 query rows of one key head, from whichever members of the
// group, and a stretch of the prefix in steps of 128 keys:
//
//     S = Q K^T             tensor memory, 128 x 128 fp32, two in turn
//     P = 2^(c S - c m)     registers, stored over S as 16-bit operand
//     O = O + P V           tensor memory, 128 x D fp32
//
// The plan says how many steps make a stretch, so that the stretches of all
// groups fill the SMs once; where a prefix is cut, each stretch leaves its
// maxima, sums and outputs in the caller's buffer, and the rows' second launch
// joins them. While one step's weights are computed the next one's scores are: a
// producer warp sends for pages, another warp issues the products, a warpgroup
// does the softmax, a thread to a row (attn_prompt_tc.cu has the same parts; the
// reference maximum moves only when a weight would pass 2^8, in fp16 2^15.5).
//
// e4m3 pages: eight more warps turn codes into fp16 in shared memory, and the
// products are those of fp16, whatever the cache's type (a query row is scaled by a
// power of two into fp16's range, as in attn_quant.cuh). With e and f the exponents
// of a key's and a value's power of two, E and F the largest among the step's 128:
//  - even steps: codes times 2^(e - E) and 2^(f - F), which fp16 holds exactly down
//    to a difference of 15. A step has one factor for all its scores, c' = c 2^a 2^E,
//    and one for its values, which the reference m follows,
//        w = 2^(c' s + F - m),   l = l + 2^-F sum w,   O = O + w V'.
//    The weights' headroom is that of a token of F, so f may differ by 6 only (a weight
//    below 2^-17 of the largest is off by 2^-28 of it at most); and F itself has its
//    bounds, so that no w falls out of fp32's range beside another step's.
//  - other steps: codes as they are, powers column by column in fp32,
//        x = (c 2^a) (2^e s),   p = 2^(x - m),   w = 2^f p,   l = l + sum p,
//    and m follows x + f: no token's size matters for another's.
// Both are exact but for the rounding of w to fp16. The second takes longer (20 groups of
// 4 rows, four layers: 310 us if every step goes that way, 187 if none does), and a
// model's tokens hardly differ like that.
//
// Measured (GB300): a step of heads of 128 takes 0.85 us of 16-bit pages, of which its
// products are 0.55, and 1.68 of e4m3 ones (shared memory: codes read, fp16 written,
// operands read), 64 blocks of rows behind 2.4 to 22 k keys. 64 rows behind 8200 keys,
// four key heads: 9 to 11 us a layer, of which the bytes would take 2.5 and two steps a
// CTA 1.7; the rest are the trips to the plan, the queries, the table and the first keys,
// and the way out.
//
// Even a group of few rows takes the whole instruction, whose 128 rows cost less
// than the prefix's bytes take to arrive: 128 keys of 128 values are 64 KB, 1.5
// us of an SM's share of the memory, and 0.55 us of products.
#pragma once

#include "attn_decode.cuh"
#include "attn_prompt_tc.cuh"

namespace rssm {

namespace {

template <int D, bool Q8>
struct SharedTcCfg {
  static constexpr int QS = 128 * D * 2;                   // the queries
  static constexpr int UNIT = 128 * D * 2;                 // a step's keys, or its values
  static constexpr int NU = D == 256 ? 2 : D == 128 ? (Q8 ? 4 : 6) : 8;  // units in the ring
  static constexpr int RAW = Q8 ? 128 * D : 0;             // the same as codes
  static constexpr int NR = !Q8 ? 0 : D == 256 ? 1 : D == 128 ? 3 : 4;
  static constexpr int NT = 256 + (Q8 ? 256 : 0);
  static constexpr int RING = QS;
  static constexpr int RAWS = RING + NU * UNIT;
  static constexpr int SCALES = RAWS + NR * RAW;           // [NR][128][2] bytes
  // Steps whose powers are kept: the converters begin step j's keys when they are done
  // with the values before them, whose place was free because step j - 1 - NU / 2 has
  // its weights.
  static constexpr int NE = Q8 ? NU / 2 + 1 : 0;
  static constexpr int POWERS = SCALES + NR * 256;         // [NE][128][2] bytes
  static constexpr int BARS = POWERS + NE * 256;
  // the queries' places as they are, or where room is short as rows and heads
  static constexpr bool FAR = !(Q8 && D == 256);
  // barriers, the rows' places (then their powers of two), the steps' E and F
  static constexpr int REST =
      (16 * (NU + NR) + 96 + (FAR ? 1024 : 512) + (Q8 && FAR ? 512 : 0) + 16 * NE + 127) / 128 * 128;
  static constexpr int SMEM = BARS + REST + 1024;          // + alignment of the base
  static constexpr uint32_t O0 = 256;                      // first column of O
  static_assert(SMEM <= 227 * 1024, "shared memory");
};

// What an even step's bytes of powers may differ by, and the bytes that its values' may
// have.
constexpr unsigned kEvenKeys = 15, kEvenValues = 6;
constexpr unsigned kEvenLeast = kScaleBias - 30, kEvenMost = kScaleBias + 30;
constexpr int kUneven = 1 << 20;  // in the place of E

// Of a word with the powers' bytes of two tokens (key's and value's, twice): 2^e, 2^f
// and f of both. The bytes are biased as fp32's exponents are.
__device__ __forceinline__ uint64_t key_powers(uint32_t w) {
  return f2(__uint_as_float(w << 23 & 0x7f800000u), __uint_as_float(w << 7 & 0x7f800000u));
}
__device__ __forceinline__ uint64_t value_powers(uint32_t w) {
  return f2(__uint_as_float(w << 15 & 0x7f800000u), __uint_as_float(w >> 1 & 0x7f800000u));
}
__device__ __forceinline__ uint64_t value_exponents(uint32_t w) {
  constexpr float kBias = -(8388608.f + kScaleBias);  // 2^23: a byte is its last places
  return add2(f2(__uint_as_float(__byte_perm(w, 0x4B000000u, 0x7441)),
                 __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7443))),
              f2(kBias, kBias));
}

struct SharedTcMaps {
  CUtensorMap k, v;
};

template <typename T, int D, bool Q8>
__global__ void __launch_bounds__(SharedTcCfg<D, Q8>::NT, 1)
    attn_shared_tc_kernel(const __grid_constant__ DecodeParams p,
                          const __grid_constant__ SharedTcMaps maps) {
  using C = SharedTcCfg<D, Q8>;
  using M = std::conditional_t<Q8, __half, T>;  // what is multiplied
  extern __shared__ unsigned char sm_raw[];
  unsigned char* sm = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(sm_raw) + 1023) & ~(uintptr_t)1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + C::BARS);  // [NU] a unit is there
  uint64_t* empty = full + C::NU;                              // [NU] its products are done
  uint64_t* rfull = empty + C::NU;                             // [NR] its codes have landed
  uint64_t* rempty = rfull + C::NR;                            // [NR] and were turned
  uint64_t* sfull = rempty + C::NR;                            // [2] scores are in tensor memory
  uint64_t* pfull = sfull + 2;                                 // [2] and the weights
  // a step's P V is done: two in turn, because not every step's is waited for, and
  // the next but one is only issued when this one is known to be over
  uint64_t* odone = pfull + 2;                                 // [2]
  uint64_t* drained = odone + 2;                               // no product is in flight
  uint64_t* qfull = drained + 1;                               // the queries are there
  uint64_t* efull = qfull + 1;                                 // [NE] a step's powers are there
  uint32_t* tslot = reinterpret_cast<uint32_t*>(efull + C::NE);
  volatile uint32_t* gave_up = tslot + 1;  // a wait ran out: nothing is stored any more
  const int tid = threadIdx.x, warp = __shfl_sync(kFull, tid >> 5, 0), lane = tid & 31;

  asm volatile("griddepcontrol.launch_dependents;");  // the rows' launch
  // ---- the CTA's stretch
  const ShareView& sv = p.share;
  static_assert(sizeof(ShareSeg) == 32, "two vectors");
  const int4 s_a = reinterpret_cast<const int4*>(sv.segs + blockIdx.x)[0];
  const int4 s_b = reinterpret_cast<const int4*>(sv.segs + blockIdx.x)[1];
  const int per = *sv.steps;
  if (!share_is_of(sv, p.B, p.T) || (int)blockIdx.x >= *sv.segments) return;
  const int begin = s_a.x;
  int slot = p.slot[s_a.y];
  if (slot < 0 || slot >= p.n_slots) slot = lead_slot(p, s_a.z);
  if (slot < 0) return;
  const int keys = min(s_a.w, p.max_pages << p.shift);
  const long long rows = s_b.x;
  const int blocks = (int)((rows + 127) / 128);
  const int part = s_b.z, blk = s_b.y % blocks, h = s_b.y / blocks;
  const int steps = (keys + 127) / 128;
  const int s0 = part * per, ns = min(steps, s0 + per) - s0;
  if (ns <= 0 || h >= p.HKV) return;
  const int R = (int)min(128ll, rows - 128ll * blk);
  bool dead = false;
  if (warp == 4 && lane == 0) {
    for (int u = 0; u < C::NU; ++u) mbar_init(&full[u], Q8 ? 256 : 1), mbar_init(&empty[u], 1);
    for (int u = 0; u < C::NR; ++u) mbar_init(&rfull[u], 1), mbar_init(&rempty[u], 256);
    for (int b = 0; b < 2; ++b)
      mbar_init(&sfull[b], 1), mbar_init(&pfull[b], 128), mbar_init(&odone[b], 1);
    mbar_init(drained, 1);
    mbar_init(qfull, C::NT - 64);
    for (int i = 0; i < C::NE; ++i) mbar_init(&efull[i], 128);
    *gave_up = 0;
    if (p.hook_cta == (int)blockIdx.x) {
      if constexpr (Q8) mbar_promise(&rfull[p.hook_unit % C::NR], 16);
      else mbar_promise(&full[p.hook_unit % C::NU], 16);
    }
    fence_mbar_init();
  }
  if (warp == 5) tmem_alloc512(tslot);
  // each row's place among the outputs (its thread's), and where its query lies
  unsigned char* places = reinterpret_cast<unsigned char*>(tslot + 2);
  long long* q_at = reinterpret_cast<long long*>(places);  // FAR: [128] elements
  int* row_at = reinterpret_cast<int*>(places);            // else: [128] token HQ + head
  // Q8: [128] 2^a; in a row's place once it is loaded, where that is all there is
  float* row_f = reinterpret_cast<float*>(places + (C::FAR ? 1024 : 0));
  int2* largest = reinterpret_cast<int2*>(places + (C::FAR ? 1536 : 512));  // Q8: [NE] E, F
  int at = 0;  // token HQ + head of row `tid`
  if (tid < 128) {
    if (tid < R) {
      const int tr = 128 * blk + tid, one = p.T * p.G;
      const int token = sv.order[begin + tr / one] * p.T + tr % one / p.G;
      const int head = h * p.G + tr % p.G;
      at = token * p.HQ + head;
      if (C::FAR) q_at[tid] = token * p.qs + (long long)head * D;
    }
    if (!C::FAR) row_at[tid] = at;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tb = *tslot;
  // the queries, by all but the two roles; rows behind the last are zeros
  if (warp != 4 && warp != 5) {
    constexpr int QU = D * 2 / 16;  // units of a row
    constexpr int THREADS = C::NT - 64;
    const int mine = (warp > 5 ? warp - 2 : warp) * 32 + lane;
    constexpr int AHEAD = 11;  // of 192 threads all that heads of 128 have
#pragma unroll 1
    for (int i0 = mine; i0 < 128 * QU; i0 += THREADS * AHEAD) {
      uint4 x[AHEAD];
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        const int i = i0 + k * THREADS;
        x[k] = make_uint4(0, 0, 0, 0);
        if (i < 128 * QU && i / QU < R) {
          long long from;
          if constexpr (C::FAR) {
            from = q_at[i / QU];
          } else {
            const int ra = row_at[i / QU];
            from = ra / p.HQ * p.qs + (long long)(ra % p.HQ) * D;
          }
          x[k] = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) + from) + i % QU);
        }
      }
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        const int i = i0 + k * THREADS;
        if constexpr (Q8) {
          // neighbouring lanes have a row, and all lanes take part
          float f[8], top = 0.f;
          Vec16<T>::unpack(x[k], f);
#pragma unroll
          for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(f[e]) < INFINITY ? fabsf(f[e]) : 0.f);
#pragma unroll
          for (int d = 1; d < QU; d <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, d));
          const int a = query_exponent(top);
          const float down = power_of(-a);
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] *= down;
          x[k] = Vec16<__half>::pack(f);
          if (i < 128 * QU && i % QU == 0) row_f[i / QU] = power_of(a);
        }
        if (i < 128 * QU) *reinterpret_cast<uint4*>(sm + unit_off<128>(i / QU, i % QU)) = x[k];
      }
    }
    fence_async_smem();
    mbar_arrive(qfull);
  }

  // Four warpgroups at 128 registers where there are converters: the softmax's takes
  // 208, that of the roles keeps 64, the converters 120 each.
  if constexpr (Q8) {
    if (warp >= 4 && warp < 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
  }
  if (warp == 4) {
    // ---- producer: keys and values by turns, boxes of up to 128 tokens of a page
    const int32_t* tab = p.table + (size_t)slot * p.max_pages;
    const int box = p.shift < 7 ? 1 << p.shift : 128;  // tokens of a box
    constexpr int COLS = Q8 ? 1 : D / 64;               // boxes side by side in a row
    int sent = 0;  // units sent for
    // the page of the lane's box in step j, looked up a step ahead of its use
    auto page_of = [&](int j) {
      const int tok = (s0 + j) * 128 + lane / COLS * box;
      return j < ns && lane / COLS * box < 128 && tok < keys ? tab[tok >> p.shift] : 0;
    };
    int next = page_of(0);
    for (int j = 0; j < ns; ++j) {
      const int tok0 = (s0 + j) * 128, n = min(128, keys - tok0), boxes = n / box;
      int page = next;
      next = page_of(j + 1);
      int row = 0;  // of the pool, of box lane / COLS
      if (lane / COLS < boxes) {
        const int tok = tok0 + lane / COLS * box;
        if (page < 0 || page >= p.n_pages) {
          page = 0;  // nothing outside the pool is read; the rows' tables differ from this one
          atomicOr(p.err, DEVERR_PAGES);
        }
        row = (int)((((p.page0 + page) * p.HKV + h) << p.shift) + (tok & ((1 << p.shift) - 1)));
      }
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const CUtensorMap* map = kv == 0 ? &maps.k : &maps.v;
        if constexpr (Q8) {
          const int u = sent % C::NR;
          if (sent >= C::NR) tc_wait(&rempty[u], (uint32_t)((sent / C::NR - 1) & 1), dead);
          dead = __any_sync(kFull, dead);
          if (dead) break;
          if (lane == 0) mbar_expect_tx(&rfull[u], (uint32_t)(n * (D + 2)));
          __syncwarp();
          constexpr int WIDE = D == 256 ? 2 : 1;  // a box is 128 bytes wide at most
          if (lane < boxes) {
            for (int w = 0; w < WIDE; ++w)
              tma_load3(smem_addr(sm + C::RAWS + u * C::RAW + w * (128 * 128) +
                                  lane * box * (D / WIDE)),
                        map, 0, row, w, &rfull[u]);
            bulk_g2s(sm + C::SCALES + u * 256 + lane * box * 2, p.scales + 2 * (size_t)row,
                     (uint32_t)(2 * box), &rfull[u]);
          }
        } else {
          const int u = sent % C::NU;
          unsigned char* to = sm + C::RING + u * C::UNIT;
          if (sent >= C::NU) tc_wait(&empty[u], (uint32_t)((sent / C::NU - 1) & 1), dead);
          dead = __any_sync(kFull, dead);
          if (dead) break;
          if (kv == 1 && n < 128) {  // values behind the last: zeros, beside what lands
            zero_rows<D>(to, n, lane);
            __threadfence_block();
            __syncwarp();
          }
          if (lane == 0) mbar_expect_tx(&full[u], (uint32_t)(n * D * 2));
          __syncwarp();
          if (lane < boxes * COLS)
            tma_load3(smem_addr(to + lane % COLS * 16384 + lane / COLS * box * 128), map, 0, row,
                      lane % COLS, &full[u]);
        }
        ++sent;
      }
      if (dead) break;
    }
    // Every copy has landed before the CTA leaves. Once a wait ran out the copies
    // on their way get one more limit between them.
    if (lane == 0) {
      bool late = false;
      constexpr int N = Q8 ? C::NR : C::NU;
      for (int k = max(0, sent - N); k < sent; ++k)
        tc_wait(Q8 ? &rfull[k % N] : &full[k % N], (uint32_t)((k / N) & 1), late);
      dead |= late;
    }
    __syncwarp();
  } else if (warp == 5) {
    // ---- products; the warp stays together and one lane issues
    constexpr uint32_t id_qk = f16_idesc<M>(128, 128, false);
    constexpr uint32_t id_pv = f16_idesc<M>(128, D, true);
    const uint32_t el = elect_lane();
    const uint32_t qd = sw128_kmajor_lo(smem_addr(sm));
    const uint32_t kd = sw128_kmajor_lo(smem_addr(sm + C::RING));
    const uint32_t vd = sw128_mnmajor_lo(smem_addr(sm + C::RING), 16384);
    auto ready = [&](int n) {
      tc_wait(&full[n % C::NU], (uint32_t)((n / C::NU) & 1), dead);
      dead = __any_sync(kFull, dead);
      tc_fence_after();
    };
    // S = Q K^T of step j; units: K0 V0 K1 V1 ...
    auto qk = [&](int j) {
      ready(2 * j);
      if (dead) return;
      const uint32_t b = kd + (2 * j % C::NU) * (C::UNIT / 16);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint32_t in = ((k / 4) * 16384 + (k % 4) * 32) / 16;
        mma16_ss(el, tb + (j & 1) * 128, qd + in, b + in, id_qk, k > 0);
      }
      mma16_commit(el, &sfull[j & 1]);
      mma16_commit(el, &empty[2 * j % C::NU]);
    };
    tc_wait(qfull, 0, dead);
    qk(0);
    for (int j = 0; j < ns && !dead; ++j) {
      if (j + 1 < ns) qk(j + 1);
      if (dead) break;
      ready(2 * j + 1);
      tc_wait(&pfull[j & 1], (uint32_t)((j >> 1) & 1), dead);
      dead = __any_sync(kFull, dead);
      if (dead) break;
      tc_fence_after();
      const uint32_t b = vd + ((2 * j + 1) % C::NU) * (C::UNIT / 16);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        mma16_ts(el, tb + C::O0, tb + (j & 1) * 128 + 8 * k, b + k * 128, id_pv, j > 0 || k > 0);
      mma16_commit(el, &odone[j & 1]);
      mma16_commit(el, &empty[(2 * j + 1) % C::NU]);
    }
    if (dead) {  // products in flight end before their memory is given back
      bool late = false;
      mma16_commit(el, drained);
      tc_wait(drained, 0, late);
    }
    __syncwarp();
  } else if (warp < 4) {
    if constexpr (Q8) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    // ---- softmax: thread `tid` has row `tid`
    const uint32_t lane_at = (uint32_t)(32 * warp) << 16;
    float m = kNegInf;  // reference maximum, base-2 exponent
    uint64_t l2[4];     // sums of the weights, in eight chains
#pragma unroll
    for (int i = 0; i < 4; ++i) l2[i] = f2(0.f, 0.f);
    float c = p.c, from = 0.f;  // a score's factor; what its values' power adds to it
    bool even = true;           // the step has one power for its keys, and one for its values
    [[maybe_unused]] float row_c = 0.f;
    [[maybe_unused]] float l = 0.f;
    if constexpr (Q8) {
      tc_wait(qfull, 0, dead, gave_up);
      row_c = p.c * row_f[tid];
    }
    for (int j = 0; j < ns; ++j) {
      if constexpr (Q8) {
        tc_wait(&efull[j % C::NE], (uint32_t)((j / C::NE) & 1), dead, gave_up);
        const int2 e = largest[j % C::NE];
        // (a vote: the warp stays together where a wait ran out and E is still being written)
        even = __all_sync(kFull, e.x != kUneven);
        // Not 0 for tiny queries, by which the -inf of a score behind the last key would be
        // NaN: a score is below 2^31, times its key's power below 2^95, so what this keeps
        // is nothing. Nor infinite for large ones, by which a score of 0 would be.
        c = even ? row_c * power_of(e.x) : row_c;
        c = fminf(fmaxf(c, 1.17549435e-38f), 3.40282347e38f);
        from = even ? (float)e.y : 0.f;
      }
      tc_wait(&sfull[j & 1], (uint32_t)((j >> 1) & 1), dead, gave_up);
      dead = __any_sync(kFull, dead);
      tc_fence_after();
      const uint32_t ts = tb + lane_at + (j & 1) * 128;
      const int n = min(128, keys - (s0 + j) * 128);  // a multiple of 16
      const uint64_t c2 = f2(c, c);
      // of step j: words of two tokens (the softmax's warps read the same at a time)
      [[maybe_unused]] const uint4* powers =
          reinterpret_cast<const uint4*>(sm + C::POWERS + (Q8 ? j % C::NE : 0) * 256);
      // of a step that is not even: quarter q's scores by their keys' powers (-inf behind
      // the last), and the powers. A quarter at a time, and from tensor memory for both of
      // its uses, so that the registers of even steps stay theirs (else those took 2% more).
      auto keyed = [&](int q, float (&y)[32], uint32_t (&w)[16]) {
        tmem_ld32(ts + 32 * q, y);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 v = powers[4 * q + i];
          w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
        }
        tmem_ld_wait32(y);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          un2(mul2(f2(y[2 * i], y[2 * i + 1]), key_powers(w[i])), y[2 * i], y[2 * i + 1]);
          y[2 * i] = 32 * q + 2 * i < n ? y[2 * i] : kNegInf;
          y[2 * i + 1] = 32 * q + 2 * i + 1 < n ? y[2 * i + 1] : kNegInf;
        }
      };
      float x[128], t[4];
      if (!Q8 || even) {
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_ld32_max(ts + 32 * q, x + 32 * q, t[q]);
#pragma unroll
        for (int q = 0; q < 4; ++q) { tmem_ld_wait32(x + 32 * q); asm volatile("" : "+f"(t[q])); }
        if (n < 128) {
#pragma unroll
          for (int i = 0; i < 128; ++i) x[i] = i < n ? x[i] : kNegInf;
#pragma unroll
          for (int k = 0; k < 4; ++k) t[k] = kNegInf;
#pragma unroll
          for (int i = 0; i < 128; i += 8) {
#pragma unroll
            for (int k = 0; k < 4; ++k) t[k] = max3(t[k], x[i + 2 * k], x[i + 2 * k + 1]);
          }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) t[k] = t[k] * c + from;  // c is not negative
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) t[k] = kNegInf;
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
          float y[32];
          uint32_t w[16];
          keyed(q, y, w);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float a, b;
            un2(fma2(f2(y[2 * i], y[2 * i + 1]), c2, value_exponents(w[i])), a, b);
            t[i & 3] = max3(t[i & 3], a, b);
          }
        }
      }
      const float mx = max3(max3(t[0], t[1], t[2]), t[3], kNegInf);  // largest weight's exponent
      // move the reference: always from -inf, else when the row outgrew it
      const bool move = mx - m > kWeightMost<M>;
      if (__any_sync(kFull, move)) {
        const float to = move ? mx - kWeightLeft<M> : m;
        if (j > 0) {
          const float f = to == kNegInf ? 1.f : exp2_fast(m - to);
          if constexpr (Q8) l = to == kNegInf ? l : brought<true>(l, m - to);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float a, b;
            un2(l2[i], a, b);
            l2[i] = f2(a * f, b * f);
          }
          tc_wait(&odone[(j - 1) & 1], (uint32_t)(((j - 1) >> 1) & 1), dead, gave_up);
          dead = __any_sync(kFull, dead);
          tc_fence_after();
#pragma unroll 1
          for (int d = 0; d < D; d += 16) {
            float o[16];
            tmem_ld16(tb + lane_at + C::O0 + d, o);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] *= f;
            tmem_st16(tb + lane_at + C::O0 + d, o);
          }
        }
        m = to;
      }
      const float base = m == kNegInf ? 0.f : m - from;
      const uint64_t b2 = f2(-base, -base);
      if (!Q8 || even) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float a, b;
            un2(fma2(f2(x[32 * q + 2 * i], x[32 * q + 2 * i + 1]), c2, b2), a, b);
            a = exp2_fast(a);
            b = exp2_fast(b);
            l2[i & 3] = add2(l2[i & 3], f2(a, b));
            w[i] = pack2<M>(a, b);
          }
          tmem_st16u(ts + 16 * q, w);
        }
      } else {
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {  // the weights lie over scores that have been read
          float y[32];
          uint32_t w[16];
          keyed(q, y, w);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float a, b;
            un2(fma2(f2(y[2 * i], y[2 * i + 1]), c2, b2), a, b);
            a = exp2_fast(a);
            b = exp2_fast(b);
            l2[i & 3] = add2(l2[i & 3], f2(a, b));
            un2(mul2(f2(a, b), value_powers(w[i])), a, b);
            w[i] = pack2<M>(a, b);
          }
          tmem_st16u(ts + 16 * q, w);
        }
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&pfull[j & 1]);
      if constexpr (Q8) {  // the step's sum, without its values' power
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float a, b;
          un2(l2[i], a, b);
          sum += a + b;
          l2[i] = f2(0.f, 0.f);
        }
        l = fmaf(sum, power_of(-(int)from), l);
      }
    }
    if constexpr (!Q8) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float a, b;
        un2(l2[i], a, b);
        l += a + b;
      }
    }
    tc_wait(&odone[(ns - 1) & 1], (uint32_t)(((ns - 1) >> 1) & 1), dead, gave_up);
    dead = __any_sync(kFull, dead || *gave_up != 0);
    tc_fence_after();
    // ---- output, 32 columns at a time through shared memory (the ring: its
    // products are done) to rows of whole lines
    constexpr int PITCH = 36;
    float* st = reinterpret_cast<float*>(sm + C::RING) + warp * (32 * PITCH);
    const bool cut = s_b.w >= 0;
    float* pout = sv.part + (cut ? s_b.w : 0) * ((long long)sv.part_rows * (D + 2));
    float* o = cut ? pout : sv.o;
    if (!dead && tid < R) {
      float2* ml = cut ? reinterpret_cast<float2*>(pout + sv.part_rows * D) + tid
                       : sv.ml + at;
      *ml = make_float2(m, l);
    }
#pragma unroll 1
    for (int d = 0; d < D; d += 32) {
      float x[32];
      tmem_ld32(tb + lane_at + C::O0 + d, x);
      tmem_ld_wait32(x);
#pragma unroll
      for (int i = 0; i < 32; i += 4)
        *reinterpret_cast<float4*>(st + lane * PITCH + i) =
            make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = 4 * i + lane / 8, rr = 32 * warp + r;
        const int other = __shfl_sync(kFull, at, r);
        const size_t to = cut ? rr : other;
        if (!dead && rr < R)
          *reinterpret_cast<float4*>(o + to * D + d + 4 * (lane % 8)) =
              *reinterpret_cast<const float4*>(st + r * PITCH + 4 * (lane % 8));
      }
      __syncwarp();
    }
  } else if (warp >= 8) {
    // ---- codes to fp16, two threads to a row of a unit. (Half the warps to the keys,
    // half to the values is no faster: 198 for 190 us of 20 groups; shared memory, which
    // feeds the products beside 96 KB a step here, is what they wait for.)
    if constexpr (Q8) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 120;");
      const int r = (tid - 256) % 128, half = (tid - 256) / 128;
      unsigned both = 0, most_k = 0, most_v = 0;  // the row's powers, and the step's largest
      bool even = true;
      for (int i = 0; i < 2 * ns; ++i) {
        const int n = min(128, keys - (s0 + i / 2) * 128);
        const int ur = i % C::NR, u = i % C::NU;
        tc_wait(&rfull[ur], (uint32_t)((i / C::NR) & 1), dead, gave_up);
        if (i >= C::NU) tc_wait(&empty[u], (uint32_t)((i / C::NU - 1) & 1), dead, gave_up);
        dead = __any_sync(kFull, dead);
        if (dead) break;
        const unsigned char* raw = sm + C::RAWS + ur * C::RAW;
        unsigned char* to = sm + C::RING + u * C::UNIT;
        if (i % 2 == 0) {  // a step's keys come first, and its powers, as bytes, with them
          const uint16_t* bytes = reinterpret_cast<const uint16_t*>(sm + C::SCALES + ur * 256);
          unsigned least_k = 255, least_v = 255;
          most_k = most_v = 0;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const bool on = lane + 32 * k < n;
            const unsigned two = bytes[lane + 32 * k];
            const unsigned key = two & 0xff, value = two >> 8;
            most_k = max(most_k, on ? key : 0), least_k = min(least_k, on ? key : 255);
            most_v = max(most_v, on ? value : 0), least_v = min(least_v, on ? value : 255);
          }
          most_k = __reduce_max_sync(kFull, most_k);
          most_v = __reduce_max_sync(kFull, most_v);
          least_k = __reduce_min_sync(kFull, least_k);
          least_v = __reduce_min_sync(kFull, least_v);
          even = most_k - least_k <= kEvenKeys && most_v - least_v <= kEvenValues &&
                 least_v >= kEvenLeast && most_v <= kEvenMost;
          both = r < n ? bytes[r] : 0;
          if (half == 0) {
            reinterpret_cast<uint16_t*>(sm + C::POWERS + i / 2 % C::NE * 256)[r] = (uint16_t)both;
            if (r == 0)
              largest[i / 2 % C::NE] = make_int2(even ? (int)most_k - kScaleBias : kUneven,
                                                 (int)most_v - kScaleBias);
            mbar_arrive(&efull[i / 2 % C::NE]);
          }
        }
        // 2^(e - E) or 2^(f - F) in fp16: normal to 2^-14, then its second largest bit
        const int d2 = (int)(i & 1 ? both >> 8 : both & 0xff) - (int)(i & 1 ? most_v : most_k);
        const uint32_t bits = !even || r >= n ? 0x3c00u
                              : d2 >= -14     ? (uint32_t)(15 + d2) << 10
                                              : 0x200u;
        const uint32_t twice = bits | bits << 16;
        const __half2 by = *reinterpret_cast<const __half2*>(&twice);
        constexpr int WIDE = D == 256 ? 2 : 1, W = D / WIDE;  // a box's width
#pragma unroll 4
        for (int d = D / 2 * half; d < D / 2 * (half + 1); d += 16) {
          // sixteen codes; neighbouring threads' rows by turns in their columns, or
          // all lanes would ask one bank
          const int at = (d + 16 * r) % D;
          const uint4 x = *reinterpret_cast<const uint4*>(raw + at / W * (128 * 128) + r * W +
                                                          at % W);
          const uint32_t w[4] = {x.x, x.y, x.z, x.w};
          uint32_t y[8];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const __half2 lo = __hmul2(e4m3x2_half2(w[k]), by);
            const __half2 hi = __hmul2(e4m3x2_half2(w[k] >> 16), by);
            // behind the last key nothing may be left, a NaN times 0 neither
            y[2 * k] = r < n ? *reinterpret_cast<const uint32_t*>(&lo) : 0u;
            y[2 * k + 1] = r < n ? *reinterpret_cast<const uint32_t*>(&hi) : 0u;
          }
#pragma unroll
          for (int k = 0; k < 2; ++k)
            *reinterpret_cast<uint4*>(to + at / 64 * 16384 + unit_off<128>(r, at % 64 / 8 + k)) =
                make_uint4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
        }
        fence_async_smem();
        mbar_arrive(&rempty[ur]);
        mbar_arrive(&full[u]);
      }
    }
  }
  if (dead && lane == 0) {
    atomicOr(p.err, DEVERR_TIMEOUT);
    atomicExch(sv.lost, 1);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 5) tmem_dealloc512(tb);
}

template <typename T, int D, bool Q8>
cudaError_t shared_tc_one(const DecodeParams* p, const void* maps, int ctas, cudaStream_t st) {
  using C = SharedTcCfg<D, Q8>;
  const auto kernel = attn_shared_tc_kernel<T, D, Q8>;
  if (p == nullptr)
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  kernel<<<ctas, C::NT, C::SMEM, st>>>(*p, *static_cast<const SharedTcMaps*>(maps));
  return cudaGetLastError();
}

template <typename T, bool Q8>
cudaError_t shared_tc_any(const DecodeParams* p, const void* maps, int D, int ctas,
                          cudaStream_t st) {
  if (D == 64) return shared_tc_one<T, 64, Q8>(p, maps, ctas, st);
  if (D == 128) return shared_tc_one<T, 128, Q8>(p, maps, ctas, st);
  if (D == 256) return shared_tc_one<T, 256, Q8>(p, maps, ctas, st);
  return cudaErrorInvalidValue;
}

}  // namespace

}  // namespace rssm
