// Causal attention over packed prompts for 16-bit types on the 5th-generation
// tensor cores: heads of 64 and 128 (attn_prompt_tc_wide.cu: 256).
//
// A CTA's tile is two streams of 128 query rows of one key head: floor(128 / G)
// tokens with their G query heads each, gathered by one TMA box, so short
// prompts fill rows and the group shares its keys. It walks the sequence's keys
// in steps of 128:
//
//     S = Q K^T             tensor memory, 128 x 128 fp32
//     P = 2^(c S - c m)     registers, stored over S as 16-bit operand
//     O = O + P V           tensor memory, 128 x D fp32
//
// One lane of a producer warp issues the TMA loads into a ring of units (a
// step's keys, or its values); one lane of another issues the products; a
// warpgroup per stream does the softmax, one thread per row, so that row sums
// need no exchange, and tensor memory finds the maxima on the way out. The two
// streams take turns on the tensor cores: while one's weights are computed the
// other's products run. Weights are handed over in halves of a step. A
// sequence's tiles of longer sight come first in the grid, sequences as given.
//
// The softmax does not depend on what its weights are relative to, as long as
// they stay in range. So that reference is only moved when a row's true maximum
// would get a weight above 2^8 (well within both types); moving it costs a pass
// over O in tensor memory and is rare after the first steps.
//
// Products with masked keys are 0 * v, which is not 0 where v is infinite or
// NaN. Values behind the sequence's last key are zeroed in shared memory; a row
// whose output comes out non-finite is looked at again, and computed again by
// selection where a value it must not see is to blame (attn_prompt_tc.cuh).
//
// What bounds it: for heads of 128 the tensor cores, which the two streams keep
// 80% busy. 14336 tokens, 16/4 heads of 128: 454 to 463 us by itself, 1.82 to
// 1.85 PFLOP/s of causal products (95 to 97% of the library's matrix product,
// burst); 495 to 512 us back to back, 1.64 to 1.70 (96 to 99% of its sustained
// rate). Heads of 64: 387 us; tensor cores and exponentials are each 46% busy, so
// neither binds: a stream's round of scores, maximum, weights and products does.
// What it took, back to back: issue by a converged warp 655 -> 531 us, coalesced output and earlier first
// loads 523, maxima by tensor memory 502. Staying on the SM for further tiles, as
// the wide form does, lost 2% here (and 13% of short ragged prompts, gaining 4% of
// long ones): what the longer-lived state costs every step is more than a tile's
// ends, one stream's beside the other's work. Taking weights before the maximum is
// known, and again where it moved, lost 2%.
#include "attn_prompt_tc.cuh"

namespace rssm {

namespace {

template <int D>
struct TcCfg {
  static constexpr int NS = 2;                       // streams
  static constexpr int UNIT = 128 * D * 2;           // a step's keys, or its values
  static constexpr int NU = D == 64 ? 8 : 5;         // units in the ring
  static constexpr int QS = 128 * D * 2;             // one stream's queries
  static constexpr int NT = NS * 128 + 128;          // softmax warpgroups, and the roles': two warps work
  static constexpr int RING = NS * QS;               // its offset
  static constexpr int BARS = RING + NU * UNIT;
  static constexpr int SMEM = BARS + 512 + 1024;     // + alignment of the base
  static constexpr uint32_t O0 = 256;                // first column of O
  static_assert(SMEM <= 227 * 1024, "shared memory");
};

template <typename T, int D>
__global__ void __launch_bounds__(TcCfg<D>::NT, 1)
    attn_prompt_tc_kernel(const __grid_constant__ PromptParams p,
                          const __grid_constant__ TcMaps maps) {
  static_assert(D <= 128, "two outputs in tensor memory");
  using C = TcCfg<D>;
  extern __shared__ unsigned char sm_raw[];
  unsigned char* sm = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(sm_raw) + 1023) & ~(uintptr_t)1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + C::BARS);  // [NU] a unit has landed
  uint64_t* empty = full + C::NU;                              // [NU] its products are done
  uint64_t* qfull = empty + C::NU;                             // queries have landed
  uint64_t* sfull = qfull + 1;                                 // [2] scores are in tensor memory
  uint64_t* pfull = sfull + 2;                                 // [2][2] half the weights are
  uint64_t* odone = pfull + 4;                                 // [2] a step's P V is done
  uint64_t* tail = odone + 2;                                  // the last values have landed
  uint64_t* drained = tail + 1;                                // no product is in flight
  uint32_t* tslot = reinterpret_cast<uint32_t*>(drained + 1);
  // A softmax warp whose wait ran out goes on without waiting, ahead of the
  // others' phases, so no warp stores what it finds after that.
  volatile uint32_t* gave_up = tslot + 1;
  PromptTile tl;
  const int tid = threadIdx.x, warp = __shfl_sync(kFull, tid >> 5, 0), lane = tid & 31;
  if (tid < 3)
    asm volatile("prefetch.tensormap [%0];" ::"l"(tid == 0 ? &maps.q : tid == 1 ? &maps.k : &maps.v)
                 : "memory");
  const int toks = 128 / p.G;                       // tokens of a stream
  const int h = (int)(blockIdx.x % (unsigned)p.HKV);  // heads of a tile side by side
  if (!find_tile(p, C::NS * toks * p.G, (int)(blockIdx.x / (unsigned)p.HKV), h == 0 && tid < 32, tl))
    return;
  const int i0 = tl.tile * C::NS * toks;
  const int past = tl.lk - tl.lq;
  // steps of 128 keys that each stream takes
  int nt[2] = {0, 0};
#pragma unroll
  for (int s = 0; s < C::NS; ++s) {
    const int a = i0 + s * toks;
    if (a < tl.lq) nt[s] = (max(0, past + min(a + toks, tl.lq)) + 127) / 128;
  }
  const int ntm = max(nt[0], nt[1]);
  const int valid = tl.lk - 128 * (ntm - 1);  // keys of the last step

  // The producer's warp sets the barriers up and sends for the first units
  // while the products' warp waits for tensor memory.
  bool dead = false;
  int issued = 0;  // units sent for
  auto unit = [&](const CUtensorMap* map, int step, uint64_t* other = nullptr) {
    const int u = issued % C::NU;
    uint64_t* bar = other != nullptr ? other : &full[u];  // completed by the loads
    if (issued >= C::NU)
      tc_wait(&empty[u], (uint32_t)((issued / C::NU - 1) & 1), dead);
    if (dead) return;
    ++issued;
    mbar_expect_tx(bar, C::UNIT);
    for (int d = 0; d < D / 64; ++d)
      tma_load3(smem_addr(sm + C::RING + u * C::UNIT + d * 16384), map, 64 * d, h,
                tl.k0 + step * 128, bar);
  };
  if (warp == 4 * C::NS && lane == 0) {
    for (int u = 0; u < C::NU; ++u) mbar_init(&full[u], 1), mbar_init(&empty[u], 1);
    mbar_init(qfull, 1);
    mbar_init(tail, 1);
    mbar_init(drained, 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sfull[b], 1);
      mbar_init(&pfull[2 * b], 128);
      mbar_init(&pfull[2 * b + 1], 128);
      mbar_init(&odone[b], 1);
    }
    *gave_up = 0;
    if (p.hook_cta == (int)blockIdx.x) promise_more<C::NU>(full, qfull, p.hook_unit);
    fence_mbar_init();
    if (ntm > 0) {
      // A stream without a step gets no queries: nothing tells it when they have
      // landed, and its block stages its output from the start.
      const int with = (nt[0] > 0) + (nt[1] > 0);
      mbar_expect_tx(qfull, (uint32_t)(with * (D / 64) * p.G * toks * 128));
#pragma unroll
      for (int s = 0; s < C::NS; ++s) {
        for (int d = 0; d < D / 64 && nt[s] > 0; ++d)
          tma_load4(smem_addr(sm + s * C::QS + d * 16384), &maps.q, 64 * d, 0, h,
                    tl.q0 + i0 + s * toks, qfull);
      }
      unit(&maps.k, 0);
    }
  }
  if (warp == 4 * C::NS + 1) tmem_alloc512(tslot);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tb = *tslot;

  if (warp >= 4 * C::NS) {
  // three warpgroups at 168 registers: two take 232, that of the roles keeps 40
  asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
  if (warp == 4 * C::NS) {
    // ---- producer: after K(0), for each step the values and the next keys in the
    // order the products take them
    if (lane == 0 && ntm > 0) {
      for (int j = 0; j < ntm; ++j) {
        unit(&maps.v, j, j + 1 == ntm && valid < 128 ? tail : nullptr);
        if (j + 1 < ntm) unit(&maps.k, j + 1);
      }
    }
    // The last unit sent for is the last step's values. Those behind the last key
    // (another sequence's) become zeros before it counts as landed.
    issued = __shfl_sync(kFull, issued, 0);
    dead = __any_sync(kFull, dead);
    if (ntm > 0 && valid < 128 && !dead) {
      const int u = (issued - 1) % C::NU;
      tc_wait(tail, 0, dead);
      dead = __any_sync(kFull, dead);
      if (!dead) {
        zero_rows<D>(sm + C::RING + u * C::UNIT, valid, lane);
        if (lane == 0) mbar_arrive(&full[u]);
      }
    }
    // Every copy has landed before the CTA leaves. Once a wait ran out the copies
    // on their way get one more limit between them.
    if (lane == 0) {
      bool late = false;
      if (ntm > 0) tc_wait(qfull, 0, late);
      for (int k = max(0, issued - C::NU); k < issued; ++k)
        tc_wait(&full[k % C::NU], (uint32_t)((k / C::NU) & 1), late);
      dead |= late;
    }
    __syncwarp();
  } else if (warp == 4 * C::NS + 1) {
    // ---- products; the warp stays together and one lane issues
    if (ntm > 0) {
      constexpr uint32_t id_qk = f16_idesc<T>(128, 128, false);
      constexpr uint32_t id_pv = f16_idesc<T>(128, D, true);
      const uint32_t el = elect_lane();
      const uint32_t qd = sw128_kmajor_lo(smem_addr(sm));
      const uint32_t kd = sw128_kmajor_lo(smem_addr(sm + C::RING));
      const uint32_t vd = sw128_mnmajor_lo(smem_addr(sm + C::RING), 16384);
      auto ready = [&](int n) { tc_wait(&full[n % C::NU], (uint32_t)((n / C::NU) & 1), dead); };
      // S_s = Q_s K^T, keys in unit n
      auto qk = [&](int s, int n) {
        ready(n);
        dead = __any_sync(kFull, dead);
        if (dead) return;
        tc_fence_after();
        const uint32_t a = qd + (s * C::QS) / 16;
        const uint32_t b = kd + (n % C::NU) * (C::UNIT / 16);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t in = ((k / 4) * 16384 + (k % 4) * 32) / 16;
          mma16_ss(el, tb + s * 128, a + in, b + in, id_qk, k > 0);
        }
        mma16_commit(el, &sfull[s]);
      };
      // O_s += P_s V of step j, values in unit n; the first 64 keys' products
      // begin when their weights are there
      auto pv = [&](int s, int j, int n) {
        ready(n);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          tc_wait(&pfull[2 * s + half], (uint32_t)(j & 1), dead);
          dead = __any_sync(kFull, dead);
          if (dead) return;
          tc_fence_after();
          const uint32_t b = vd + (n % C::NU) * (C::UNIT / 16);
#pragma unroll
          for (int k = 4 * half; k < 4 * half + 4; ++k)
            mma16_ts(el, tb + C::O0 + s * D, tb + s * 128 + 8 * k, b + k * 128, id_pv,
                     j > 0 || k > 0);
        }
        mma16_commit(el, &odone[s]);
      };
      auto free_unit = [&](int n) {
        if (!dead) mma16_commit(el, &empty[n % C::NU]);
      };
      tc_wait(qfull, 0, dead);
      // units: K0 V0 K1 V1 ...
      for (int s = 0; s < 2; ++s)
        if (nt[s] > 0) qk(s, 0);
      free_unit(0);
      for (int j = 0; j < ntm; ++j) {
        const int nv = 2 * j + 1, nk = nv + 1;
        for (int s = 0; s < 2; ++s) {
          if (j < nt[s]) pv(s, j, nv);
          if (j + 1 < nt[s]) qk(s, nk);
        }
        free_unit(nv);
        if (j + 1 < ntm) free_unit(nk);
      }
      if (__any_sync(kFull, dead)) {  // products in flight end before their memory is given back
        bool late = false;
        mma16_commit(el, drained);
        tc_wait(drained, 0, late);
      }
    }
    __syncwarp();
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
    // ---- softmax: thread `row` of stream s
    const int s = warp >> 2, row = tid & 127;
    const uint32_t lane_at = (uint32_t)(32 * (warp & 3)) << 16;
    const int tok0 = i0 + s * toks;                            // within the sequence
    const int R = max(0, min(toks, tl.lq - tok0)) * p.G;       // rows in use
    const int rr = min(row, max(R - 1, 0));
    const int lim = max(0, past + tok0 + rr / p.G + 1);        // keys the row sees
    const int fewest = __reduce_min_sync(kFull, lim);
    float m = kNegInf;                                         // reference maximum (raw score)
    uint64_t l2[4];  // sums of the weights, in eight chains
#pragma unroll
    for (int i = 0; i < 4; ++i) l2[i] = f2(0.f, 0.f);
    const float c = p.c;
    const int n_steps = nt[s];
    for (int j = 0; j < n_steps; ++j) {
      tc_wait(&sfull[s], (uint32_t)(j & 1), dead, gave_up);
      dead = __any_sync(kFull, dead);
      tc_fence_after();
      const uint32_t ts = tb + lane_at + s * 128;
      float x[128], t[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) tmem_ld32_max(ts + 32 * i, x + 32 * i, t[i]);
#pragma unroll
      for (int i = 0; i < 4; ++i) { tmem_ld_wait32(x + 32 * i); asm volatile("" : "+f"(t[i])); }
      const int key0 = j * 128;
      if (key0 + 128 > fewest) {
        const int n = lim - key0;
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
      const float mx = max3(max3(t[0], t[1], t[2]), t[3], m);
      // move the reference: always from -inf, else when the row outgrew it
      const bool move = (mx - m) * c > 8.f;
      if (__any_sync(kFull, move)) {
        const float to = move ? mx : m;
        if (j > 0) {
          const float f = to == kNegInf ? 1.f : exp2_fast((m - to) * c);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float a, b;
            un2(l2[i], a, b);
            l2[i] = f2(a * f, b * f);
          }
          tc_wait(&odone[s], (uint32_t)((j - 1) & 1), dead, gave_up);
          dead = __any_sync(kFull, dead);
          tc_fence_after();
          const uint32_t to_o = tb + lane_at + C::O0 + s * D;
#pragma unroll 1
          for (int d = 0; d < D; d += 16) {
            float o[16];
            tmem_ld16(to_o + d, o);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] *= f;
            tmem_st16(to_o + d, o);
          }
        }
        m = to;
      }
      const float base = m == kNegInf ? 0.f : m * c;
      const uint64_t c2 = f2(c, c), b2 = f2(-base, -base);
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
          w[i] = pack2<T>(a, b);
        }
        tmem_st16u(ts + 16 * q, w);
        if (q & 1) {
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(&pfull[2 * s + (q >> 1)]);
        }
      }
    }

    // ---- output: through the stream's query block (its products are done) to
    // rows of whole lines
    float l = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a, b;
      un2(l2[i], a, b);
      l += a + b;
    }
    const bool none = lim == 0;
    const float inv = none ? 0.f : 1.f / l;
    const size_t orow = (size_t)(tl.q0 + tok0 + rr / p.G) * p.HQ + h * p.G + rr % p.G;
    bool bad = false;
    if (n_steps > 0) {
      tc_wait(&odone[s], (uint32_t)((n_steps - 1) & 1), dead, gave_up);
      dead = __any_sync(kFull, dead || *gave_up != 0);
      tc_fence_after();
    }
    const bool mine = row < R && !dead;
    unsigned char* st = sm + s * C::QS + (warp & 3) * (32 * D * 2);  // the warp's 32 rows
#pragma unroll 2
    for (int d = 0; d < D; d += 32) {
      float o[32];
      if (n_steps > 0) {
        tmem_ld32(tb + lane_at + C::O0 + s * D + d, o);
        tmem_ld_wait32(o);
      }
      float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        o[i] = none ? 0.f : o[i] * inv;
        t[i & 3] = fmaf(o[i], 0.f, t[i & 3]);  // NaN where any is non-finite
      }
      bad |= t[0] + t[1] + (t[2] + t[3]) != 0.f;
#pragma unroll
      for (int i = 0; i < 32; i += 8)
        *reinterpret_cast<uint4*>(st + unit_off<32>(lane, (d + i) / 8)) =
            make_uint4(pack2<T>(o[i], o[i + 1]), pack2<T>(o[i + 2], o[i + 3]),
                       pack2<T>(o[i + 4], o[i + 5]), pack2<T>(o[i + 6], o[i + 7]));
    }
    __syncwarp();
    if (!dead) {
      constexpr int U = D * 2 / 16;  // 16-byte units of a row
#pragma unroll 4
      for (int i = 0; i < U; ++i) {
        const int r = (32 * i + lane) / U, u = lane % U;
        const size_t to = __shfl_sync(kFull, orow, r);  // the row's place, from its thread
        if (32 * (warp & 3) + r < R)
          reinterpret_cast<uint4*>(static_cast<T*>(p.o) + to * D)[u] =
              *reinterpret_cast<const uint4*>(st + unit_off<32>(r, u));
      }
    }
    __syncwarp();  // before any of these rows is written again
    if (mine && p.lse != nullptr) p.lse[orow] = none ? kNegInf : lse_of(m * c, l);
    if (__any_sync(kFull, bad && mine))
      again<T, D>(p, tl, h, tok0, 32 * (warp & 3), R, min(128 * n_steps, tl.lk), lane);
  }
  if (dead && lane == 0) atomicOr(p.err, DEVERR_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  if (warp == 4 * C::NS + 1) tmem_dealloc512(tb);
}

template <typename F>
cudaError_t pick(int D, int dt, F f) {
#define RSSM_CASE(TT, DD) \
  if (D == DD) return f(attn_prompt_tc_kernel<TT, DD>, TcCfg<DD>::NT, TcCfg<DD>::SMEM);
  if (dt == DT_BF16) {
    RSSM_CASE(__nv_bfloat16, 64) RSSM_CASE(__nv_bfloat16, 128)
  } else {
    RSSM_CASE(__half, 64) RSSM_CASE(__half, 128)
  }
#undef RSSM_CASE
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t attn_prompt_tc_prepare(int D, int dt) {
  if (tma_encoder() == nullptr) return cudaErrorNotSupported;
  if (D == 256) return attn_prompt_tc_wide_prepare(dt);
  return pick(D, dt, [](auto kernel, int, int smem) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  });
}

cudaError_t attn_prompt_tc_launch(const PromptParams& p, cudaStream_t st) {
  if (p.D == 256) return attn_prompt_tc_wide_launch(p, st);
  TcMaps maps;
  if (!encode_maps(p, &maps)) return cudaErrorInvalidValue;
  // every sequence has at most one tile that is not full of tokens
  const long long ctas = ((long long)p.N / (2 * (128 / p.G)) + p.B) * p.HKV;
  if (ctas > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  return pick(p.D, p.dt, [&](auto kernel, int nt, int smem) {
    kernel<<<(unsigned)ctas, nt, smem, st>>>(p, maps);
    return cudaGetLastError();
  });
}

}  // namespace rssm
