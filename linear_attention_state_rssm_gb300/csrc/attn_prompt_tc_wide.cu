// Causal attention over packed prompts for 16-bit types on the 5th-generation
// tensor cores: heads of 256 (attn_prompt_tc.cu: 64 and 128, and the method).
//
// Tensor memory holds one output of 128 rows x 256 and two buffers of scores, so
// there is one stream, whose consecutive steps take turns: while a step's
// weights are computed the next one's scores are. Units of the ring are 128
// keys x 128 dimensions, two to a step's keys and two to its values.
//
// Nothing fills the tensor cores while a tile of one stream begins and ends
// (13 k cycles, as much as 5 steps), so a CTA stays on its SM and takes over
// the tiles of CTAs that have not begun (cluster launch control): the next
// tile's queries and keys are loaded, and its first scores computed, while the
// last one's output is written. Eight prompts of 64 to 4096 tokens, 16/4 heads:
// 305 us with a CTA per tile, 275 us so, back to back (1.39 PFLOP/s of causal
// products, 72% of the library's matrix product); 257 us by itself.
//
// What bounds it: shared memory. A step's products take 2048 cycles; feeding
// them reads 192 KB and writes 128 KB there, 2500 cycles at 128 bytes (tensor
// cores 66% busy). Two CTAs sharing their keys (cta_group::2) would halve that.
#include "attn_prompt_tc.cuh"

namespace rssm {

namespace {

struct TcWide {
  static constexpr int DU = 128;                     // head dimensions of a unit
  static constexpr int UPT = 2;                      // units of a step's keys (or values)
  static constexpr int UNIT = 128 * DU * 2;
  static constexpr int NU = 5;                       // units in the ring
  static constexpr int NT = 128 + 128;               // softmax warps, then four with roles
  static constexpr int RING = 128 * 256 * 2;         // its offset, behind the queries
  static constexpr int BARS = RING + NU * UNIT;
  static constexpr int SMEM = BARS + 512 + 1024;     // + alignment of the base
  static constexpr uint32_t O0 = 256;                // first column of O
  static_assert(SMEM <= 227 * 1024, "shared memory");
};

// A tile as the roles see it.
struct TcTile {
  PromptTile t;
  int h, live;  // key head; 0: no tile any more
};

// Asks for a CTA of this launch that has not begun, to do its work here; the
// answer (16 bytes) lands in shared memory and completes `bar`.
__device__ __forceinline__ void ask_for_cta(void* answer, uint64_t* bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], "
      "[%1];" ::"r"(smem_addr(answer)),
      "r"(smem_addr(bar))
      : "memory");
}
// Its index, or -1: every CTA has begun.
__device__ __forceinline__ int cta_answered(const void* answer) {
  int x, ok;
  asm volatile(
      "{\n.reg .b128 a;\n.reg .pred p;\n.reg .b32 y, z, w;\n"
      "ld.shared.b128 a, [%2];\n"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n"
      "selp.b32 %1, 1, 0, p;\n"
      "mov.b32 %0, 0;\n"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%0, y, z, w}, a;\n}\n"
      : "=r"(x), "=r"(ok)
      : "r"(smem_addr(answer))
      : "memory");
  return ok ? x : -1;
}

// Steps of 128 keys that a tile takes.
__device__ __forceinline__ int steps_of(const PromptTile& tl, int toks) {
  return (max(0, tl.lk - tl.lq + min((tl.tile + 1) * toks, tl.lq)) + 127) / 128;
}

template <typename T>
__global__ void __launch_bounds__(TcWide::NT, 1)
    attn_prompt_tc_wide_kernel(const __grid_constant__ PromptParams p,
                          const __grid_constant__ TcMaps maps) {
  constexpr int D = 256;
  using C = TcWide;
  extern __shared__ unsigned char sm_raw[];
  unsigned char* sm = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(sm_raw) + 1023) & ~(uintptr_t)1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + C::BARS);  // [NU] a unit has landed
  uint64_t* empty = full + C::NU;                              // [NU] its products are done
  uint64_t* qfull = empty + C::NU;                             // queries have landed
  uint64_t* qempty = qfull + 1;                                // their products are done
  uint64_t* sfull = qempty + 1;                                // [2] scores are in tensor memory
  uint64_t* pfull = sfull + 2;                                 // [2][2] half the weights are
  uint64_t* odone = pfull + 4;                                 // a step's P V is done
  uint64_t* tfull = odone + 1;                                 // [2] a tile is known
  uint64_t* tempty = tfull + 2;                                // [2] every role has it
  uint64_t* sent = tempty + 2;                                 // a tile's loads are all on their way
  uint64_t* answered = sent + 1;                               // a CTA was asked for
  uint64_t* drained = answered + 1;                            // no product is in flight
  uint4* answer = reinterpret_cast<uint4*>(sm + C::BARS + 272);
  TcTile* tiles = reinterpret_cast<TcTile*>(sm + C::BARS + 288);  // [2]
  uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + C::BARS + 288 + 2 * sizeof(TcTile));
  volatile uint32_t* gave_up = tslot + 1;  // as in attn_prompt_tc.cu
  static_assert((2 * C::NU + 18) * 8 <= 272 && 288 + 2 * sizeof(TcTile) + 8 <= 512, "barriers");
  const int tid = threadIdx.x, warp = __shfl_sync(kFull, tid >> 5, 0), lane = tid & 31;
  const int toks = 128 / p.G;  // tokens of a stream
  constexpr int W0 = 4;  // first of the warps with roles

  if (tid < 3)
    asm volatile("prefetch.tensormap [%0];" ::"l"(tid == 0 ? &maps.q : tid == 1 ? &maps.k : &maps.v)
                 : "memory");
  if (warp == W0 && lane == 0) {
    for (int u = 0; u < C::NU; ++u) mbar_init(&full[u], 1), mbar_init(&empty[u], 1);
    mbar_init(qfull, 1);
    mbar_init(qempty, 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sfull[b], 1);
      mbar_init(&pfull[2 * b], 128);
      mbar_init(&pfull[2 * b + 1], 128);
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 2 + 4);
    }
    mbar_init(odone, 1);
    mbar_init(sent, 1);
    mbar_init(answered, 1);
    mbar_init(drained, 1);
    *gave_up = 0;
    if (p.hook_cta == (int)blockIdx.x) promise_more<C::NU>(full, qfull, p.hook_unit);
    fence_mbar_init();
  }
  if (warp == W0 + 1) tmem_alloc512(tslot);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tb = *tslot;
  bool dead = false;
  // the k-th tile, once it is known; the role's warp then says that it has it
  auto tile = [&](int k) {
    tc_wait(&tfull[k & 1], (uint32_t)((k >> 1) & 1), dead);
    dead = __any_sync(kFull, dead);
    // the same in every lane, and known to be: the products' operands follow
    // from it, and only where all lanes agree do they need no gathering
    const TcTile& r = tiles[k & 1];
    TcTile t;
    t.t.tile = __shfl_sync(kFull, r.t.tile, 0);
    t.t.q0 = __shfl_sync(kFull, r.t.q0, 0);
    t.t.k0 = __shfl_sync(kFull, r.t.k0, 0);
    t.t.lq = __shfl_sync(kFull, r.t.lq, 0);
    t.t.lk = __shfl_sync(kFull, r.t.lk, 0);
    t.h = __shfl_sync(kFull, r.h, 0);
    t.live = dead ? 0 : __shfl_sync(kFull, r.live, 0);
    return t;
  };

  if (warp >= W0) {
  if (warp == W0) {
    // ---- producer: per tile the queries, K(0), then for each step the values
    // and the next keys in the order the products take them
    int n = 0, nq = 0;  // units and queries sent for
    for (int k = 0;; ++k) {
      const TcTile tt = tile(k);
      if (!tt.live) break;
      const PromptTile& tl = tt.t;
      const int ntm = steps_of(tl, toks);
      if (lane == 0) {
        auto unit = [&](const CUtensorMap* map, int step, int part) {
          const int u = n % C::NU;
          if (n >= C::NU) tc_wait(&empty[u], (uint32_t)((n / C::NU - 1) & 1), dead);
          if (dead) return;
          ++n;
          mbar_expect_tx(&full[u], C::UNIT);
          for (int d = 0; d < C::DU / 64; ++d)
            tma_load3(smem_addr(sm + C::RING + u * C::UNIT + d * 16384), map,
                      part * C::DU + 64 * d, tt.h, tl.k0 + step * 128, &full[u]);
        };
        auto units = [&](const CUtensorMap* map, int step) {
          for (int i = 0; i < C::UPT; ++i) unit(map, step, i);
        };
        if (ntm > 0) {
          units(&maps.k, 0);
          if (nq > 0) tc_wait(qempty, (uint32_t)((nq - 1) & 1), dead);
          if (!dead) {
            ++nq;
            mbar_expect_tx(qfull, (uint32_t)((D / 64) * p.G * toks * 128));
            for (int d = 0; d < D / 64; ++d)
              tma_load4(smem_addr(sm + d * 16384), &maps.q, 64 * d, 0, tt.h, tl.q0 + tl.tile * toks,
                        qfull);
          }
        }
        for (int j = 0; j < ntm; ++j) {
          if (j + 1 < ntm) units(&maps.k, j + 1);
          units(&maps.v, j);
        }
        mbar_arrive(sent);
        mbar_arrive(&tempty[k & 1]);
      }
      dead = __any_sync(kFull, dead);
    }
    // every copy has landed before the CTA leaves
    if (lane == 0) {
      bool late = false;
      for (int u = max(0, n - C::NU); u < n; ++u)
        tc_wait(&full[u % C::NU], (uint32_t)((u / C::NU) & 1), late);
      if (nq > 0) tc_wait(qfull, (uint32_t)((nq - 1) & 1), late);
      dead |= late;
    }
    __syncwarp();
  } else if (warp == W0 + 1) {
    // ---- products; the warp stays together and one lane issues
    constexpr uint32_t id_qk = f16_idesc<T>(128, 128, false);
    constexpr uint32_t id_pv = f16_idesc<T>(128, C::DU, true);
    const uint32_t el = elect_lane();
    const uint32_t qd = sw128_kmajor_lo(smem_addr(sm));
    const uint32_t kd = sw128_kmajor_lo(smem_addr(sm + C::RING));
    const uint32_t vd = sw128_mnmajor_lo(smem_addr(sm + C::RING), 16384);
    int n0 = 0, nq = 0;         // units and queries taken by the tiles before
    uint32_t np = 0;            // bits 0 and 1: parity of the weights to take, per S buffer
    uint32_t steps = 0;         // steps of the tiles before
    auto ready = [&](int n) { tc_wait(&full[n % C::NU], (uint32_t)((n / C::NU) & 1), dead); };
    // S[buf] = Q K^T, keys in units n ..
    auto qk = [&](int buf, int n) {
      for (int i = 0; i < C::UPT; ++i) {
        ready(n + i);
        dead = __any_sync(kFull, dead);
        if (dead) return;
        tc_fence_after();
        const uint32_t a = qd + i * (32768 / 16);
        const uint32_t b = kd + ((n + i) % C::NU) * (C::UNIT / 16);
#pragma unroll
        for (int k = 0; k < C::DU / 16; ++k) {
          const uint32_t in = ((k / 4) * 16384 + (k % 4) * 32) / 16;
          mma16_ss(el, tb + buf * 128, a + in, b + in, id_qk, i > 0 || k > 0);
        }
      }
      mma16_commit(el, &sfull[buf]);
    };
    // O += P V, weights in buffer buf, values in units n ..; the first 64
    // keys' products begin when their weights are there
    auto pv = [&](int buf, int n, bool acc) {
      for (int i = 0; i < C::UPT; ++i) ready(n + i);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        tc_wait(&pfull[2 * buf + half], (np >> buf) & 1, dead);
        dead = __any_sync(kFull, dead);
        if (dead) return;
        tc_fence_after();
        for (int i = 0; i < C::UPT; ++i) {
          const uint32_t b = vd + ((n + i) % C::NU) * (C::UNIT / 16);
#pragma unroll
          for (int k = 4 * half; k < 4 * half + 4; ++k)
            mma16_ts(el, tb + C::O0 + i * 128, tb + buf * 128 + 8 * k, b + k * 128, id_pv,
                     acc || k > 0);
        }
      }
      np ^= 1u << buf;
      mma16_commit(el, odone);
    };
    auto free_units = [&](int n) {
      for (int i = 0; i < C::UPT; ++i)
        if (!dead) mma16_commit(el, &empty[(n + i) % C::NU]);
    };
    // zeros in the values of units n .. from key v of the step on
    auto zero_values = [&](int n, int v) {
      for (int i = 0; i < C::UPT; ++i) {
        ready(n + i);
        zero_rows<C::DU>(sm + C::RING + ((n + i) % C::NU) * C::UNIT, v, lane);
      }
    };
    for (int k = 0;; ++k) {
      const TcTile tt = tile(k);
      __syncwarp();
      if (lane == 0 && !dead) mbar_arrive(&tempty[k & 1]);
      if (!tt.live) break;
      const int ntm = steps_of(tt.t, toks);
      if (ntm == 0) continue;
      const int valid = tt.t.lk - 128 * (ntm - 1);  // keys of the last step
      tc_wait(qfull, (uint32_t)(nq & 1), dead);
      ++nq;
      // units: K0 K1 V0 K2 V1 ...
      qk(steps & 1, n0);
      free_units(n0);
      if (ntm == 1 && !dead) mma16_commit(el, qempty);
      for (int j = 0; j < ntm; ++j) {
        const bool more = j + 1 < ntm;
        const int nk = n0 + C::UPT * (2 * j + 1);
        const int nv = more ? nk + C::UPT : nk;
        if (more) {
          qk((steps + j + 1) & 1, nk);
          free_units(nk);
          if (j + 2 == ntm && !dead) mma16_commit(el, qempty);
        }
        if (!more && valid < 128) zero_values(nv, valid);
        pv((steps + j) & 1, nv, j > 0);
        free_units(nv);
      }
      n0 += 2 * C::UPT * ntm;
      steps += (uint32_t)ntm;
    }
    if (dead) {  // products in flight end before their memory is given back
      bool late = false;
      mma16_commit(el, drained);
      tc_wait(drained, 0, late);
    }
    __syncwarp();
  } else if (warp == W0 + 2) {
    // ---- tiles: this CTA's, then those of CTAs that have not begun
    int index = (int)blockIdx.x;
    for (int k = 0;; ++k) {
      TcTile tt;
      tt.h = index % p.HKV;  // heads of a tile side by side
      tt.live = index >= 0 && find_tile(p, toks * p.G, index / p.HKV, tt.h == 0, tt.t);
      if (k >= 2) tc_wait(&tempty[k & 1], (uint32_t)((k / 2 - 1) & 1), dead);
      dead = __any_sync(kFull, dead);
      if (dead) break;
      if (lane == 0) {
        tiles[k & 1] = tt;
        mbar_arrive(&tfull[k & 1]);
      }
      if (!tt.live) break;
      // the next is asked for when this one's last loads have been sent: early
      // enough to hide, late enough that CTAs end together
      tc_wait(sent, (uint32_t)(k & 1), dead);
      if (lane == 0 && !dead) {
        mbar_expect_tx(answered, 16);
        ask_for_cta(answer, answered);
      }
      tc_wait(answered, (uint32_t)(k & 1), dead);
      dead = __any_sync(kFull, dead);
      index = dead ? -1 : cta_answered(answer);
      fence_async_smem();  // the answer is read before the next one is written
      __syncwarp();
    }
  }
  } else {
    // ---- softmax: a thread per row
    const int row = tid;
    const uint32_t lane_at = (uint32_t)(32 * (warp & 3)) << 16;
    const float c = p.c;
    uint32_t done = 0;  // steps of the tiles before
    for (int k = 0;; ++k) {
      const TcTile tt = tile(k);
      __syncwarp();
      if (lane == 0 && !dead) mbar_arrive(&tempty[k & 1]);
      if (!tt.live) break;
      const PromptTile& tl = tt.t;
      const int tok0 = tl.tile * toks;                           // within the sequence
      const int n_steps = steps_of(tl, toks);
      const int R = max(0, min(toks, tl.lq - tok0)) * p.G;       // rows in use
      const int rr = min(row, max(R - 1, 0));
      const int lim = max(0, tl.lk - tl.lq + tok0 + rr / p.G + 1);  // keys the row sees
      const int fewest = __reduce_min_sync(kFull, lim);
      float m = kNegInf;  // reference maximum (raw score)
      uint64_t l2[4];     // sums of the weights, in eight chains
#pragma unroll
      for (int i = 0; i < 4; ++i) l2[i] = f2(0.f, 0.f);
      for (int j = 0; j < n_steps; ++j) {
        const uint32_t at = done + (uint32_t)j;
        const int buf = at & 1;
        tc_wait(&sfull[buf], (at >> 1) & 1, dead, gave_up);
        dead = __any_sync(kFull, dead);
        tc_fence_after();
        const uint32_t ts = tb + lane_at + buf * 128;
        float x[128], t[4];  // scores; the largest of each quarter
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_ld32_max(ts + 32 * i, x + 32 * i, t[i]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          tmem_ld_wait32(x + 32 * i);
          asm volatile("" : "+f"(t[i]));  // not read before the wait
        }
        const int key0 = j * 128;
        if (key0 + 128 > fewest) {
          const int n = lim - key0;
#pragma unroll
          for (int i = 0; i < 128; ++i) x[i] = i < n ? x[i] : kNegInf;
#pragma unroll
          for (int e = 0; e < 4; ++e) t[e] = kNegInf;
#pragma unroll
          for (int i = 0; i < 128; i += 8) {
#pragma unroll
            for (int e = 0; e < 4; ++e) t[e] = max3(t[e], x[i + 2 * e], x[i + 2 * e + 1]);
          }
        }
        const float mx = max3(max3(t[0], t[1], t[2]), t[3], m);
        const bool move = (mx - m) * c > kWeightMost<T> - kWeightLeft<T>;
        if (j == 0 || __any_sync(kFull, move)) {
          const float to = move ? mx : m;
          if (j > 0) {
            const float f = to == kNegInf ? 1.f : exp2_fast((m - to) * c);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float a, b;
              un2(l2[i], a, b);
              l2[i] = f2(a * f, b * f);
            }
            tc_wait(odone, (at - 1) & 1, dead, gave_up);
            dead = __any_sync(kFull, dead);
            tc_fence_after();
            const uint32_t to_o = tb + lane_at + C::O0;
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
        const float base = m == kNegInf ? 0.f : kWeightLeft<T> - m * c;
        const uint64_t c2 = f2(c, c), b2 = f2(base, base);
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
            // A parity tells a phase only from its neighbours, so every phase
            // of odone is seen before the next can end: the scores of step j
            // do not wait for P V of step j - 1.
            if (q == 1 && j > 0) tc_wait(odone, (at - 1) & 1, dead, gave_up);
            tc_fence_before();
            mbar_arrive(&pfull[2 * buf + (q >> 1)]);
          }
        }
      }
      done += (uint32_t)n_steps;

      // ---- output, two whole sectors of a row to four lanes
      float l = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float a, b;
        un2(l2[i], a, b);
        l += a + b;
      }
      const bool none = lim == 0;
      const float inv = none ? 0.f : 1.f / l;
      const size_t orow = (size_t)(tl.q0 + tok0 + rr / p.G) * p.HQ + tt.h * p.G + rr % p.G;
      bool bad = false;
      if (n_steps > 0) {
        tc_wait(odone, (done - 1) & 1, dead, gave_up);
        dead = __any_sync(kFull, dead || *gave_up != 0);
        tc_fence_after();
      }
      T* to[4];  // the lane's sixteen bytes in the rows of its four lanes
      bool put[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        to[r] = static_cast<T*>(p.o) + __shfl_sync(kFull, orow, (lane & ~3) + r) * D + 8 * (lane & 3);
        put[r] = !dead && 32 * (warp & 3) + (lane & ~3) + r < R;
      }
#pragma unroll 2
      for (int d = 0; d < D; d += 32) {
        float o[32];
        if (n_steps > 0) {
          tmem_ld32(tb + lane_at + C::O0 + d, o);
          tmem_ld_wait32(o);
        }
        float t[4] = {0.f, 0.f, 0.f, 0.f};
        uint32_t w[4][4];  // sixteen bytes of the lane's row, times four
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          o[i] = none ? 0.f : o[i] * inv;
          t[i & 3] = fmaf(o[i], 0.f, t[i & 3]);  // NaN where any is non-finite
        }
        bad |= t[0] + t[1] + (t[2] + t[3]) != 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i / 4][i % 4] = pack2<T>(o[2 * i], o[2 * i + 1]);
        // four lanes transpose: lane i ends with the i-th sixteen bytes of each row
#pragma unroll
        for (int x = 1; x < 4; x <<= 1) {
          const bool up = (lane & x) != 0;
#pragma unroll
          for (int a = 0; a < 4; ++a) {
            if (a & x) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t got = __shfl_xor_sync(kFull, up ? w[a][e] : w[a | x][e], x);
              if (up) w[a][e] = got; else w[a | x][e] = got;
            }
          }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if (put[r])
            *reinterpret_cast<uint4*>(to[r] + d) = make_uint4(w[r][0], w[r][1], w[r][2], w[r][3]);
        }
      }
      const bool mine = row < R && !dead;
      if (mine && p.lse != nullptr) p.lse[orow] = none ? kNegInf : lse_of(m * c - kWeightLeft<T>, l);
      if (__any_sync(kFull, bad && mine)) {
        __syncwarp();  // these rows' outputs come before what is put in their place
        again<T, D>(p, tl, tt.h, tok0, 32 * (warp & 3), R, min(128 * n_steps, tl.lk), lane);
      }
      tc_fence_before();
    }
  }
  if (dead && lane == 0) atomicOr(p.err, DEVERR_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  if (warp == W0 + 1) tmem_dealloc512(tb);
}

template <typename F>
cudaError_t pick(int dt, F f) {
  return dt == DT_BF16 ? f(attn_prompt_tc_wide_kernel<__nv_bfloat16>)
                       : f(attn_prompt_tc_wide_kernel<__half>);
}

}  // namespace

cudaError_t attn_prompt_tc_wide_prepare(int dt) {
  return pick(dt, [](auto kernel) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, TcWide::SMEM);
  });
}

cudaError_t attn_prompt_tc_wide_launch(const PromptParams& p, cudaStream_t st) {
  TcMaps maps;
  if (!encode_maps(p, &maps)) return cudaErrorInvalidValue;
  // every sequence has at most one tile that is not full of tokens
  const long long ctas = ((long long)p.N / (128 / p.G) + p.B) * p.HKV;
  if (ctas > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  return pick(p.dt, [&](auto kernel) {
    kernel<<<(unsigned)ctas, TcWide::NT, TcWide::SMEM, st>>>(p, maps);
    return cudaGetLastError();
  });
}

}  // namespace rssm
