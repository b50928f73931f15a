// Causal attention over packed prompts for 16-bit types on the 5th-generation
// tensor cores.
//
// A CTA holds 128 query rows (D = 256) or two streams of 128 (D <= 128) of one
// key head: floor(128 / G) tokens with their G query heads each, gathered by
// one TMA box, so short prompts fill rows and the group shares its keys. It
// walks the sequence's keys in tiles of 128:
//
//     S = Q K^T             tensor memory, 128 x 128 fp32
//     P = 2^(c S - c m)     registers, stored over S as 16-bit operand
//     O = O + P V           tensor memory, 128 x D fp32
//
// One thread of a producer warp issues the TMA loads into a ring of units of
// 128 keys x min(D, 128) values; one thread of another issues the products; a
// warpgroup per stream does the softmax, one thread per row, so that row sums
// and maxima need no exchange. The two streams take turns on the tensor cores:
// while one's weights are computed the other's products run. D = 256 leaves
// tensor memory for one output only, and its two S buffers do the same for
// consecutive tiles of one stream.
//
// The maximum that the weights are relative to is only moved when a row's true
// maximum is more than 2^8 above it (weights stay below 2^8, exact in range for
// both types); moving it costs a pass over O in tensor memory and is rare
// after the first tiles.
//
// Products with masked keys are 0 * v, which is not 0 where v is infinite or
// NaN. A row whose output comes out non-finite is therefore computed again, its
// masked keys left out by selection (attn_core.cuh): nothing is spent on it
// unless such values occur.
//
// What bounds it: 4 D products per (query, key) pair on the tensor cores
// against one exponential per pair on the special-function units.
#include "attn_tc.cuh"
#include "attn_tiles.cuh"
#include "attn_tma.h"
#include "kv_common.cuh"

namespace rssm {

namespace {

template <int D>
struct TcCfg {
  static constexpr int NS = D == 256 ? 1 : 2;        // streams
  static constexpr int DU = D < 128 ? D : 128;       // head dimensions of a unit
  static constexpr int UPT = D / DU;                 // units per tile of keys (or values)
  static constexpr int UNIT = 128 * DU * 2;
  static constexpr int NU = D == 64 ? 8 : 5;         // units in the ring
  static constexpr int QS = 128 * D * 2;             // one stream's queries
  static constexpr int NT = NS * 128 + 128;          // the producer's warpgroup: two warps work
  static constexpr int RING = NS * QS;               // its offset
  static constexpr int BARS = RING + NU * UNIT;
  static constexpr int SMEM = BARS + 512 + 1024;     // + alignment of the base
  static constexpr uint32_t O0 = 256;                // first column of O
  static_assert(SMEM <= 227 * 1024, "shared memory");
};

struct TcMaps {
  CUtensorMap q, k, v;
};

// Rows of one warp that came out non-finite, again: 16 rows at a time, 16 keys
// at a time, masked keys left out by selection.
template <typename T, int D>
__device__ __noinline__ void again(const PromptParams& p, const PromptTile& tl, int h, int tok0,
                                   int row0, int rows, unsigned char* sm, int lane) {
  constexpr int QU = D * 2 / 16;
  unsigned char* qs = sm;
  unsigned char* ks = sm + 16 * D * 2;
  unsigned char* vs = ks + 16 * D * 2;
  const int past = tl.lk - tl.lq;
  for (int r0 = row0; r0 < row0 + 32 && r0 < rows; r0 += 16) {
    for (int i = lane; i < 16 * QU; i += 32) {
      const int rr = min(r0 + i / QU, rows - 1), u = i % QU;
      const T* q = static_cast<const T*>(p.q) + (long long)(tok0 + rr / p.G) * p.qs +
                   (long long)(h * p.G + rr % p.G) * D;
      *reinterpret_cast<uint4*>(qs + unit_off<16>(i / QU, u)) =
          reinterpret_cast<const uint4*>(q)[u];
    }
    int lim[1][2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int rr = min(r0 + 8 * e + (lane >> 2), rows - 1);
      lim[0][e] = max(0, past + (tok0 - tl.q0) + rr / p.G + 1);
    }
    const int fewest = max(0, past + (tok0 - tl.q0) + r0 / p.G + 1);
    const int keys = max(0, past + (tok0 - tl.q0) + min(r0 + 15, rows - 1) / p.G + 1);
    WarpAttn<T, D, 1, 16, 16> w;
    w.clear();
    for (int key0 = 0; key0 < keys; key0 += 16) {
      __syncwarp();
      for (int i = lane; i < 16 * QU; i += 32) {
        const int kr = i / QU, u = i % QU;
        const bool live = key0 + kr < keys;
        const long long key = tl.k0 + (live ? key0 + kr : 0);
        const uint4* kg = reinterpret_cast<const uint4*>(static_cast<const T*>(p.k) + key * p.ks +
                                                         (long long)h * D) + u;
        const uint4* vg = reinterpret_cast<const uint4*>(static_cast<const T*>(p.v) + key * p.vs +
                                                         (long long)h * D) + u;
        const uint4 z = make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4*>(ks + unit_off<16>(kr, u)) = live ? *kg : z;
        *reinterpret_cast<uint4*>(vs + unit_off<16>(kr, u)) = live ? *vg : z;
      }
      __syncwarp();
      float x[1][2][4];
      w.template weights<2>(x, qs, ks, key0, lim, fewest, p.c, lane);
      w.template add<2>(x, vs, key0, lim, fewest, lane);
    }
    w.finish();
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int rr = r0 + 8 * e + (lane >> 2);
      if (rr < rows) {
        const bool none = lim[0][e] == 0;
        const float inv = none ? 0.f : 1.f / w.l[0][e];
        const size_t row = (size_t)(tok0 + rr / p.G) * p.HQ + h * p.G + rr % p.G;
        T* o = static_cast<T*>(p.o) + row * D;
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
          store2(o + w.col(i, lane & 3), w.o[0][i][2 * e] * inv, w.o[0][i][2 * e + 1] * inv);
        if (p.lse != nullptr && (lane & 3) == 0)
          p.lse[row] = none ? kNegInf : lse_of(w.m[0][e], w.l[0][e]);
      }
    }
    __syncwarp();
  }
}

// A wait that gives up after the usual limit; after the first that did, none
// of the thread's later waits waits.
__device__ __forceinline__ void tc_wait(uint64_t* bar, uint32_t parity, bool& dead) {
  if (!dead && !mbar_wait_bounded(bar, parity)) dead = true;
}

template <typename T, int D>
__global__ void __launch_bounds__(TcCfg<D>::NT, 1)
    attn_prompt_tc_kernel(const __grid_constant__ PromptParams p,
                          const __grid_constant__ TcMaps maps) {
  using C = TcCfg<D>;
  extern __shared__ unsigned char sm_raw[];
  unsigned char* sm = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(sm_raw) + 1023) & ~(uintptr_t)1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + C::BARS);  // [NU] a unit has landed
  uint64_t* empty = full + C::NU;                              // [NU] its products are done
  uint64_t* qfull = empty + C::NU;                             // queries have landed
  uint64_t* sfull = qfull + 1;                                 // [2] scores are in tensor memory
  uint64_t* pfull = sfull + 2;                                 // [2][2] half the weights are
  uint64_t* odone = pfull + 4;                                 // [2] a tile's P V is done
  uint32_t* tslot = reinterpret_cast<uint32_t*>(odone + 2);
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
  // tiles of keys that each stream sees
  int nt[2] = {0, 0};
#pragma unroll
  for (int s = 0; s < C::NS; ++s) {
    const int a = i0 + s * toks;
    if (a < tl.lq) nt[s] = (max(0, past + min(a + toks, tl.lq)) + 127) / 128;
  }
  const int ntm = max(nt[0], nt[1]);

  // The producer's warp sets the barriers up and sends for the first units
  // while the products' warp waits for tensor memory.
  bool dead = false;
  int issued = 0;  // units sent for
  auto unit = [&](const CUtensorMap* map, int tile, int part) {
    const int u = issued % C::NU;
    if (issued >= C::NU)
      tc_wait(&empty[u], (uint32_t)((issued / C::NU - 1) & 1), dead);
    ++issued;
    if (dead) return;
    mbar_expect_tx(&full[u], C::UNIT);
    for (int d = 0; d < C::DU / 64; ++d)
      tma_load3(smem_addr(sm + C::RING + u * C::UNIT + d * 16384), map, part * C::DU + 64 * d, h,
                tl.k0 + tile * 128, &full[u]);
  };
  auto tile_units = [&](const CUtensorMap* map, int tile) {
    for (int i = 0; i < C::UPT; ++i) unit(map, tile, i);
  };
  if (warp == 4 * C::NS && lane == 0) {
    for (int u = 0; u < C::NU; ++u) mbar_init(&full[u], 1), mbar_init(&empty[u], 1);
    mbar_init(qfull, 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sfull[b], 1);
      mbar_init(&pfull[2 * b], 128);
      mbar_init(&pfull[2 * b + 1], 128);
      mbar_init(&odone[b], 1);
    }
    fence_mbar_init();
    if (ntm > 0) {
      mbar_expect_tx(qfull, (uint32_t)(C::NS * (D / 64) * p.G * toks * 128));
#pragma unroll
      for (int s = 0; s < C::NS; ++s) {
        for (int d = 0; d < D / 64; ++d)
          tma_load4(smem_addr(sm + s * C::QS + d * 16384), &maps.q, 64 * d, 0, h,
                    tl.q0 + i0 + s * toks, qfull);
      }
      tile_units(&maps.k, 0);
    }
  }
  if (warp == 4 * C::NS + 1) tmem_alloc512(tslot);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tb = *tslot;

  if (warp >= 4 * C::NS) {
  // three warpgroups at 168 registers: two take 232, the producers' keeps 40
  if constexpr (C::NS == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
  if (warp == 4 * C::NS) {
    // ---- producer: after K(0), for each tile the values and the next keys in
    // the order the products take them
    if (lane == 0 && ntm > 0) {
      for (int j = 0; j < ntm; ++j) {
        if (C::NS == 1 && j + 1 < ntm) tile_units(&maps.k, j + 1);
        tile_units(&maps.v, j);
        if (C::NS == 2 && j + 1 < ntm) tile_units(&maps.k, j + 1);
      }
      // every copy has landed before the CTA leaves
      bool late = false;
      for (int k = max(0, issued - C::NU); k < issued; ++k)
        tc_wait(&full[k % C::NU], (uint32_t)((k / C::NU) & 1), late);
      dead |= late;
    }
    __syncwarp();
  } else if (warp == 4 * C::NS + 1) {
    // ---- products; the warp stays together and one lane issues
    if (ntm > 0) {
      constexpr uint32_t id_qk = f16_idesc<T>(128, 128, false);
      constexpr uint32_t id_pv = f16_idesc<T>(128, C::DU, true);
      const uint32_t el = elect_lane();
      const uint32_t qd = sw128_kmajor_lo(smem_addr(sm));
      const uint32_t kd = sw128_kmajor_lo(smem_addr(sm + C::RING));
      const uint32_t vd = sw128_mnmajor_lo(smem_addr(sm + C::RING), 16384);
      auto ready = [&](int n) { tc_wait(&full[n % C::NU], (uint32_t)((n / C::NU) & 1), dead); };
      // S[buf] = Q_s K^T, keys in units n ..
      auto qk = [&](int s, int buf, int n) {
        for (int i = 0; i < C::UPT; ++i) {
          ready(n + i);
          dead = __any_sync(kFull, dead);
          if (dead) return;
          tc_fence_after();
          const uint32_t a = qd + (s * C::QS + i * 32768) / 16;
          const uint32_t b = kd + ((n + i) % C::NU) * (C::UNIT / 16);
#pragma unroll
          for (int k = 0; k < C::DU / 16; ++k) {
            const uint32_t in = ((k / 4) * 16384 + (k % 4) * 32) / 16;
            mma16_ss(el, tb + buf * 128, a + in, b + in, id_qk, i > 0 || k > 0);
          }
        }
        mma16_commit(el, &sfull[buf]);
      };
      // O_s += P V, weights in buffer buf (its turn's parity), values in units
      // n ..; the first 64 keys' products begin when their weights are there
      auto pv = [&](int s, int buf, uint32_t par, int n, bool acc) {
        for (int i = 0; i < C::UPT; ++i) ready(n + i);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          tc_wait(&pfull[2 * buf + half], par, dead);
          dead = __any_sync(kFull, dead);
          if (dead) return;
          tc_fence_after();
          for (int i = 0; i < C::UPT; ++i) {
            const uint32_t b = vd + ((n + i) % C::NU) * (C::UNIT / 16);
#pragma unroll
            for (int k = 4 * half; k < 4 * half + 4; ++k)
              mma16_ts(el, tb + C::O0 + s * D + i * 128, tb + buf * 128 + 8 * k, b + k * 128,
                       id_pv, acc || k > 0);
          }
        }
        mma16_commit(el, &odone[s]);
      };
      auto free_units = [&](int n) {
        for (int i = 0; i < C::UPT; ++i)
          if (!dead) mma16_commit(el, &empty[(n + i) % C::NU]);
      };
      tc_wait(qfull, 0, dead);
      if constexpr (C::NS == 2) {
        // units: K0 V0 K1 V1 ...
        for (int s = 0; s < 2; ++s)
          if (nt[s] > 0) qk(s, s, 0);
        free_units(0);
        for (int j = 0; j < ntm; ++j) {
          const int nv = C::UPT * (2 * j + 1), nk = nv + C::UPT;
          for (int s = 0; s < 2; ++s) {
            if (j < nt[s]) pv(s, s, (uint32_t)(j & 1), nv, j > 0);
            if (j + 1 < nt[s]) qk(s, s, nk);
          }
          free_units(nv);
          if (j + 1 < ntm) free_units(nk);
        }
      } else {
        // units: K0 K1 V0 K2 V1 ...
        qk(0, 0, 0);
        free_units(0);
        for (int j = 0; j < ntm; ++j) {
          const bool more = j + 1 < ntm;
          const int nk = C::UPT * (2 * j + 1);
          const int nv = more ? nk + C::UPT : nk;
          if (more) {
            qk(0, (j + 1) & 1, nk);
            free_units(nk);
          }
          pv(0, j & 1, (uint32_t)((j >> 1) & 1), nv, j > 0);
          free_units(nv);
        }
      }
      if (__any_sync(kFull, dead)) {  // products in flight end before their memory is given back
        bool late = false;
        mma16_commit(el, qfull);
        tc_wait(qfull, 1, late);
      }
    }
    __syncwarp();
  }
  } else {
    if constexpr (C::NS == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
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
    const int n_tiles = nt[s];
    for (int j = 0; j < n_tiles; ++j) {
      const int buf = C::NS == 2 ? s : j & 1;
      const uint32_t par = (uint32_t)(C::NS == 2 ? j & 1 : (j >> 1) & 1);
      tc_wait(&sfull[buf], par, dead);
      dead = __any_sync(kFull, dead);
      tc_fence_after();
      const uint32_t ts = tb + lane_at + buf * 128;
      float x[128];
#pragma unroll
      for (int i = 0; i < 4; ++i) tmem_ld32(ts + 32 * i, x + 32 * i);
#pragma unroll
      for (int i = 0; i < 4; ++i) tmem_ld_wait32(x + 32 * i);
      const int key0 = j * 128;
      if (key0 + 128 > fewest) {
        const int n = lim - key0;
#pragma unroll
        for (int i = 0; i < 128; ++i) x[i] = i < n ? x[i] : kNegInf;
      }
      float t[4] = {m, kNegInf, kNegInf, kNegInf};
#pragma unroll
      for (int i = 0; i < 128; i += 8) {
#pragma unroll
        for (int k = 0; k < 4; ++k) t[k] = max3(t[k], x[i + 2 * k], x[i + 2 * k + 1]);
      }
      const float mx = max3(fmaxf(t[0], t[1]), t[2], t[3]);
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
          tc_wait(&odone[s], (uint32_t)((j - 1) & 1), dead);
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
          // A parity tells a phase only from its neighbours, so every phase of
          // odone is seen before the next can end. With two streams the scores
          // of tile j follow P V of tile j - 1; with one they do not.
          if (C::NS == 1 && q == 1 && j > 0) tc_wait(&odone[s], (uint32_t)((j - 1) & 1), dead);
          tc_fence_before();
          mbar_arrive(&pfull[2 * buf + (q >> 1)]);
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
    if (n_tiles > 0) {
      tc_wait(&odone[s], (uint32_t)((n_tiles - 1) & 1), dead);
      dead = __any_sync(kFull, dead);
      tc_fence_after();
    }
    const bool mine = row < R && !dead;
    unsigned char* st = sm + s * C::QS + (warp & 3) * (32 * D * 2);  // the warp's 32 rows
#pragma unroll 2
    for (int d = 0; d < D; d += 32) {
      float o[32];
      if (n_tiles > 0) {
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
    bad = __any_sync(kFull, bad && mine);
    // the ring is free once every stream's products are done
    named_sync(1, C::NS * 128);
    if (bad)
      again<T, D>(p, tl, h, tl.q0 + tok0, 32 * (warp & 3), R, sm + C::RING + warp * (48 * D * 2),
                  lane);
  }
  if (dead && lane == 0) atomicOr(p.err, DEVERR_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  if (warp == 4 * C::NS + 1) tmem_dealloc512(tb);
}

bool encode(CUtensorMap* map, int dt, int rank, const void* base, const cuuint64_t* dims,
            const cuuint64_t* strides, const cuuint32_t* box) {
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  return tma_encoder()(map, dt == DT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                      : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                   (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, ones,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename F>
cudaError_t pick(int D, int dt, F f) {
#define RSSM_CASE(TT, DD) \
  if (D == DD) return f(attn_prompt_tc_kernel<TT, DD>, TcCfg<DD>::NT, TcCfg<DD>::SMEM, TcCfg<DD>::NS);
#define RSSM_CASES(TT) RSSM_CASE(TT, 64) RSSM_CASE(TT, 128) RSSM_CASE(TT, 256)
  if (dt == DT_BF16) {
    RSSM_CASES(__nv_bfloat16)
  } else {
    RSSM_CASES(__half)
  }
#undef RSSM_CASES
#undef RSSM_CASE
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t attn_prompt_tc_prepare(int D, int dt) {
  if (tma_encoder() == nullptr) return cudaErrorNotSupported;
  return pick(D, dt, [](auto kernel, int, int smem, int) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  });
}

cudaError_t attn_prompt_tc_launch(const PromptParams& p, cudaStream_t st) {
  TcMaps maps;
  const cuuint64_t es = 2, D = p.D, G = p.G;
  const int toks = 128 / p.G;
  {
    const cuuint64_t dims[4] = {D, G, (cuuint64_t)p.HKV, (cuuint64_t)p.N};
    const cuuint64_t strides[3] = {D * es, G * D * es, (cuuint64_t)p.qs * es};
    const cuuint32_t box[4] = {64, (cuuint32_t)G, 1, (cuuint32_t)toks};
    if (!encode(&maps.q, p.dt, 4, p.q, dims, strides, box)) return cudaErrorInvalidValue;
  }
  // without any key the maps are never read through
  const bool any = p.M > 0;
  const cuuint64_t dims[3] = {D, (cuuint64_t)p.HKV, (cuuint64_t)(any ? p.M : 1)};
  const cuuint32_t box[3] = {64, 1, 128};
  const cuuint64_t ks[2] = {D * es, (cuuint64_t)(any ? p.ks : p.qs) * es};
  const cuuint64_t vs[2] = {D * es, (cuuint64_t)(any ? p.vs : p.qs) * es};
  if (!encode(&maps.k, p.dt, 3, any ? p.k : p.q, dims, ks, box) ||
      !encode(&maps.v, p.dt, 3, any ? p.v : p.q, dims, vs, box))
    return cudaErrorInvalidValue;
  return pick(p.D, p.dt, [&](auto kernel, int nt, int smem, int ns) {
    // every sequence has at most one tile that is not full of tokens
    const long long ctas = ((long long)p.N / (ns * toks) + p.B) * p.HKV;
    if (ctas > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    kernel<<<(unsigned)ctas, nt, smem, st>>>(p, maps);
    return cudaGetLastError();
  });
}

}  // namespace rssm
