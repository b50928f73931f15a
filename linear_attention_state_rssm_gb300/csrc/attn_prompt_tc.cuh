// What the two tensor-core forms of prompt attention share: their tensor maps,
// bounded waits, and the rows that values they must not see have spoilt.
#pragma once

#include "attn_tc.cuh"
#include "attn_tiles.cuh"
#include "attn_tma.h"
#include "kv_common.cuh"

namespace rssm {

struct TcMaps {
  CUtensorMap q, k, v;
};

// Whether any value of keys [k0, k1) of head h is infinite or NaN (whole warp).
template <typename T, int D>
__device__ __forceinline__ bool unfinite_values(const PromptParams& p, int h, long long k0,
                                                long long k1, int lane) {
  bool bad = false;
  for (long long i = lane; i < (k1 - k0) * (D / 2); i += 32) {
    const T* v = static_cast<const T*>(p.v) + (k0 + i / (D / 2)) * p.vs + (long long)h * D +
                 2 * (i % (D / 2));
    bad |= !isfinite(attn_f32(v[0])) || !isfinite(attn_f32(v[1]));
  }
  return __any_sync(kFull, bad);
}

// Rows [row0, row0 + 32) of a stream (one warp's) whose outputs are not all
// finite, again where a value that some of them must not see is to blame. Keys
// and values come straight from global memory: the ring is the next tile's.
template <typename T, int D>
__device__ __noinline__ void again(const PromptParams& p, const PromptTile& tl, int h, int tok0,
                                   int row0, int rows, int keys, int lane) {
  const int g = lane >> 2, t = lane & 3;
  const int past = tl.lk - tl.lq;
  auto sees = [&](int rr) { return max(0, past + tok0 + rr / p.G + 1); };
  for (int r0 = row0; r0 < row0 + 32 && r0 < rows; r0 += 16) {
    const int fewest = sees(r0), most = sees(min(r0 + 15, rows - 1));
    if (!unfinite_values<T, D>(p, h, (long long)tl.k0 + fewest, (long long)tl.k0 + keys, lane))
      continue;
    int lim[1][2];
    const T* q[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int rr = min(r0 + 8 * e + g, rows - 1);
      lim[0][e] = sees(rr);
      q[e] = static_cast<const T*>(p.q) + (long long)(tl.q0 + tok0 + rr / p.G) * p.qs +
             (long long)(h * p.G + rr % p.G) * D + 2 * t;
    }
    auto word = [](const T* x) { return *reinterpret_cast<const uint32_t*>(x); };
    WarpAttn<T, D, 1, 16, 16> w;
    w.clear();
    for (int key0 = 0; key0 < most; key0 += 16) {
      auto key = [&](int k) { return (long long)tl.k0 + min(key0 + k, most - 1); };
      const T* kg[2];
#pragma unroll
      for (int n = 0; n < 2; ++n)
        kg[n] = static_cast<const T*>(p.k) + key(8 * n + g) * p.ks + (long long)h * D + 2 * t;
      float x[1][2][4] = {};
#pragma unroll 4
      for (int d = 0; d < D; d += 16) {
        const uint32_t a[4] = {word(q[0] + d), word(q[1] + d), word(q[0] + d + 8),
                               word(q[1] + d + 8)};
#pragma unroll
        for (int n = 0; n < 2; ++n) mma16<T>(x[0][n], a, word(kg[n] + d), word(kg[n] + d + 8));
      }
      w.template soften<2>(x, key0, lim, 0, p.c, lane);
      w.template pv_select<2>(
          x,
          [&](int k, int d) {
            const T* v = static_cast<const T*>(p.v) + key(k) * p.vs + (long long)h * D + d;
            return make_float2(attn_f32(v[0]), attn_f32(v[1]));
          },
          key0, lim, lane);
    }
    w.finish();
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int rr = r0 + 8 * e + g;
      if (rr < rows) {
        const bool none = lim[0][e] == 0;
        const float inv = none ? 0.f : 1.f / w.l[0][e];
        const size_t row = (size_t)(tl.q0 + tok0 + rr / p.G) * p.HQ + h * p.G + rr % p.G;
        T* o = static_cast<T*>(p.o) + row * D;
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
          store2(o + w.col(i, t), w.o[0][i][2 * e] * inv, w.o[0][i][2 * e + 1] * inv);
        if (p.lse != nullptr && t == 0) p.lse[row] = none ? kNegInf : lse_of(w.m[0][e], w.l[0][e]);
      }
    }
  }
}

// A wait that gives up after the usual limit; after the first that did, none
// of the thread's later waits waits. The hardware parks the warp meanwhile: a
// warp that polls takes issue slots from the softmax warp beside it.
// `told` (may be null) becomes non-zero when it gives up.
__device__ __forceinline__ void tc_wait(uint64_t* bar, uint32_t parity, bool& dead,
                                        volatile uint32_t* told = nullptr) {
  if (dead || mbar_try_wait(bar, parity)) return;
  const unsigned long long t0 = global_ns();
  while (!mbar_try_wait_hint(bar, parity, 20000)) {
    if (global_ns() - t0 > kWaitLimitNs) {
      dead = true;
      if (told != nullptr) *told = 1;
      return;
    }
  }
}

// Test hook: the first copy into place `unit` of the ring, or of the queries
// (the place behind it), is promised more than it brings.
template <int NU>
__device__ __forceinline__ void promise_more(uint64_t* full, uint64_t* qfull, int unit) {
  const int place = unit % (NU + 1);
  mbar_promise(place < NU ? full + place : qfull, 16);
}

inline bool encode(CUtensorMap* map, int dt, int rank, const void* base, const cuuint64_t* dims,
            const cuuint64_t* strides, const cuuint32_t* box) {
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  return tma_encoder()(map, dt == DT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                      : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                   (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, ones,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Queries in boxes of 64 dimensions, G heads and floor(128 / G) tokens; keys and
// values in boxes of 64 dimensions and 128 tokens.
inline bool encode_maps(const PromptParams& p, TcMaps* maps) {
  const cuuint64_t es = 2, D = p.D, G = p.G;
  {
    const cuuint64_t dims[4] = {D, G, (cuuint64_t)p.HKV, (cuuint64_t)p.N};
    const cuuint64_t strides[3] = {D * es, G * D * es, (cuuint64_t)p.qs * es};
    const cuuint32_t box[4] = {64, (cuuint32_t)G, 1, (cuuint32_t)(128 / p.G)};
    if (!encode(&maps->q, p.dt, 4, p.q, dims, strides, box)) return false;
  }
  // without any key the maps are never read through
  const bool any = p.M > 0;
  const cuuint64_t dims[3] = {D, (cuuint64_t)p.HKV, (cuuint64_t)(any ? p.M : 1)};
  const cuuint32_t box[3] = {64, 1, 128};
  const cuuint64_t ks[2] = {D * es, (cuuint64_t)(any ? p.ks : p.qs) * es};
  const cuuint64_t vs[2] = {D * es, (cuuint64_t)(any ? p.vs : p.qs) * es};
  return encode(&maps->k, p.dt, 3, any ? p.k : p.q, dims, ks, box) &&
         encode(&maps->v, p.dt, 3, any ? p.v : p.q, dims, vs, box);
}

// Zeros in 128-byte rows [v, 128) of the 64-wide columns of a unit: values
// behind the last key (whole warp). Not inlined: used once a tile, it would
// stand amid the loops of the role that calls it (5% of heads of 64).
template <int DU>
__device__ __noinline__ void zero_rows(unsigned char* unit, int v, int lane) {
#pragma unroll 1
  for (int d = 0; d < DU / 64; ++d) {
    uint4* u = reinterpret_cast<uint4*>(unit + d * 16384);
#pragma unroll 1
    for (int e = 8 * v + lane; e < 128 * 8; e += 32) u[e] = make_uint4(0, 0, 0, 0);
  }
  fence_async_smem();
  __syncwarp();
}

}  // namespace rssm
