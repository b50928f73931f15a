// Causal attention over whole prompts, packed sequences of different lengths,
// grouped heads: the warp-level form, for fp32.
//
// Sequence b has Lq query tokens and Lk keys (its last Lq keys are the query
// tokens' own; Lk = Lq when nothing came before); query i sees keys
// 0 .. Lk - Lq + i. A row that sees no key (Lk < Lq) gives 0.
//
// A CTA takes 64 query rows of one key head: floor(64 / G) tokens with their G
// query heads, so that short prompts fill rows and the keys of a head are read
// once for its whole group. Tiles of 32 keys and values are staged by 16-byte
// async copies, one tile ahead. Rows of longer sight come first in the grid.
#include "attn_core.cuh"
#include "kv_common.cuh"
#include "attn_tiles.cuh"

namespace rssm {

namespace {

template <typename T, int D>
struct PromptCfg {
  static constexpr int NW = 4;
  static constexpr int NT = NW * 32;
  static constexpr int ROWS = 16 * NW;
  static constexpr int KEYS = 32;
  static constexpr int QBYTES = ROWS * D * (int)sizeof(T);
  static constexpr int TBYTES = KEYS * D * (int)sizeof(T);
  static constexpr int SMEM = QBYTES + 4 * TBYTES;
};

template <typename T, int D>
__global__ void __launch_bounds__(PromptCfg<T, D>::NT) attn_prompt_kernel(const __grid_constant__ PromptParams p) {
  using C = PromptCfg<T, D>;
  extern __shared__ __align__(1024) unsigned char sm[];
  PromptTile tl;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int toks = C::ROWS / p.G;  // query tokens of a tile
  const int h = (int)(blockIdx.x % (unsigned)p.HKV);    // heads of a tile side by side
  if (!find_tile(p, toks, (int)(blockIdx.x / (unsigned)p.HKV), h == 0 && tid < 32, tl)) return;
  const int i0 = tl.tile * toks;                        // first query token of the tile
  const int R = min(toks, tl.lq - i0) * p.G;            // rows in use
  const int past = tl.lk - tl.lq;                       // may be negative
  const int keys = max(0, min(tl.lk, past + min(i0 + toks, tl.lq)));  // keys any row sees
  unsigned char* qs = sm;
  unsigned char* kv = sm + C::QBYTES;

  constexpr int QU = D * (int)sizeof(T) / 16;
  for (int i = tid; i < C::ROWS * QU; i += C::NT) {
    const int rr = i / QU, u = i % QU;
    const bool live = rr < R;
    const int tr = live ? rr : 0;
    const T* q = static_cast<const T*>(p.q) + (long long)(tl.q0 + i0 + tr / p.G) * p.qs +
                 (long long)(h * p.G + tr % p.G) * D;
    *reinterpret_cast<uint4*>(qs + unit_off<C::ROWS>(rr, u)) =
        live ? reinterpret_cast<const uint4*>(q)[u] : make_uint4(0, 0, 0, 0);
  }

  auto issue = [&](int j) {
    const int key0 = j * C::KEYS;
    if (key0 < keys) {
      const uint32_t kd = smem_addr(kv + (j & 1) * 2 * C::TBYTES), vd = kd + C::TBYTES;
      for (int i = tid; i < C::KEYS * QU; i += C::NT) {
        const int rr = i / QU, u = i % QU;
        const bool live = key0 + rr < keys;
        const long long key = tl.k0 + (live ? key0 + rr : 0);
        const T* k = static_cast<const T*>(p.k) + key * p.ks + (long long)h * D;
        const T* v = static_cast<const T*>(p.v) + key * p.vs + (long long)h * D;
        cp_async16_or_zero(kd + unit_off<C::KEYS>(rr, u), reinterpret_cast<const uint4*>(k) + u, live);
        cp_async16_or_zero(vd + unit_off<C::KEYS>(rr, u), reinterpret_cast<const uint4*>(v) + u, live);
      }
    }
    cp_async_commit();
  };

  int lim[1][2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int rr = min(16 * warp + 8 * e + (lane >> 2), R - 1);
    lim[0][e] = max(0, past + i0 + rr / p.G + 1);
  }
  const int r_first = min(16 * warp, R - 1), r_last = min(16 * warp + 15, R - 1);
  const int fewest = max(0, past + i0 + r_first / p.G + 1);
  const int most = max(0, past + i0 + r_last / p.G + 1);

  WarpAttn<T, D, 1, C::ROWS, C::KEYS> w;
  w.clear();
  const int nt = (keys + C::KEYS - 1) / C::KEYS;
  issue(0);
  issue(1);
  for (int j = 0; j < nt; ++j) {
    cp_async_wait<1>();
    __syncthreads();
    const unsigned char* ks = kv + (j & 1) * 2 * C::TBYTES;
    const int key0 = j * C::KEYS;
    if (key0 < most && 16 * warp < R) {
      float x[1][C::KEYS / 8][4];
      w.template weights<C::KEYS / 8>(x, qs + 16 * warp * 128, ks, key0, lim, fewest,
                                      p.c, lane);
      w.template add<C::KEYS / 8>(x, ks + C::TBYTES, key0, lim, fewest, lane);
    }
    __syncthreads();
    issue(j + 2);
  }
  cp_async_wait<0>();
  w.finish();

  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int rr = 16 * warp + 8 * e + g;
    if (rr < R) {
      const bool none = lim[0][e] == 0;
      const float inv = none ? 0.f : 1.f / w.l[0][e];
      const size_t row = (size_t)(tl.q0 + i0 + rr / p.G) * p.HQ + h * p.G + rr % p.G;
      T* o = static_cast<T*>(p.o) + row * D;
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        store2(o + w.col(i, t), w.o[0][i][2 * e] * inv, w.o[0][i][2 * e + 1] * inv);
      if (p.lse != nullptr && t == 0) p.lse[row] = none ? kNegInf : lse_of(w.m[0][e], w.l[0][e]);
    }
  }
}

template <typename F>
cudaError_t pick(int D, F f) {
  switch (D) {
    case 64: return f(attn_prompt_kernel<float, 64>, PromptCfg<float, 64>::SMEM);
    case 128: return f(attn_prompt_kernel<float, 128>, PromptCfg<float, 128>::SMEM);
    case 256: return f(attn_prompt_kernel<float, 256>, PromptCfg<float, 256>::SMEM);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t attn_prompt_prepare(int D, int dt) {
  if (dt != DT_F32) return attn_prompt_tc_prepare(D, dt);
  return pick(D, [](auto kernel, int smem) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  });
}

cudaError_t attn_prompt_launch(const PromptParams& p, cudaStream_t st) {
  if (p.dt != DT_F32) return attn_prompt_tc_launch(p, st);
  // every sequence has at most one tile that is not full of tokens
  const int toks = 64 / p.G;
  const long long ctas = ((long long)p.N / toks + p.B) * p.HKV;
  if (ctas > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  return pick(p.D, [&](auto kernel, int smem) {
    kernel<<<(unsigned)ctas, 128, smem, st>>>(p);
    return cudaGetLastError();
  });
}

}  // namespace rssm
