// Causal attention over whole prompts, packed sequences of different lengths,
// grouped heads: the form for fp32, on the FMA units.
//
// Sequence b has Lq query tokens and Lk keys (its last Lq keys are the query
// tokens' own; Lk = Lq when nothing came before); query i sees keys
// 0 .. Lk - Lq + i. A row that sees no key (Lk < Lq) gives 0.
//
// A CTA takes 32 query rows of one key head: a row is a token and one of the G
// query heads that share the key head, so that short prompts fill rows and the
// keys of a head are read once for its whole group. KG groups of one or two
// warps share the keys out in tiles of 16, each staging its own by 16-byte async
// copies one tile ahead, and are joined at the end: the FMA units want many
// warps, and a prompt of a thousand tokens has few rows. (64 rows and one group
// of four warps: 104 us where this takes 51 us, five prompts of 302 to 957 keys.)
// A sequence's tiles of longer sight come first in the grid, sequences as given.
// Longer prompts (eight, the longest
// of 2048 tokens: 299 us) issue on 63% of cycles with shared memory 61% busy, no unit
// full: 12 warps per SM wait out shared loads and reductions (168 registers and
// 203 KB leave no room for more).
#include "attn_core.cuh"
#include "attn_tiles.cuh"
#include "kv_common.cuh"

namespace rssm {

namespace {

template <int D>
struct PromptCfg {
  static constexpr int MB = D == 64 ? 2 : 1;                      // sixteens of rows of a warp
  static constexpr int RW = 2 / MB;                               // row warps of a group
  static constexpr int KG = D == 64 ? 12 : D == 128 ? 6 : 3;      // groups: registers, then shared
  static constexpr int NT = 32 * RW * KG;                         // memory, hold no more
  static constexpr int ROWS = 16 * MB * RW;
  static constexpr int KEYS = 16;
  static constexpr int QBYTES = ROWS * D * 4;
  static constexpr int TBYTES = KEYS * D * 4;
  static constexpr int OP = D + 8;                                // row pitch of the join (floats)
  static constexpr int STATS = 2 * KG * ROWS * 4;
  static constexpr int SMEM = QBYTES + 4 * KG * TBYTES + STATS;
  static_assert(KG * ROWS * OP * 4 <= QBYTES + 4 * KG * TBYTES, "the join fits the tiles");
  static_assert(SMEM <= 227 * 1024, "shared memory");
};

template <int D>
__global__ void __launch_bounds__(PromptCfg<D>::NT, 1)
    attn_prompt_kernel(const __grid_constant__ PromptParams p) {
  using T = float;
  using C = PromptCfg<D>;
  extern __shared__ __align__(1024) unsigned char sm[];
  PromptTile tl;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int grp = warp / C::RW, wr = 16 * C::MB * (warp % C::RW);  // keys' group, first row
  const int gtid = tid % (32 * C::RW);
  const int h = (int)(blockIdx.x % (unsigned)p.HKV);    // heads of a tile side by side
  if (!find_tile(p, C::ROWS, (int)(blockIdx.x / (unsigned)p.HKV), h == 0 && tid < 32, tl)) return;
  const long long r0 = (long long)tl.tile * C::ROWS;    // first query row of the tile
  const int R = (int)min((long long)C::ROWS, (long long)tl.lq * p.G - r0);  // rows in use
  auto token = [&](int rr) { return (int)((r0 + rr) / p.G); };
  auto head = [&](int rr) { return h * p.G + (int)((r0 + rr) % p.G); };
  const int past = tl.lk - tl.lq;                       // may be negative
  const int keys = max(0, past + token(R - 1) + 1);  // keys any row sees
  unsigned char* qs = sm;
  unsigned char* kv = sm + C::QBYTES + grp * 4 * C::TBYTES;  // [2] keys, values

  constexpr int QU = D * 4 / 16;
  auto issue = [&](int i) {  // the group's i-th tile
    const int key0 = (grp + i * C::KG) * C::KEYS;
    if (key0 < keys) {
      const uint32_t kd = smem_addr(kv + (i & 1) * 2 * C::TBYTES), vd = kd + C::TBYTES;
#pragma unroll 4
      for (int e = gtid; e < C::KEYS * QU; e += 32 * C::RW) {
        const int rr = e / QU, u = e % QU;
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
  issue(0);
  issue(1);
  for (int i = tid; i < C::ROWS * QU; i += C::NT) {
    const int rr = i / QU, u = i % QU;
    const bool live = rr < R;
    const int tr = live ? rr : 0;
    const T* q = static_cast<const T*>(p.q) + (long long)(tl.q0 + token(tr)) * p.qs +
                 (long long)head(tr) * D;
    *reinterpret_cast<uint4*>(qs + unit_off<C::ROWS>(rr, u)) =
        live ? reinterpret_cast<const uint4*>(q)[u] : make_uint4(0, 0, 0, 0);
  }

  int lim[C::MB][2];
#pragma unroll
  for (int b = 0; b < C::MB; ++b) {
#pragma unroll
    for (int e = 0; e < 2; ++e)
      lim[b][e] = max(0, past + token(min(wr + 16 * b + 8 * e + (lane >> 2), R - 1)) + 1);
  }
  const int fewest = max(0, past + token(min(wr, R - 1)) + 1);
  const int most = max(0, past + token(min(wr + 16 * C::MB - 1, R - 1)) + 1);

  WarpAttn<T, D, C::MB, C::ROWS, C::KEYS> w;
  auto sync = [&] {  // the group's warps
    if constexpr (C::RW == 1) {
      __syncwarp();
    } else {
      named_sync(1 + grp, 32 * C::RW);
    }
  };
  w.clear();
  __syncthreads();
  for (int i = 0; (grp + i * C::KG) * C::KEYS < keys; ++i) {
    const int key0 = (grp + i * C::KG) * C::KEYS;
    cp_async_wait<1>();
    sync();
    const unsigned char* ks = kv + (i & 1) * 2 * C::TBYTES;
    if (key0 < most && wr < R) {
      float x[C::MB][C::KEYS / 8][4];
      w.template weights<C::KEYS / 8>(x, qs + wr * 128, ks, key0, lim, fewest, p.c, lane);
      w.template add<C::KEYS / 8>(x, ks + C::TBYTES, key0, lim, fewest, lane);
    }
    sync();
    issue(i + 2);
  }
  cp_async_wait<0>();
  w.finish();

  // ---- join the groups
  float* sm_m = reinterpret_cast<float*>(sm + C::QBYTES + 4 * C::KG * C::TBYTES);  // [KG][ROWS]
  float* sm_l = sm_m + C::KG * C::ROWS;
  const int g = lane >> 2, t = lane & 3;
  if (t == 0) {
#pragma unroll
    for (int b = 0; b < C::MB; ++b) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        sm_m[grp * C::ROWS + wr + 16 * b + 8 * e + g] = w.m[b][e];
        sm_l[grp * C::ROWS + wr + 16 * b + 8 * e + g] = w.l[b][e];
      }
    }
  }
  __syncthreads();
  float* os = reinterpret_cast<float*>(sm);
#pragma unroll
  for (int b = 0; b < C::MB; ++b) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int rr = wr + 16 * b + 8 * e + g;
      float mx = kNegInf;
#pragma unroll
      for (int k = 0; k < C::KG; ++k) mx = fmaxf(mx, sm_m[k * C::ROWS + rr]);
      const float f = exp2_fast(w.m[b][e] - (mx == kNegInf ? 0.f : mx));
      if (rr < R) {
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
          *reinterpret_cast<float2*>(os + (grp * C::ROWS + rr) * C::OP + w.col(i, t)) =
              make_float2(w.o[b][i][2 * e] * f, w.o[b][i][2 * e + 1] * f);
      }
    }
  }
  __syncthreads();
  for (int i = tid; i < R * (D / 4); i += C::NT) {
    const int rr = i / (D / 4), d = 4 * (i % (D / 4));
    float mx = kNegInf, l = 0.f;
#pragma unroll
    for (int k = 0; k < C::KG; ++k) mx = fmaxf(mx, sm_m[k * C::ROWS + rr]);
    const float mu = mx == kNegInf ? 0.f : mx;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < C::KG; ++k) {
      l += sm_l[k * C::ROWS + rr] * exp2_fast(sm_m[k * C::ROWS + rr] - mu);
      const float4 y = *reinterpret_cast<const float4*>(os + (k * C::ROWS + rr) * C::OP + d);
      a.x += y.x;
      a.y += y.y;
      a.z += y.z;
      a.w += y.w;
    }
    const bool none = past + token(rr) + 1 <= 0;
    const float inv = none ? 0.f : 1.f / l;
    const size_t row = (size_t)(tl.q0 + token(rr)) * p.HQ + head(rr);
    *reinterpret_cast<float4*>(static_cast<T*>(p.o) + row * D + d) =
        none ? make_float4(0.f, 0.f, 0.f, 0.f)
             : make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
    if (p.lse != nullptr && d == 0) p.lse[row] = none ? kNegInf : lse_of(mx, l);
  }
}

template <typename F>
cudaError_t pick(int D, F f) {
  switch (D) {
    case 64: return f(attn_prompt_kernel<64>, PromptCfg<64>::NT, PromptCfg<64>::SMEM);
    case 128: return f(attn_prompt_kernel<128>, PromptCfg<128>::NT, PromptCfg<128>::SMEM);
    case 256: return f(attn_prompt_kernel<256>, PromptCfg<256>::NT, PromptCfg<256>::SMEM);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t attn_prompt_prepare(int D, int dt) {
  if (dt != DT_F32) return attn_prompt_tc_prepare(D, dt);
  return pick(D, [](auto kernel, int, int smem) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  });
}

cudaError_t attn_prompt_launch(const PromptParams& p, cudaStream_t st) {
  if (p.dt != DT_F32) return attn_prompt_tc_launch(p, st);
  // every sequence has at most one tile that is not full
  const long long ctas = ((long long)p.N * p.G / 32 + p.B) * p.HKV;
  if (ctas > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  return pick(p.D, [&](auto kernel, int nt, int smem) {
    kernel<<<(unsigned)ctas, nt, smem, st>>>(p);
    return cudaGetLastError();
  });
}

}  // namespace rssm
