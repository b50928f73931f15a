// Attention of a window of T new tokens per request over its paged cache.
//
// For row r with slot s: query token t (its key and value already appended at
// cache position length[s] + t) sees the cache positions 0 .. length[s] + t.
// The T G query rows of one key head (G query heads share it) form blocks of
// 16 MB rows; a block reads the keys and values of its head once, from HBM.
//
// Bytes bound it: 2 D values per key and head, 2 T G D products with them. So
// the loads have to be many and wide, and the work has to be even whatever the
// lengths: the tiles (128 keys) of every (row, key head, block) are laid on
// one line, and each CTA of one wave takes an equal stretch of it. A stretch
// that begins or ends inside a row leaves a part (running maximum, sum and
// unnormalised output) in the work buffer; the last CTA to leave one for a row
// joins them, in the order of the keys whoever it is, so results do not depend
// on the order of arrival.
//
// Within a CTA each warp streams its own chunks of 16 keys (chunk w, w + NW,
// ...) through a private ring of shared memory by 16-byte async copies, keys
// and values as separate units; no barrier between warps until the row ends.
#include "attn_core.cuh"
#include "kv_common.cuh"

namespace rssm {

namespace {

constexpr int kChunk = 16;  // keys of a warp's step: within one page (pages of 16 k keys)

template <typename T, int D, int MB>
struct DecCfg {
  static constexpr int NW = std::is_same<T, float>::value && D == 256 ? 4 : 8;
  static constexpr int NT = NW * 32;
  static constexpr int ROWS = 16 * MB;
  static constexpr int TILE = kChunk * NW;             // keys of a tile
  static constexpr int UNIT = kChunk * D * (int)sizeof(T);
  static constexpr int NS = 196608 / NW / UNIT;        // units in a warp's ring
  static constexpr int RING = NS * UNIT;               // bytes per warp
  static constexpr int QBYTES = ROWS * D * (int)sizeof(T);
  static constexpr int OP = D + 8;                     // row pitch of the warps' outputs (floats)
  static constexpr int STATS = 2 * NW * ROWS * 4;      // every warp's m and l
  static constexpr int SMEM = NW * RING + QBYTES + STATS + ROWS * 8 + 256;
  static_assert(NS >= 3, "keys, values and the next keys");
  static_assert(NW * ROWS * OP * 4 <= NW * RING, "the warps' outputs fit the ring");
  static_assert(SMEM <= 227 * 1024, "shared memory");
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

__device__ __forceinline__ long long warp_scan(long long x, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long y = __shfl_up_sync(kFull, x, d);
    if (lane >= d) x += y;
  }
  return x;
}

template <typename T, int D, int MB>
__global__ void __launch_bounds__(DecCfg<T, D, MB>::NT, 1)
    attn_decode_kernel(const __grid_constant__ DecodeParams p) {
  using C = DecCfg<T, D, MB>;
  constexpr int NW = C::NW;
  extern __shared__ __align__(1024) unsigned char sm[];
  unsigned char* qs = sm + NW * C::RING;
  float* sm_m = reinterpret_cast<float*>(qs + C::QBYTES);  // [NW][ROWS]
  float* sm_l = sm_m + NW * C::ROWS;
  float* row_m = sm_l + NW * C::ROWS;                      // [ROWS]
  float* row_l = row_m + C::ROWS;
  long long* scan = reinterpret_cast<long long*>(row_l + C::ROWS);  // [NW + 3]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  unsigned char* ring = sm + warp * C::RING;
  const int items = p.HKV * p.nmb;
  const size_t head_bytes = ((size_t)D * sizeof(T)) << p.shift;   // one head of a page
  const size_t page_bytes = head_bytes * p.HKV;

  // ---- this CTA's stretch of the line of tiles
  long long mine = 0;
  for (int r = tid; r < p.B; r += C::NT) {
    int s;
    const int n = row_keys(p, r, blockIdx.x == 0, s);
    mine += (n + C::TILE - 1) / C::TILE;
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) mine += __shfl_xor_sync(kFull, mine, d);
  if (lane == 0) scan[warp] = mine;
  __syncthreads();
  long long total = 0;
  for (int w = 0; w < NW; ++w) total += scan[w];
  __syncthreads();
  total *= items;
  const long long share = (total + gridDim.x - 1) / gridDim.x;
  long long pos = share * blockIdx.x;
  const long long end = pos + share < total ? pos + share : total;
  if (pos >= end) return;

  // ---- the row that holds tile `pos`
  int row = 0;
  long long row0 = 0;  // its first tile
  for (int r0 = 0; r0 < p.B; r0 += C::NT) {
    const int r = r0 + tid;
    int s, n = 0;
    if (r < p.B) n = row_keys(p, r, false, s);
    const long long w = (long long)((n + C::TILE - 1) / C::TILE) * items;
    const long long incl = warp_scan(w, lane);
    if (lane == 31) scan[warp] = incl;
    if (tid == 0) scan[NW] = -1;
    __syncthreads();
    long long at = row0 + incl - w;
    for (int i = 0; i < warp; ++i) at += scan[i];
    if (at <= pos && pos < at + w) {
      scan[NW] = r;
      scan[NW + 1] = at;
    }
    long long sum = 0;
    for (int i = 0; i < NW; ++i) sum += scan[i];
    __syncthreads();
    const long long found = scan[NW];
    if (found >= 0) {
      row = (int)found;
      row0 = scan[NW + 1];
      break;
    }
    row0 += sum;
    __syncthreads();
  }
  __syncthreads();

  while (pos < end) {
    int slot;
    const int keys = row_keys(p, row, false, slot);
    const int tiles = (keys + C::TILE - 1) / C::TILE;
    if (tiles == 0) {
      ++row;
      continue;
    }
    if (pos >= row0 + (long long)tiles * items) {
      row0 += (long long)tiles * items;
      ++row;
      continue;
    }
    const int item = (int)((pos - row0) / tiles);
    const int t0 = (int)((pos - row0) % tiles);
    const long long item0 = row0 + (long long)item * tiles;
    const int t1 = (long long)tiles - t0 <= end - pos ? tiles : t0 + (int)(end - pos);
    const int h = item / p.nmb, mb = item % p.nmb;
    const int base = mb * C::ROWS;                     // first of the block's T G rows
    const int R = min(C::ROWS, p.T * p.G - base);      // rows in use

    // ---- query rows (zeros behind the last)
    constexpr int QU = D * (int)sizeof(T) / 16;        // units per row
    for (int i = tid; i < C::ROWS * QU; i += C::NT) {
      const int rr = i / QU, u = i % QU;
      const bool live = rr < R;
      const int tr = live ? base + rr : 0;
      const T* q = static_cast<const T*>(p.q) + ((long long)row * p.T + tr / p.G) * p.qs +
                   (long long)(h * p.G + tr % p.G) * D;
      *reinterpret_cast<uint4*>(qs + unit_off<T, D>(rr, u)) =
          live ? reinterpret_cast<const uint4*>(q)[u] : make_uint4(0, 0, 0, 0);
    }
    __syncthreads();

    // ---- how many keys the lane's rows see
    const int first = keys - p.T;  // committed keys
    int lim[MB][2];
#pragma unroll
    for (int b = 0; b < MB; ++b) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int rr = min(16 * b + 8 * e + (lane >> 2), R - 1);
        lim[b][e] = first + (base + rr) / p.G + 1;
      }
    }
    const int fewest = first + base / p.G + 1;

    // ---- the warp's stream: chunks t0 NW + warp, + NW, ... below t1 NW
    const int c0 = t0 * NW + warp;
    const int c_end = min(t1 * NW, (keys + kChunk - 1) / kChunk);
    const int nc = c0 < c_end ? (c_end - c0 + NW - 1) / NW : 0;
    const int32_t* tab = p.table + (size_t)slot * p.max_pages;
    WarpAttn<T, D, MB> w;
    w.clear();
    int page = nc > 0 ? tab[(c0 * kChunk) >> p.shift] : 0;
    const unsigned char* at = nullptr;  // the chunk's first key within the pool
    bool known = false;
    auto issue = [&](int u) {  // unit u: keys (even) or values (odd) of chunk u / 2
      if (u < 2 * nc) {
        const int key0 = (c0 + (u >> 1) * NW) * kChunk;
        if ((u & 1) == 0) {
          known = page >= 0 && page < p.n_pages;
          if (!known && lane == 0) atomicOr(p.err, DEVERR_PAGES);
          const size_t off = (size_t)(known ? page : 0) * page_bytes + h * head_bytes +
                             (size_t)(key0 & ((1 << p.shift) - 1)) * (D * sizeof(T));
          at = p.kp + off;
          if ((u >> 1) + 1 < nc) page = tab[(key0 + NW * kChunk) >> p.shift];
        } else {
          at = p.vp + (at - p.kp);
        }
        const uint32_t dst = smem_addr(ring + (u % C::NS) * C::UNIT);
        const int live = known ? keys - key0 : 0;
#pragma unroll 8
        for (int i = lane; i < kChunk * QU; i += 32) {
          const int rr = i / QU, un = i % QU;
          cp_async16_or_zero(dst + unit_off<T, D>(rr, un), at + (size_t)i * 16, rr < live);
        }
      }
      cp_async_commit();
    };
#pragma unroll
    for (int u = 0; u < C::NS; ++u) issue(u);
    for (int i = 0; i < nc; ++i) {
      // one group per unit: the oldest has landed when NS - 1 are on their way
      const int key0 = (c0 + i * NW) * kChunk;
      float x[MB][2][4];
      cp_async_wait<C::NS - 1>();
      __syncwarp();
      w.template weights<2>(x, qs, ring + ((2 * i) % C::NS) * C::UNIT, key0, lim, fewest, p.c,
                            lane);
      __syncwarp();
      issue(2 * i + C::NS);
      cp_async_wait<C::NS - 1>();
      __syncwarp();
      w.template add<2>(x, ring + ((2 * i + 1) % C::NS) * C::UNIT, key0, lim, fewest, keys, lane);
      __syncwarp();
      issue(2 * i + 1 + C::NS);
    }
    cp_async_wait<0>();
    w.finish();

    // ---- join the warps
    const int g = lane >> 2, tq = lane & 3;
    if (tq == 0) {
#pragma unroll
      for (int b = 0; b < MB; ++b) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          sm_m[warp * C::ROWS + 16 * b + 8 * e + g] = w.m[b][e];
          sm_l[warp * C::ROWS + 16 * b + 8 * e + g] = w.l[b][e];
        }
      }
    }
    __syncthreads();  // statistics written; every warp is done with its ring
    float* ow = reinterpret_cast<float*>(sm) + warp * C::ROWS * C::OP;
#pragma unroll
    for (int b = 0; b < MB; ++b) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int rr = 16 * b + 8 * e + g;
        if (rr < R) {
          float mx = kNegInf;
#pragma unroll
          for (int k = 0; k < NW; ++k) mx = fmaxf(mx, sm_m[k * C::ROWS + rr]);
          const float mu = mx == kNegInf ? 0.f : mx;
          const float f = exp2_fast(w.m[b][e] - mu);
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            *reinterpret_cast<float2*>(ow + rr * C::OP + w.col(i, tq)) =
                make_float2(w.o[b][i][2 * e] * f, w.o[b][i][2 * e + 1] * f);
          }
          if (warp == 0 && tq == 0) {
            float sum = 0.f;
#pragma unroll
            for (int k = 0; k < NW; ++k)
              sum += sm_l[k * C::ROWS + rr] * exp2_fast(sm_m[k * C::ROWS + rr] - mu);
            row_m[rr] = mx;
            row_l[rr] = sum;
          }
        }
      }
    }
    __syncthreads();

    const bool whole = t0 == 0 && t1 == tiles;
    const bool head = item0 < share * blockIdx.x;  // the row began in an earlier CTA
    float* part = p.part + (size_t)(2 * blockIdx.x + (head ? 0 : 1)) * (kPartFloats + kPartStats);
    const float* os = reinterpret_cast<const float*>(sm);
    for (int i = tid; i < R * (D / 2); i += C::NT) {
      const int rr = i / (D / 2), d = 2 * (i % (D / 2));
      float2 a = make_float2(0.f, 0.f);
#pragma unroll
      for (int k = 0; k < NW; ++k) {
        const float2 y =
            *reinterpret_cast<const float2*>(os + (k * C::ROWS + rr) * C::OP + d);
        a.x += y.x;
        a.y += y.y;
      }
      if (whole) {
        const float inv = 1.f / row_l[rr];
        const int tr = base + rr;
        T* o = static_cast<T*>(p.o) + (((size_t)row * p.T + tr / p.G) * p.HQ + h * p.G + tr % p.G) * D;
        store2(o + d, a.x * inv, a.y * inv);
      } else {
        *reinterpret_cast<float2*>(part + rr * D + d) = a;
      }
    }
    if (tid < R) {
      if (!whole) {
        part[kPartFloats + tid] = row_m[tid];
        part[kPartFloats + 64 + tid] = row_l[tid];
      } else if (p.lse != nullptr) {
        const int tr = base + tid;
        p.lse[((size_t)row * p.T + tr / p.G) * p.HQ + h * p.G + tr % p.G] =
            lse_of(row_m[tid], row_l[tid]);
      }
    }

    if (!whole) {
      // ---- the last part to arrive joins the row's parts
      const int cta0 = (int)(item0 / share);
      const int parts = (int)((item0 + tiles - 1) / share) - cta0 + 1;
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        const int n = atomicAdd(p.count + cta0, 1);
        if (n == parts - 1) p.count[cta0] = 0;  // free for the next call
        scan[NW + 2] = n == parts - 1;
        __threadfence();
      }
      __syncthreads();
      if (scan[NW + 2]) {
        const size_t stride = kPartFloats + kPartStats;
        // part k of the row: the first CTA's second slot, then first slots
        const float* parts0 = p.part + (size_t)(2 * cta0 + 1) * stride;
        const float* partsn = p.part + (size_t)(2 * cta0) * stride;
        auto at_part = [&](int k) { return k == 0 ? parts0 : partsn + (size_t)2 * k * stride; };
        float* wt = reinterpret_cast<float*>(sm);  // [parts][R] weights
        for (int i = tid; i < parts * R; i += C::NT)
          wt[i] = __ldcg(at_part(i / R) + kPartFloats + i % R);
        __syncthreads();
        if (tid < R) {
          float mx = kNegInf;
          for (int k = 0; k < parts; ++k) mx = fmaxf(mx, wt[k * R + tid]);
          row_m[tid] = mx;
        }
        __syncthreads();
        for (int i = tid; i < parts * R; i += C::NT) {
          const float mu = row_m[i % R] == kNegInf ? 0.f : row_m[i % R];
          wt[i] = exp2_fast(wt[i] - mu);
        }
        __syncthreads();
        if (tid < R) {
          float sum = 0.f;
          for (int k = 0; k < parts; ++k)
            sum += wt[k * R + tid] * __ldcg(at_part(k) + kPartFloats + 64 + tid);
          row_l[tid] = sum;
        }
        __syncthreads();
        for (int i = tid; i < R * (D / 4); i += C::NT) {
          const int rr = i / (D / 4), d = 4 * (i % (D / 4));
          float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
          for (int k = 0; k < parts; ++k) {
            const float4 y = __ldcg(reinterpret_cast<const float4*>(at_part(k) + rr * D + d));
            const float f = wt[k * R + rr];
            a.x = fmaf(f, y.x, a.x);
            a.y = fmaf(f, y.y, a.y);
            a.z = fmaf(f, y.z, a.z);
            a.w = fmaf(f, y.w, a.w);
          }
          const float inv = 1.f / row_l[rr];
          const int tr = base + rr;
          T* o = static_cast<T*>(p.o) +
                 (((size_t)row * p.T + tr / p.G) * p.HQ + h * p.G + tr % p.G) * D;
          store2(o + d, a.x * inv, a.y * inv);
          store2(o + d + 2, a.z * inv, a.w * inv);
        }
        if (tid < R && p.lse != nullptr) {
          const int tr = base + tid;
          p.lse[((size_t)row * p.T + tr / p.G) * p.HQ + h * p.G + tr % p.G] =
              lse_of(row_m[tid], row_l[tid]);
        }
      }
    }
    __syncthreads();  // shared memory is free for the next stretch
    pos += t1 - t0;
  }
}

// blocks of 16 rows a warp carries at once: outputs of 16 MB D values in
// registers (128 a lane at most)
int blocks_for(int D, int dt, int rows) {
  if (dt == DT_F32 || D == 256 || rows <= 16) return 1;
  if (D == 128 || rows <= 32) return 2;
  return 4;
}

template <typename F>
cudaError_t pick(int D, int dt, int mb, F f) {
#define RSSM_CASE(TT, DD, MM) \
  if (D == DD && mb == MM) return f(attn_decode_kernel<TT, DD, MM>, DecCfg<TT, DD, MM>::NT, DecCfg<TT, DD, MM>::SMEM);
#define RSSM_CASES16(TT)                                                  \
  RSSM_CASE(TT, 64, 1) RSSM_CASE(TT, 64, 2) RSSM_CASE(TT, 64, 4)          \
  RSSM_CASE(TT, 128, 1) RSSM_CASE(TT, 128, 2) RSSM_CASE(TT, 256, 1)
  if (dt == DT_F32) {
    RSSM_CASE(float, 64, 1) RSSM_CASE(float, 128, 1) RSSM_CASE(float, 256, 1)
  } else if (dt == DT_BF16) {
    RSSM_CASES16(__nv_bfloat16)
  } else {
    RSSM_CASES16(__half)
  }
#undef RSSM_CASES16
#undef RSSM_CASE
  return cudaErrorInvalidValue;
}

}  // namespace

int attn_decode_block_rows(int D, int dt, int rows) { return 16 * blocks_for(D, dt, rows); }

cudaError_t attn_decode_prepare(int D, int dt) {
  for (int mb = 1; mb <= 4; mb *= 2) {
    if (mb > blocks_for(D, dt, 64)) break;
    const cudaError_t e = pick(D, dt, mb, [](auto kernel, int, int smem) {
      return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    });
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t attn_decode_launch(const DecodeParams& p, int D, int dt, int num_sms,
                               cudaStream_t st) {
  const int grid = num_sms < kMaxParts ? num_sms : kMaxParts;
  return pick(D, dt, blocks_for(D, dt, p.T * p.G), [&](auto kernel, int nt, int smem) {
    kernel<<<grid, nt, smem, st>>>(p);
    return cudaGetLastError();
  });
}

}  // namespace rssm
