// Vectors of 16 bytes as fp32 values, the row and the place of a packed token, and
// the e4m3 values of quantised pages.
//
// A token's keys (or values) of one head are held as e4m3 values and a power of
// two: with a = max |x_i| over the finite ones, e is the least whole number with
// a <= 448 2^e (448 is the type's largest), kept within [-64, 63], and
//     code_i = e4m3(x_i 2^-e), rounded to nearest even;   x_i ~ code_i 2^e.
// Scaling by a power of two rounds nothing, so an element is rounded once, by
// half a step of e4m3 (2^-4 of it, or 2^-10 2^e below 2^(e - 6)); a scale of 23
// bits would gain nothing but the last part of a binade and cost three bytes.
// Infinities and NaN are kept as NaN; beyond 448 2^63 values saturate. The byte
// beside the values is e + 127: shifted by 23 it is 2^e in fp32.
#pragma once

#include <cuda_fp8.h>

#include "attn_core.cuh"
#include "kv_common.cuh"

namespace rssm {

template <typename T>
struct Vec16 {
  static constexpr int E = 16 / (int)sizeof(T);
  static __device__ __forceinline__ void unpack(const uint4& u, float* v) {
    const T* t = reinterpret_cast<const T*>(&u);
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = attn_f32(t[i]);
  }
  static __device__ __forceinline__ uint4 pack(const float* v) {
    uint4 u;
    uint32_t* w = reinterpret_cast<uint32_t*>(&u);
    if constexpr (std::is_same<T, float>::value) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(v[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = pack2<T>(v[2 * i], v[2 * i + 1]);
    }
    return u;
  }
};

constexpr int kScaleBias = 127;
constexpr int kScaleLeast = -64, kScaleMost = 63;

// e for the largest finite magnitude a >= 0
__device__ __forceinline__ int scale_exponent(float a) {
  const uint32_t u = __float_as_uint(a);
  // a = 1.m 2^(x - 127) <= 448 2^e = 1.75 2^(8 + e)
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u);
  return e < kScaleLeast ? kScaleLeast : e > kScaleMost ? kScaleMost : e;
}
__device__ __forceinline__ float power_of(int e) {  // 2^e, e in [-126, 127]
  return __uint_as_float((uint32_t)(e + 127) << 23);
}
// four values, e4m3 of x 2^-e (no infinities among x); beyond 448 2^e they saturate
__device__ __forceinline__ uint32_t e4m3x4(const float* x, float down) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[0] * down, x[1] * down),
                                               __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[2] * down, x[3] * down),
                                               __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}
// two e4m3 values as fp16, exactly
__device__ __forceinline__ __half2 e4m3x2_half2(uint32_t two) {
  const __half2_raw r =
      __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(two & 0xffffu), __NV_E4M3);
  return *reinterpret_cast<const __half2*>(&r);
}
__device__ __forceinline__ void e4m3x4_values(uint32_t four, float up, float* x) {
  const float2 a = __half22float2(e4m3x2_half2(four)), b = __half22float2(e4m3x2_half2(four >> 16));
  x[0] = a.x * up, x[1] = a.y * up, x[2] = b.x * up, x[3] = b.y * up;
}

// Row of packed token `tok`, and its place i in the row's window; false where it
// is outside every window or in one that is refused. cu null: T tokens a row.
__device__ __forceinline__ bool token_row(const int32_t* cu, int B, int T, int N, int tok, int& r,
                                          int& i) {
  if (cu == nullptr) {
    r = tok / T;
    i = tok - r * T;
    return true;
  }
  int lo = 0, hi = B;  // last row that begins at or before the token
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= tok) lo = mid; else hi = mid;
  }
  r = lo;
  const int first = cu[r], end = cu[r + 1];
  i = tok - first;
  return first >= 0 && tok >= first && tok < end && end <= N;
}

// The rows' offsets in shared memory where a CTA's threads can take one each: a
// search there costs no trips to memory. All threads; the barrier is the caller's.
template <int THREADS>
__device__ __forceinline__ const int32_t* copy_offsets(const int32_t* cu, int B, int32_t* room,
                                                       int tid) {
  if (cu == nullptr || B >= THREADS) return cu;
  if (tid <= B) room[tid] = cu[tid];
  return room;
}

struct TokenPlace {
  size_t off;             // bytes of its first head within the layer's pages
  int pos[kMaxRopeAxes];
  int live;
};

// Row, page and positions of token `tok`; token_bytes: of one head in the pages.
// cu: the call's offsets, or a copy of them.
__device__ __forceinline__ TokenPlace place_of(const AppendParams& p, const int32_t* cu, int tok,
                                               int token_bytes) {
  TokenPlace t{};
  int r, i;  // the token's row and place in its window
  if (!token_row(cu, p.B, p.T, p.N, tok, r, i)) return t;
  const int s = p.slot[r];
  // looked up beside the slot, not behind its page
  if (p.rope != nullptr && p.positions != nullptr) {
#pragma unroll
    for (int a = 0; a < kMaxRopeAxes; ++a) {
      if (a < p.axes) t.pos[a] = p.positions[(size_t)a * p.N + tok];
    }
  }
  if (s < 0) return t;
  uint32_t bad = 0;
  int len = 0;
  if (s >= p.n_slots) {
    bad = DEVERR_SLOT;
  } else {
    len = p.length[s];
    const int held = p.held[s];
    if (len < 0) {
      bad = DEVERR_CURSOR;
    } else if (held < 0 || held > p.max_pages || (long long)len + i >= ((long long)held << p.shift)) {
      bad = DEVERR_PAGES;
    }
  }
  int page = 0;
  if (bad == 0) {
    page = p.table[(size_t)s * p.max_pages + ((len + i) >> p.shift)];
    if (page < 0 || page >= p.n_pages) bad = DEVERR_PAGES;
  }
  if (p.rope != nullptr && bad == 0) {
#pragma unroll
    for (int a = 0; a < kMaxRopeAxes; ++a) {
      if (a >= p.axes || p.positions == nullptr) t.pos[a] = len + i;
      if (a < p.axes && (t.pos[a] < 0 || t.pos[a] >= p.max_pos)) bad = DEVERR_POSITION;
    }
  }
  if (bad) {
    atomicOr(p.err, bad);
    return t;
  }
  t.off = ((size_t)page * p.HKV << p.shift) * token_bytes +
          (size_t)((len + i) & ((1 << p.shift) - 1)) * token_bytes;
  t.live = 1;
  return t;
}

}  // namespace rssm
