// One warp's share of softmax attention over quantised pages: sixteen query
// rows against a chunk of e4m3 keys and values in shared memory, each key's and
// value's power of two beside them (kv_tokens.cuh).
//
//     x_ij = c 2^(a_i) 2^(e_j) (q'_i . k'_j)     q' = q 2^-a_i in fp16, k' the codes
//     p_ij = 2^(x_ij - m),   w_ij = 2^(f_j) p_ij
//     l    = sum_j p_ij;     o = sum_j w_ij v'_j;           output o / l
//
// e4m3 values are fp16 values, so a pair is one conversion and the products are
// those of fp16 on the tensor cores (m16n8k16), exact but for their fp32 sums. A
// row of q is scaled by a power of two so that its largest lies in [2^13, 2^14):
// bf16's eight bits and fp16's eleven pass whole, but for values under 2^-27 of
// the row's largest.
//
// The weights that the tensor cores read are w, with the value's power of two in
// them, because fp32 sums over keys cannot be scaled key by key afterwards. So
// that fp16 holds them whatever the powers are, the reference m follows w, not
// p: m = max_j (x_ij + f_j) - 14 and w <= 2^14; weights down to 2^-28 of the
// largest keep eleven bits, those below are off by 2^-39 of it. l sums p in fp32,
// p <= 2^(14 + 64). o and l refer to one m, so streams and parts join as those of
// other pages.
//
// Eight-bit matrices are loaded as if they were of 16-bit pairs. A lane's word of
// keys is then four neighbouring dimensions of one key, which serve as k = 2t,
// 2t + 1, 2t + 8, 2t + 9 of a product (q lies permuted to match); a word of
// values, transposed, is two dimensions of two neighbouring keys: one permutation
// of bytes parts it into the even and the odd dimension's pair. Of the outputs a
// lane holds dimensions 16 j + 4 t + {0, 2} in o[2 j] and {1, 3} in o[2 j + 1].
//
// Keys that a row must not see are left out by selection as in attn_core.cuh; the
// code NaN is looked for where other pages' infinities and NaN are.
#pragma once

#include "attn_core.cuh"
#include "kv_tokens.cuh"

namespace rssm {

constexpr float kWeightTop = 14.f;  // log2 of the largest weight

// Byte offset of 16-byte unit u of row r, e4m3 rows of D values in boxes of KR
// rows: columns of 128 bytes under the 128-byte swizzle, or rows of 64 under the
// 64-byte one.
template <int D, int KR>
__device__ __forceinline__ uint32_t code_off(int r, int u) {
  if constexpr (D == 64) {
    return (uint32_t)(r * 64 + (((u ^ (r >> 1)) & 3) << 4));
  } else {
    return (uint32_t)(r / KR) * (KR * D) + unit_off<KR>(r % KR, u);
  }
}

// Sixteen dimensions of q in place, from T to fp16 and permuted: words 0, 2, 4, 6
// then 1, 3, 5, 7 of the sixteen's eight.
__device__ __forceinline__ void permute_words(const uint32_t (&w)[8], uint4& lo, uint4& hi) {
  lo = make_uint4(w[0], w[2], w[4], w[6]);
  hi = make_uint4(w[1], w[3], w[5], w[7]);
}

// One row of q in shared memory (swizzled units of a block of ROWS rows), by D /
// 16 neighbouring lanes, `part` of them: scaled, permuted, in place. Returns 2^a.
template <typename T, int D, int ROWS>
__device__ __forceinline__ float scale_query(unsigned char* qs, int row, int part) {
  constexpr int L = D / 16;
  uint4* u0 = reinterpret_cast<uint4*>(qs + unit_off<ROWS>(row, 2 * part));
  uint4* u1 = reinterpret_cast<uint4*>(qs + unit_off<ROWS>(row, 2 * part + 1));
  float x[16];
  Vec16<T>::unpack(*u0, x);
  Vec16<T>::unpack(*u1, x + 8);
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float y = fabsf(x[i]);
    top = fmaxf(top, y < INFINITY ? y : 0.f);
  }
#pragma unroll
  for (int d = 1; d < L; d <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, d));
  // largest in [2^13, 2^14); a row of zeros (or of values under 2^-87) as it is
  int a = top > 0.f ? (int)(__float_as_uint(top) >> 23) - 127 - 13 : 0;
  a = a < -100 ? -100 : a;
  const float down = power_of(-a);
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = pack2<__half>(x[2 * i] * down, x[2 * i + 1] * down);
  permute_words(w, *u0, *u1);
  return power_of(a);
}

template <int D, int QR, int KR>
struct WarpAttnQuant {
  float o[1][D / 8][4];
  float m[1][2], l[1][2];  // l: this lane's share of the row's sum

  // dimension of value e of o[i] for rows g (e < 2) and g + 8, once ordered()
  static __device__ __forceinline__ int col(int i, int t) {
    return 16 * (i >> 1) + 4 * t + 2 * (i & 1);
  }

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
#pragma unroll
      for (int e = 0; e < 4; ++e) o[0][i][e] = 0.f;
    }
    m[0][0] = m[0][1] = kNegInf;
    l[0][0] = l[0][1] = 0.f;
  }

  // neighbouring dimensions side by side (and back)
  __device__ __forceinline__ void ordered() {
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float x = o[0][2 * j][2 * r + 1];
        o[0][2 * j][2 * r + 1] = o[0][2 * j + 1][2 * r];
        o[0][2 * j + 1][2 * r] = x;
      }
    }
  }

  // Weights w of a chunk of 8 NT keys, m, l and o brought to the new reference.
  // sc: the chunk's powers of two ([8 NT][2] bytes); rf: c 2^a of the lane's rows.
  template <int NT>
  __device__ __forceinline__ void weights(float (&x)[1][NT][4], const unsigned char* qs,
                                          const unsigned char* ks, const unsigned char* sc,
                                          int key0, const int (&lim)[1][2], int all,
                                          const float (&rf)[2], int lane) {
    static_assert(NT % 2 == 0, "keys in sixteens");
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[0][n][e] = 0.f;
    }
    const int i = lane >> 3, r = lane & 7, t = lane & 3;
    const uint32_t qb = smem_addr(qs), kb = smem_addr(ks);
#pragma unroll
    for (int u = 0; u < D / 16; u += 2) {
      uint32_t a[2][4];
#pragma unroll
      for (int s = 0; s < 2; ++s)
        ldsm4(a[s], qb + unit_off<QR>((i & 1) * 8 + r, 2 * (u + s) + (i >> 1)));
#pragma unroll
      for (int n = 0; n < NT / 2; ++n) {
        uint32_t kf[4];
        ldsm4(kf, kb + code_off<D, KR>(16 * n + (i >> 1) * 8 + r, u + (i & 1)));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const __half2 b0 = e4m3x2_half2(kf[2 * h + s]), b1 = e4m3x2_half2(kf[2 * h + s] >> 16);
            mma16<__half>(x[0][2 * n + h], a[s], *reinterpret_cast<const uint32_t*>(&b0),
                          *reinterpret_cast<const uint32_t*>(&b1));
          }
        }
      }
    }
    const bool masked = key0 + 8 * NT > all;
    float vs[NT][2];  // powers of two of the lane's values
    float top[2] = {kNegInf, kNegInf};
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(sc + 2 * (8 * n + 2 * t));
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t kb8 = (w >> (16 * e)) & 0xffu, vb8 = (w >> (16 * e + 8)) & 0xffu;
        const float kscale = __uint_as_float(kb8 << 23);
        const float f = (float)((int)vb8 - kScaleBias);
        vs[n][e] = __uint_as_float(vb8 << 23);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float y = x[0][n][2 * h + e] * rf[h] * kscale;
          if (masked && key0 + 8 * n + 2 * t + e >= lim[0][h]) y = kNegInf;
          x[0][n][2 * h + e] = y;
          top[h] = fmaxf(top[h], y + f);
        }
      }
    }
    float a[2], base[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      top[h] = fmaxf(top[h], __shfl_xor_sync(kFull, top[h], 1));
      top[h] = fmaxf(top[h], __shfl_xor_sync(kFull, top[h], 2));
      const float to = fmaxf(m[0][h], top[h] - kWeightTop);
      base[h] = to == kNegInf ? 0.f : to;
      a[h] = exp2_fast(m[0][h] - base[h]);
      m[0][h] = to;
      l[0][h] *= a[h];
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float p = exp2_fast(x[0][n][e] - base[e >> 1]);
        l[0][e >> 1] += p;
        // a key that is not seen has no weight, whatever its bytes hold
        x[0][n][e] = masked && p == 0.f ? 0.f : p * vs[n][e & 1];
      }
    }
    if (__any_sync(kFull, a[0] != 1.f || a[1] != 1.f)) {
#pragma unroll
      for (int j = 0; j < D / 8; ++j) {
#pragma unroll
        for (int e = 0; e < 4; ++e) o[0][j][e] *= a[e >> 1];
      }
    }
  }

  // the code NaN among the chunk's values (whole warp)
  template <int NT>
  static __device__ __forceinline__ bool any_nan(const unsigned char* vs, int lane) {
    constexpr int W = 8 * NT * D / 16;
    bool bad = false;
    for (int i = lane; i < W; i += 32) {
      const uint4 u = reinterpret_cast<const uint4*>(vs)[i];
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) bad |= __vcmpeq4(w[j] & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0;
    }
    return __any_sync(kFull, bad);
  }

  // o += w v
  template <int NT>
  __device__ __forceinline__ void add(const float (&w)[1][NT][4], const unsigned char* vs,
                                      int key0, const int (&lim)[1][2], int all, int lane) {
    if (key0 + 8 * NT > all && any_nan<NT>(vs, lane)) {
      add_selected<NT>(w, vs, key0, lim, lane);
      return;
    }
    const int i = lane >> 3, r = lane & 7;
    const uint32_t vb = smem_addr(vs);
#pragma unroll
    for (int n = 0; n < NT / 2; ++n) {
      uint32_t a[4];
      a[0] = pack2<__half>(w[0][2 * n][0], w[0][2 * n][1]);
      a[1] = pack2<__half>(w[0][2 * n][2], w[0][2 * n][3]);
      a[2] = pack2<__half>(w[0][2 * n + 1][0], w[0][2 * n + 1][1]);
      a[3] = pack2<__half>(w[0][2 * n + 1][2], w[0][2 * n + 1][3]);
#pragma unroll
      for (int u = 0; u < D / 16; u += 2) {
        uint32_t vf[4];  // keys 0-7 and 8-15 of unit u, of unit u + 1
        ldsm4_t(vf, vb + code_off<D, KR>(16 * n + (i & 1) * 8 + r, u + (i >> 1)));
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const uint32_t b0 = __byte_perm(vf[2 * s], 0, 0x3120);
          const uint32_t b1 = __byte_perm(vf[2 * s + 1], 0, 0x3120);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const __half2 h0 = e4m3x2_half2(b0 >> (16 * h)), h1 = e4m3x2_half2(b1 >> (16 * h));
            mma16<__half>(o[0][2 * (u + s) + h], a, *reinterpret_cast<const uint32_t*>(&h0),
                          *reinterpret_cast<const uint32_t*>(&h1));
          }
        }
      }
    }
  }

  // the same with the keys that a row does not see left out by selection
  template <int NT>
  __device__ __forceinline__ void add_selected(const float (&w)[1][NT][4], const unsigned char* vs,
                                            int key0, const int (&lim)[1][2], int lane) {
    const int t = lane & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll 1
      for (int j = 0; j < 8; ++j) {
        const int from = (lane & ~3) | (j >> 1), key = 8 * n + j;
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = __shfl_sync(kFull, w[0][n][e], from);
        const float p0 = (j & 1) ? y[1] : y[0], p1 = (j & 1) ? y[3] : y[2];
        const bool s0 = key0 + key < lim[0][0], s1 = key0 + key < lim[0][1];
#pragma unroll
        for (int d = 0; d < D / 16; ++d) {
          const uint32_t four =
              *reinterpret_cast<const uint32_t*>(vs + code_off<D, KR>(key, d) + 4 * t);
          float v[4];
          e4m3x4_values(four, 1.f, v);
          if (s0) {
            o[0][2 * d][0] = fmaf(p0, v[0], o[0][2 * d][0]);
            o[0][2 * d + 1][0] = fmaf(p0, v[1], o[0][2 * d + 1][0]);
            o[0][2 * d][1] = fmaf(p0, v[2], o[0][2 * d][1]);
            o[0][2 * d + 1][1] = fmaf(p0, v[3], o[0][2 * d + 1][1]);
          }
          if (s1) {
            o[0][2 * d][2] = fmaf(p1, v[0], o[0][2 * d][2]);
            o[0][2 * d + 1][2] = fmaf(p1, v[1], o[0][2 * d + 1][2]);
            o[0][2 * d][3] = fmaf(p1, v[2], o[0][2 * d][3]);
            o[0][2 * d + 1][3] = fmaf(p1, v[3], o[0][2 * d + 1][3]);
          }
        }
      }
    }
  }

  // sums of l over the row's lanes, outputs in order
  __device__ __forceinline__ void finish() {
    ordered();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[0][h] += __shfl_xor_sync(kFull, l[0][h], 1);
      l[0][h] += __shfl_xor_sync(kFull, l[0][h], 2);
    }
  }
};

}  // namespace rssm
