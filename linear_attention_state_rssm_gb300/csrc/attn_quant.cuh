// One warp's share of softmax attention over quantised pages: 8 NQ query rows
// against a chunk of e4m3 keys and values in shared memory, each key's and
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
// other pages; but where two references lie more than 2^126 apart (values of zeros, f =
// -64, beside ones of 2^71), l is brought over in two steps.
//
// The products are transposed, S' = K q' and O' = V' P': the sixteen rows of an
// instruction are keys, or dimensions, all of them of use, and its eight columns
// queries, of which a single token has few. A code is converted once whatever
// the number of queries is. (With queries as the rows, sixteen for four in use,
// 56 rows of 1 to 8 k tokens, 16/4 heads of 256, took 100 us; so 78.)
//
// Eight-bit matrices are loaded as if they were of 16-bit pairs. A lane's word of
// keys is then four neighbouring dimensions of one key, which serve as k = 2t,
// 2t + 1, 2t + 8, 2t + 9 of a product (q lies permuted to match); a word of
// values, transposed, is two dimensions of two neighbouring keys: one permutation
// of bytes parts it into the even and the odd dimension's pair, rows g and g + 8
// of the instruction. Weights come out as [key][query] and go in as [query][key]
// by way of movmatrix.
//
// Keys that a row must not see are left out by selection as in attn_core.cuh; the
// code NaN is looked for where other pages' infinities and NaN are.
#pragma once

#include "attn_core.cuh"
#include "kv_tokens.cuh"

namespace rssm {

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

// a for a row whose largest is `top`: 2^-a brings that into [2^13, 2^14) (a row of
// zeros stays as it is, one of values under 2^-87 smaller).
__device__ __forceinline__ int query_exponent(float top) {
  const int a = top > 0.f ? (int)(__float_as_uint(top) >> 23) - 127 - 13 : 0;
  return a < -100 ? -100 : a;
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
  const int a = query_exponent(top);
  const float down = power_of(-a);
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = pack2<__half>(x[2 * i] * down, x[2 * i + 1] * down);
  permute_words(w, *u0, *u1);
  return power_of(a);
}

// The transpose of an 8x8 matrix of 16-bit values (rows by lanes' fours).
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <int D, int NQ, int QR, int KR>
struct WarpAttnQuant {
  // lane (g, t): columns 2t, 2t + 1 of queries 8 n + .., rows g and g + 8 of o[j],
  // which are dimensions 16 j + 2 g and 16 j + 2 g + 1
  float o[D / 16][NQ][4];
  float m[2 * NQ], l[2 * NQ];  // l: this lane's share of the row's sum

  // ---- a lane's rows and pairs of dimensions (as WarpAttn has them)
  static constexpr int RL = 2 * NQ, PAIRS = D / 16, WROWS = 8 * NQ;
  static __device__ __forceinline__ int row(int e, int lane) {
    return 8 * (e >> 1) + 2 * (lane & 3) + (e & 1);
  }
  static __device__ __forceinline__ int dim(int i, int lane) { return 16 * i + 2 * (lane >> 2); }
  static __device__ __forceinline__ bool tells(int lane) { return lane < 4; }
  __device__ __forceinline__ float2 pair(int i, int e) const {
    return make_float2(o[i][e >> 1][e & 1], o[i][e >> 1][2 + (e & 1)]);
  }
  __device__ __forceinline__ void set_pair(int i, int e, float2 y) {
    o[i][e >> 1][e & 1] = y.x;
    o[i][e >> 1][2 + (e & 1)] = y.y;
  }
  __device__ __forceinline__ float& top(int e) { return m[e]; }
  __device__ __forceinline__ float& sum(int e) { return l[e]; }

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][n][e] = 0.f;
      }
    }
#pragma unroll
    for (int e = 0; e < RL; ++e) m[e] = kNegInf, l[e] = 0.f;
  }

  // Address of the lane's row of a chunk's first sixteen and its unit of the first two,
  // and of sixteen n and unit u on: units differ in bits that the swizzle has for
  // itself, so one register and an exclusive or serve a whole chunk. (With addresses of
  // their own kept in registers, windows of 32 query rows spilled.)
  static __device__ __forceinline__ uint32_t codes_of(const unsigned char* xs, int lane) {
    return smem_addr(xs) + code_off<D, KR>((lane >> 3 & 1) * 8 + (lane & 7), lane >> 4);
  }
  static __device__ __forceinline__ uint32_t code_at(uint32_t base, int n, int u) {
    return (base ^ (u % 8) << 4) + u / 8 * (KR * 128) + n * (16 * (D < 128 ? D : 128));
  }

  // Weights w of a chunk of 16 NT keys (x[.][.][2 h + e]: key 16 n + 8 h + g, row e
  // of the lane's pair), m, l and o brought to the new reference. sc: the chunk's
  // powers of two ([16 NT][2] bytes); rf: c 2^a of the lane's rows.
  template <int NT>
  __device__ __forceinline__ void weights(float (&x)[NT][NQ][4], const unsigned char* qs,
                                          const unsigned char* ks, const unsigned char* sc,
                                          int key0, const int (&lim)[RL], int all,
                                          const float (&rf)[RL], int lane) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[n][q][e] = 0.f;
      }
    }
    const int i = lane >> 3, r = lane & 7, g = lane >> 2;
    const uint32_t qb = smem_addr(qs) + unit_off<QR>(r, i), kb = codes_of(ks, lane);
#pragma unroll
    for (int u = 0; u < D / 16; u += 2) {
      uint32_t b[NQ][4];  // k-steps u and u + 1
#pragma unroll
      for (int q = 0; q < NQ; ++q)
        ldsm4(b[q], (qb ^ (2 * u % 8) << 4) + 2 * u / 8 * QR * 128 + q * 1024);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        uint32_t kf[4];  // keys 0-7 and 8-15 of unit u, of unit u + 1
        ldsm4(kf, code_at(kb, n, u));
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          uint32_t a[4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const __half2 lo = e4m3x2_half2(kf[2 * s + h]), hi = e4m3x2_half2(kf[2 * s + h] >> 16);
            a[h] = *reinterpret_cast<const uint32_t*>(&lo);
            a[2 + h] = *reinterpret_cast<const uint32_t*>(&hi);
          }
#pragma unroll
          for (int q = 0; q < NQ; ++q) mma16<__half>(x[n][q], a, b[q][2 * s], b[q][2 * s + 1]);
        }
      }
    }
    const bool masked = key0 + 16 * NT > all;
    float vs[NT][2];  // powers of two of the lane's values
    float top[RL];
#pragma unroll
    for (int e = 0; e < RL; ++e) top[e] = kNegInf;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int key = 16 * n + 8 * h + g;
        const uint32_t w = *reinterpret_cast<const uint16_t*>(sc + 2 * key);
        const float kscale = __uint_as_float((w & 0xffu) << 23);
        const float f = (float)((int)(w >> 8) - kScaleBias);
        vs[n][h] = __uint_as_float((w >> 8) << 23);
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            // in this order: rf kscale may pass fp32's range where the score does not
            float& y = x[n][q][2 * h + e];
            y = y * kscale * rf[2 * q + e];
          }
        }
        if (masked) {
#pragma unroll
          for (int e = 0; e < RL; ++e) {
            if (key0 + key >= lim[e]) x[n][e >> 1][2 * h + (e & 1)] = kNegInf;
          }
        }
#pragma unroll
        for (int e = 0; e < RL; ++e)
          top[e] = fmaxf(top[e], x[n][e >> 1][2 * h + (e & 1)] + f);
      }
    }
    float base[RL];
    bool moved = false;
    float a[RL];
#pragma unroll
    for (int e = 0; e < RL; ++e) {
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) top[e] = fmaxf(top[e], __shfl_xor_sync(kFull, top[e], d));
      const float to = fmaxf(m[e], top[e] - kWeightTop);
      base[e] = to == kNegInf ? 0.f : to;
      // in two halves: l, up to 2^78 a key, counts where a alone is below fp32's range
      const float half = exp2_fast(0.5f * (m[e] - base[e]));
      a[e] = half * half;
      moved |= a[e] != 1.f;
      m[e] = to;
      l[e] = l[e] * half * half;
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float p = exp2_fast(x[n][q][e] - base[2 * q + (e & 1)]);
          l[2 * q + (e & 1)] += p;
          x[n][q][e] = p * vs[n][e >> 1];
        }
      }
    }
    if (masked) {  // a key that is not seen has no weight, whatever its bytes hold
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int e = 0; e < RL; ++e) {
            if (key0 + 16 * n + 8 * h + g >= lim[e]) x[n][e >> 1][2 * h + (e & 1)] = 0.f;
          }
        }
      }
    }
    if (__any_sync(kFull, moved)) {
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
#pragma unroll
          for (int e = 0; e < 4; ++e) o[j][q][e] *= a[2 * q + (e & 1)];
        }
      }
    }
  }

  // the code NaN among the chunk's values (whole warp)
  template <int NT>
  static __device__ __forceinline__ bool any_nan(const unsigned char* vs, int lane) {
    constexpr int W = 16 * NT * D / 16;
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
  __device__ __forceinline__ void add(const float (&w)[NT][NQ][4], const unsigned char* vs,
                                      int key0, const int (&lim)[RL], int all, int lane) {
    if (key0 + 16 * NT > all && any_nan<NT>(vs, lane)) {
      add_selected<NT>(w, vs, key0, lim, lane);
      return;
    }
    const uint32_t vb = codes_of(vs, lane);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      uint32_t b[NQ][2];
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        b[q][0] = movmatrix(pack2<__half>(w[n][q][0], w[n][q][1]));
        b[q][1] = movmatrix(pack2<__half>(w[n][q][2], w[n][q][3]));
      }
#pragma unroll
      for (int u = 0; u < D / 16; u += 2) {
        uint32_t vf[4];  // keys 0-7 and 8-15 of unit u, of unit u + 1
        ldsm4_t(vf, code_at(vb, n, u));
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          uint32_t a[4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t y = __byte_perm(vf[2 * s + h], 0, 0x3120);
            const __half2 even = e4m3x2_half2(y), odd = e4m3x2_half2(y >> 16);
            a[2 * h] = *reinterpret_cast<const uint32_t*>(&even);
            a[2 * h + 1] = *reinterpret_cast<const uint32_t*>(&odd);
          }
#pragma unroll
          for (int q = 0; q < NQ; ++q) mma16<__half>(o[u + s][q], a, b[q][0], b[q][1]);
        }
      }
    }
  }

  // the same with the keys that a row does not see left out by selection
  template <int NT>
  __device__ __forceinline__ void add_selected(const float (&w)[NT][NQ][4],
                                               const unsigned char* vs, int key0,
                                               const int (&lim)[RL], int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll 1
      for (int j = 0; j < 16; ++j) {
        const int key = 16 * n + j, from = (j & 7) * 4 + t;
        float p[RL];
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
          // both halves' values, then one of them (an index that is not known when
          // compiling would put w into local memory for every use)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float lo = __shfl_sync(kFull, w[n][q][e], from);
            const float hi = __shfl_sync(kFull, w[n][q][2 + e], from);
            p[2 * q + e] = j < 8 ? lo : hi;
          }
        }
#pragma unroll
        for (int d = 0; d < D / 16; ++d) {
          const uint32_t two =
              *reinterpret_cast<const uint16_t*>(vs + code_off<D, KR>(key, d) + 2 * g);
          const float2 v = __half22float2(e4m3x2_half2(two));
#pragma unroll
          for (int e = 0; e < RL; ++e) {
            if (key0 + key < lim[e]) {
              float* y = o[d][e >> 1];
              y[e & 1] = fmaf(p[e], v.x, y[e & 1]);
              y[2 + (e & 1)] = fmaf(p[e], v.y, y[2 + (e & 1)]);
            }
          }
        }
      }
    }
  }

  // sums of l over the row's lanes
  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int e = 0; e < RL; ++e) {
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) l[e] += __shfl_xor_sync(kFull, l[e], d);
    }
  }
};

}  // namespace rssm
