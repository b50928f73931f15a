// One warp's share of softmax attention: sixteen query rows (or several blocks
// of sixteen) against a chunk of keys and values in shared memory, with the
// running maximum and sum of the softmax in registers.
//
//     x_ij = c (q_i . k_j),  c = scale log2(e)      (base-2 exponent)
//     m'   = max(m, max_j x_ij);  a = 2^(m - m');  p_ij = 2^(x_ij - m')
//     l    = a l + sum_j p_ij;    o = a o + sum_j p_ij v_j;     output o / l
//
// Products of 16-bit types run on the warp-level tensor cores (m16n8k16), those
// of fp32 on the FMA units. The fragments of x are those of p's operand: a row's
// values never leave the registers of its four lanes. l adds the weights in fp32
// as they are; their product with v takes them rounded to the input type,
// because that is what the tensor cores read (relative error 2^-8 at most for
// bf16 and 2^-11 for fp16, independent from weight to weight, as the rounding of
// the output); fp32 rounds nothing.
//
// Blocks in shared memory are cut in columns of 128 bytes: row r of a column is
// 128 bytes after row r - 1, and within it 16-byte unit u lies at unit
// u ^ (r % 8), so that eight rows' same unit falls in eight different bank
// groups (ldmatrix and the fp32 loads below are free of conflicts). That is
// what a TMA box of 128 bytes by rows by columns writes under the 128-byte
// swizzle.
//
// A key that a row must not see is left out by selection: its x becomes -inf,
// so p = 0. That leaves 0 * v, which is not 0 where v is infinite or NaN
// (rejected drafts, another sequence's tokens). A chunk that some rows see only
// in part is therefore looked through for such values of v, and where there is
// one the chunk's products are taken by selection too (pv_select).
#pragma once

#include <cmath>
#include <type_traits>

#include <cuda.h>

#include "rssm_common.cuh"

namespace rssm {

constexpr float kNegInf = -INFINITY;

__device__ __forceinline__ float attn_f32(float x) { return x; }
__device__ __forceinline__ float attn_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float attn_f32(__half x) { return __half2float(x); }

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// 2^x (ex2.approx.ftz: 2 ulp; 0 at -inf)
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}

template <typename T>
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                      uint32_t b1);
template <>
__device__ __forceinline__ void mma16<__nv_bfloat16>(float (&c)[4], const uint32_t (&a)[4],
                                                     uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16<__half>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                              uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 16-byte async copy global -> shared; zeros where `live` is false (nothing is
// read then).
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(live ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Tiled TMA loads; the inner coordinate is a multiple of 16 bytes.
__device__ __forceinline__ void tma_load3(uint32_t dst, const CUtensorMap* map, int x, int y,
                                          int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, "
      "{%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
      : "memory");
}
// Test hook of the bounded waits: the barrier's phase waits for `bytes` more
// than its copies bring, so every wait on it runs out.
__device__ __forceinline__ void mbar_promise(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)),
               "r"(bytes)
               : "memory");
}
// Byte offset of 16-byte unit u of row r in a block of ROWS rows.
template <int ROWS>
__device__ __forceinline__ uint32_t unit_off(int r, int u) {
  return (uint32_t)((u >> 3) * (ROWS * 128) + r * 128 + (((u ^ r) & 7) << 4));
}
// MB blocks of 16 rows; QR, KR: rows of the query block and of a block of keys
// in shared memory (their columns' heights); a chunk is one block of keys or
// several on end.
template <typename T, int D, int MB, int QR, int KR>
struct WarpAttn {
  static constexpr bool F32 = std::is_same<T, float>::value;
  // lane (g, t) = (lane / 4, lane % 4): columns col(i, t), + 1 of rows g (first
  // two) and g + 8 of block b
  float o[MB][D / 8][4];
  float m[MB][2], l[MB][2];  // l: this lane's share of the row's sum

  // the fragment of the matrix instructions, or whole 16-byte units for fp32
  static __device__ __forceinline__ int col(int i, int t) {
    return F32 ? 16 * (i >> 1) + 4 * t + 2 * (i & 1) : 8 * i + 2 * t;
  }
  // 16-byte unit u of key r of a chunk
  static __device__ __forceinline__ uint32_t key_off(int r, int u) {
    return (uint32_t)(r / KR) * (KR * D * (uint32_t)sizeof(T)) + unit_off<KR>(r % KR, u);
  }
  static __device__ __forceinline__ float4 key4(const unsigned char* base, int r, int u) {
    return *reinterpret_cast<const float4*>(base + key_off(r, u));
  }
  template <int ROWS>
  static __device__ __forceinline__ float4 vec4(const unsigned char* base, int r, int u) {
    return *reinterpret_cast<const float4*>(base + unit_off<ROWS>(r, u));
  }

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int b = 0; b < MB; ++b) {
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
#pragma unroll
        for (int e = 0; e < 4; ++e) o[b][i][e] = 0.f;
      }
      m[b][0] = m[b][1] = kNegInf;
      l[b][0] = l[b][1] = 0.f;
    }
  }

  // x = q k over the chunk's 8 NT keys (row r of the chunk at ks)
  template <int NT>
  __device__ __forceinline__ void scores(float (&x)[MB][NT][4], const unsigned char* qs,
                                         const unsigned char* ks, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int b = 0; b < MB; ++b) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[b][n][e] = 0.f;
      }
    }
    if constexpr (F32) {
#pragma unroll 4
      for (int u = 0; u < D / 4; ++u) {
        float4 q[MB][2];
#pragma unroll
        for (int b = 0; b < MB; ++b) {
          q[b][0] = vec4<QR>(qs, 16 * b + g, u);
          q[b][1] = vec4<QR>(qs, 16 * b + g + 8, u);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float4 k = key4(ks, 8 * n + 2 * t + e, u);
#pragma unroll
            for (int b = 0; b < MB; ++b) {
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                float& y = x[b][n][2 * r + e];
                y = fmaf(q[b][r].x, k.x, y);
                y = fmaf(q[b][r].y, k.y, y);
                y = fmaf(q[b][r].z, k.z, y);
                y = fmaf(q[b][r].w, k.w, y);
              }
            }
          }
        }
      }
    } else {
      static_assert(NT % 2 == 0, "keys in sixteens");
      const int i = lane >> 3, r = lane & 7;
      const uint32_t qb = smem_addr(qs), kb = smem_addr(ks);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        uint32_t kf[NT / 2][4];
#pragma unroll
        for (int n = 0; n < NT / 2; ++n)
          ldsm4(kf[n], kb + key_off(16 * n + (i >> 1) * 8 + r, 2 * kk + (i & 1)));
#pragma unroll
        for (int b = 0; b < MB; ++b) {
          uint32_t a[4];
          ldsm4(a, qb + unit_off<QR>(16 * b + (i & 1) * 8 + r, 2 * kk + (i >> 1)));
#pragma unroll
          for (int n = 0; n < NT / 2; ++n) {
            mma16<T>(x[b][2 * n], a, kf[n][0], kf[n][1]);
            mma16<T>(x[b][2 * n + 1], a, kf[n][2], kf[n][3]);
          }
        }
      }
    }
  }

  // o += p v on the tensor cores
  template <int NT>
  __device__ __forceinline__ void pv(const float (&p)[MB][NT][4], const unsigned char* vs,
                                     int lane) {
    if constexpr (F32) {
      const int t = lane & 3;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int from = (lane & ~3) | (j >> 1);
          float w[MB][2];
#pragma unroll
          for (int b = 0; b < MB; ++b) {
            w[b][0] = __shfl_sync(kFull, p[b][n][j & 1], from);
            w[b][1] = __shfl_sync(kFull, p[b][n][2 + (j & 1)], from);
          }
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            const float4 v = key4(vs, 8 * n + j, 4 * i + t);
#pragma unroll
            for (int b = 0; b < MB; ++b) {
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                float* y0 = &o[b][2 * i][2 * r];
                float* y1 = &o[b][2 * i + 1][2 * r];
                y0[0] = fmaf(w[b][r], v.x, y0[0]);
                y0[1] = fmaf(w[b][r], v.y, y0[1]);
                y1[0] = fmaf(w[b][r], v.z, y1[0]);
                y1[1] = fmaf(w[b][r], v.w, y1[1]);
              }
            }
          }
        }
      }
    } else {
      const int i = lane >> 3, r = lane & 7;
      const uint32_t vb = smem_addr(vs);
#pragma unroll
      for (int n = 0; n < NT / 2; ++n) {
        uint32_t a[MB][4];
#pragma unroll
        for (int b = 0; b < MB; ++b) {
          a[b][0] = pack2<T>(p[b][2 * n][0], p[b][2 * n][1]);
          a[b][1] = pack2<T>(p[b][2 * n][2], p[b][2 * n][3]);
          a[b][2] = pack2<T>(p[b][2 * n + 1][0], p[b][2 * n + 1][1]);
          a[b][3] = pack2<T>(p[b][2 * n + 1][2], p[b][2 * n + 1][3]);
        }
#pragma unroll
        for (int d = 0; d < D / 16; ++d) {
          uint32_t vf[4];
          ldsm4_t(vf, vb + key_off(16 * n + (i & 1) * 8 + r, 2 * d + (i >> 1)));
#pragma unroll
          for (int b = 0; b < MB; ++b) {
            mma16<T>(o[b][2 * d], a[b], vf[0], vf[1]);
            mma16<T>(o[b][2 * d + 1], a[b], vf[2], vf[3]);
          }
        }
      }
    }
  }

  // o += p v with the keys that a row does not see left out by selection;
  // fetch(key, d): values d, d + 1 of a key of the chunk
  template <int NT, typename F>
  __device__ __forceinline__ void pv_select(const float (&p)[MB][NT][4], F fetch, int key0,
                                            const int (&lim)[MB][2], int lane) {
    const int t = lane & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll 1
      for (int j = 0; j < 8; ++j) {
        const int from = (lane & ~3) | (j >> 1), key = 8 * n + j;
#pragma unroll
        for (int b = 0; b < MB; ++b) {
          // both of the holder's two, then one of them: an index that is not
          // known when compiling would put p into local memory for every use
          float w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = __shfl_sync(kFull, p[b][n][e], from);
          const float p0 = (j & 1) ? w[1] : w[0], p1 = (j & 1) ? w[3] : w[2];
          const bool s0 = key0 + key < lim[b][0], s1 = key0 + key < lim[b][1];
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            const float2 v = fetch(key, col(i, t));
            const float v0 = v.x, v1 = v.y;
            if (s0) o[b][i][0] = fmaf(p0, v0, o[b][i][0]), o[b][i][1] = fmaf(p0, v1, o[b][i][1]);
            if (s1) o[b][i][2] = fmaf(p1, v0, o[b][i][2]), o[b][i][3] = fmaf(p1, v1, o[b][i][3]);
          }
        }
      }
    }
  }

  // any infinite or NaN value in the chunk's 8 NT rows (whole warp)
  template <int NT>
  static __device__ __forceinline__ bool any_unfinite(const unsigned char* vs, int lane) {
    constexpr int W = 8 * NT * D * (int)sizeof(T) / 16;
    constexpr uint32_t E = F32                                     ? 0x7f800000u
                           : std::is_same<T, __half>::value ? 0x7c007c00u
                                                                   : 0x7f807f80u;
    bool bad = false;
    for (int i = lane; i < W; i += 32) {
      const uint4 u = reinterpret_cast<const uint4*>(vs)[i];
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (F32) {
          bad |= (w[j] & E) == E;
        } else {
          bad |= (w[j] & E & 0xffffu) == (E & 0xffffu) || (w[j] & (E & 0xffff0000u)) == (E & 0xffff0000u);
        }
      }
    }
    return __any_sync(kFull, bad);
  }

  // One chunk of 8 NT keys, the first of them key0: the weights p of the chunk,
  // with m, l and o brought to the new maximum. lim: how many keys the lane's
  // two rows of each block see; all: the fewest any row of the warp sees.
  template <int NT>
  __device__ __forceinline__ void weights(float (&x)[MB][NT][4], const unsigned char* qs,
                                          const unsigned char* ks, int key0,
                                          const int (&lim)[MB][2], int all, float c, int lane) {
    scores<NT>(x, qs, ks, lane);
    soften<NT>(x, key0, lim, all, c, lane);
  }

  // x: scores in, weights out
  template <int NT>
  __device__ __forceinline__ void soften(float (&x)[MB][NT][4], int key0,
                                         const int (&lim)[MB][2], int all, float c, int lane) {
    const int t = lane & 3;
    const bool masked = key0 + 8 * NT > all;
#pragma unroll
    for (int b = 0; b < MB; ++b) {
      float mx[2] = {m[b][0], m[b][1]};
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float y = x[b][n][e] * c;
          if (masked && key0 + 8 * n + 2 * t + (e & 1) >= lim[b][e >> 1]) y = kNegInf;
          x[b][n][e] = y;
          mx[e >> 1] = fmaxf(mx[e >> 1], y);
        }
      }
      float a[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        mx[h] = fmaxf(mx[h], __shfl_xor_sync(kFull, mx[h], 1));
        mx[h] = fmaxf(mx[h], __shfl_xor_sync(kFull, mx[h], 2));
        const float base = mx[h] == kNegInf ? 0.f : mx[h];
        a[h] = exp2_fast(m[b][h] - base);
        m[b][h] = mx[h];
        l[b][h] *= a[h];
        mx[h] = base;
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[b][n][e] = exp2_fast(x[b][n][e] - mx[e >> 1]);
          l[b][e >> 1] += x[b][n][e];
        }
      }
      if (__any_sync(kFull, a[0] != 1.f || a[1] != 1.f)) {
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
#pragma unroll
          for (int e = 0; e < 4; ++e) o[b][i][e] *= a[e >> 1];
        }
      }
    }
  }

  // o += p v
  template <int NT>
  __device__ __forceinline__ void add(const float (&p)[MB][NT][4], const unsigned char* vs,
                                      int key0, const int (&lim)[MB][2], int all, int lane) {
    static_assert(8 * NT % KR == 0, "whole blocks of keys");
    if (key0 + 8 * NT > all && any_unfinite<NT>(vs, lane)) {
      pv_select<NT>(
          p,
          [&](int key, int d) {
            constexpr int E = 16 / (int)sizeof(T);  // d is even: two values of one unit
            const T* v = reinterpret_cast<const T*>(vs + key_off(key, d / E)) + d % E;
            return make_float2(attn_f32(v[0]), attn_f32(v[1]));
          },
          key0, lim, lane);
    } else {
      pv<NT>(p, vs, lane);
    }
  }

  // sums of l over the row's lanes
  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int b = 0; b < MB; ++b) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        l[b][h] += __shfl_xor_sync(kFull, l[b][h], 1);
        l[b][h] += __shfl_xor_sync(kFull, l[b][h], 2);
      }
    }
  }
};

// Two neighbouring values as the output type
template <typename T>
__device__ __forceinline__ void store2(T* p, float a, float b) {
  if constexpr (std::is_same<T, float>::value) {
    *reinterpret_cast<float2*>(p) = make_float2(a, b);
  } else {
    *reinterpret_cast<uint32_t*>(p) = pack2<T>(a, b);
  }
}

// ln of the row's sum of exponentials, from base-2 statistics
__device__ __forceinline__ float lse_of(float m, float l) {
  return (m + log2f(l)) * 0.69314718055994531f;
}

}  // namespace rssm
