// The append with more in its pass: norms of queries and keys head by head before
// the rotation, pages quantised as they are written, keys and values in a row as
// the pages hold them.
//
//     n_i = x_i w_i / sqrt(mean_i x_i^2 + eps)       (queries, keys)
//     rotation as in kv_append.cu                    (queries, keys)
//     pages: n in the cache's type, or codes and a power of two (kv_tokens.cuh)
//
// All of it in fp32, rounded once. Every value is read once and written once, so
// HBM bounds it, if the arithmetic stays out of the way: a norm with quantisation
// is some 30 operations a value. A head belongs to D / 16 neighbouring lanes (D / 8
// of fp32), whose sums and maxima meet in shuffles. A group of lanes stays with a
// token: its cosines and sines are looked up once for all its heads, and the
// weights of queries, then of keys, lie in registers; products go in pairs of
// fp32. Where tokens are few, groups share out a token's heads. Loads of four
// heads are on their way at a time.
//
// Measured (GB300, in a graph): 14.2 k tokens, 16/4 heads of 256, norms, rotation of
// 64 dimensions, e4m3 pages: 73 us, 5.2 TB/s (77% of the copy rate); 2816 tokens,
// 32/8 heads of 128, three axes, bf16 pages: 19 us, 3.7 TB/s (one wave of CTAs that
// begin and end together); 56 single tokens 5.2 us, trips to memory. With a thread for
// a vector of a head, cosines looked up by each, 115 us; in pairs of fp32 110.
#include "attn_tc.cuh"
#include "kv_common.cuh"
#include "kv_tokens.cuh"

namespace rssm {

namespace {

constexpr int kNormThreads = 128;
constexpr int kNormCtas = 4;   // of an SM
constexpr int kNormAhead = 4;  // heads

// What a lane has of its group's token for all heads.
template <typename T, int D>
struct NormLane {
  static constexpr int E = Vec16<T>::E, P = E / 2;  // values of a vector, pairs
  static constexpr int IP = D / (2 * E);            // lanes of a head
  static_assert(IP >= 4 && IP <= 32, "a head in a warp");
  uint64_t cs[P], sn[P];
  int j;          // place in the head
  bool turn;      // its vectors turn into one another
  int v0, v1;     // places of its vectors of queries and keys
  unsigned mask;  // the head's lanes
};

enum : int { KIND_Q = 0, KIND_K = 1, KIND_V = 2 };

// Heads first, first + split, ... of n of one kind: from src to the row (contiguous
// heads, or null) and, but for queries, to the pages, a head head_bytes behind
// another; scale: the token's powers of two of the first head.
template <typename T, bool E4M3, int D, int KIND>
__device__ __forceinline__ void write_heads(const NormLane<T, D>& ln, const T* src, T* row,
                                            unsigned char* page, size_t head_bytes,
                                            unsigned char* scale, size_t head_scale, int first,
                                            int n, int split, const float* weight, float eps) {
  using V = Vec16<T>;
  using L = NormLane<T, D>;
  constexpr int E = L::E, P = L::P, IP = L::IP;
  const int at0 = KIND == KIND_V ? 2 * ln.j : ln.v0, at1 = KIND == KIND_V ? 2 * ln.j + 1 : ln.v1;
  uint64_t w[2 * P];
  if (KIND != KIND_V && weight != nullptr) {
#pragma unroll
    for (int e = 0; e < E; e += 4) {
      const float4 w0 = __ldg(reinterpret_cast<const float4*>(weight + at0 * E + e));
      const float4 w1 = __ldg(reinterpret_cast<const float4*>(weight + at1 * E + e));
      w[e / 2] = f2(w0.x, w0.y), w[e / 2 + 1] = f2(w0.z, w0.w);
      w[P + e / 2] = f2(w1.x, w1.y), w[P + e / 2 + 1] = f2(w1.z, w1.w);
    }
  }
  for (int h0 = first; h0 < n; h0 += split * kNormAhead) {
    uint4 a[kNormAhead], b[kNormAhead];
#pragma unroll
    for (int k = 0; k < kNormAhead; ++k) {
      const int h = h0 + k * split;
      if (h < n) {
        const uint4* x = reinterpret_cast<const uint4*>(src + (size_t)h * D);
        a[k] = __ldcs(x + at0);
        b[k] = __ldcs(x + at1);
      }
    }
#pragma unroll
    for (int k = 0; k < kNormAhead; ++k) {
      const int h = h0 + k * split;
      if (h >= n) break;
      uint4 ya = a[k], yb = b[k];
      if (KIND != KIND_V || E4M3) {
        float f[2 * E];
        V::unpack(a[k], f);
        V::unpack(b[k], f + E);
        if constexpr (KIND != KIND_V) {
          uint64_t x[2 * P];
#pragma unroll
          for (int e = 0; e < 2 * P; ++e) x[e] = f2(f[2 * e], f[2 * e + 1]);
          if (weight != nullptr) {
            uint64_t s2[2] = {0, 0};
#pragma unroll
            for (int e = 0; e < 2 * P; ++e) s2[e & 1] = fma2(x[e], x[e], s2[e & 1]);
            float sa, sb;
            un2(add2(s2[0], s2[1]), sa, sb);
            float ss = sa + sb;
#pragma unroll
            for (int d = 1; d < IP; d <<= 1) ss += __shfl_xor_sync(ln.mask, ss, d);
            float inv = __frsqrt_rn(fmaf(ss, 1.f / D, eps));
            if (!(ss <= 3.4028235e38f)) {
              // squares past fp32: the same of x 2^-70 (an infinity or NaN among x stays one)
              constexpr float kDown = 8.470329472543003e-22f;  // 2^-70
              ss = 0.f;
#pragma unroll
              for (int e = 0; e < 2 * E; ++e) ss = fmaf(f[e] * kDown, f[e] * kDown, ss);
#pragma unroll
              for (int d = 1; d < IP; d <<= 1) ss += __shfl_xor_sync(ln.mask, ss, d);
              inv = __frsqrt_rn(ss * (1.f / D)) * kDown;
            }
            const uint64_t inv2 = f2(inv, inv);
#pragma unroll
            for (int e = 0; e < 2 * P; ++e) x[e] = mul2(mul2(x[e], inv2), w[e]);
          }
          if (ln.turn) {
            const uint64_t minus = f2(-1.f, -1.f);
#pragma unroll
            for (int e = 0; e < P; ++e) {
              const uint64_t xa = x[e], xb = x[P + e];
              x[e] = fma2(xa, ln.cs[e], mul2(mul2(xb, minus), ln.sn[e]));
              x[P + e] = fma2(xb, ln.cs[e], mul2(xa, ln.sn[e]));
            }
          }
#pragma unroll
          for (int e = 0; e < 2 * P; ++e) un2(x[e], f[2 * e], f[2 * e + 1]);
        }
        if constexpr (E4M3 && KIND != KIND_Q) {
          float top = 0.f;
#pragma unroll
          for (int e = 0; e < 2 * E; ++e) top = fmaxf(top, fabsf(f[e]));  // NaN is left out
#pragma unroll
          for (int d = 1; d < IP; d <<= 1) top = fmaxf(top, __shfl_xor_sync(ln.mask, top, d));
          if (top == INFINITY) {  // infinities are kept as NaN, and count for nothing
            top = 0.f;
#pragma unroll
            for (int e = 0; e < 2 * E; ++e) {
              if (fabsf(f[e]) == INFINITY) f[e] = __uint_as_float(0x7fffffffu);
              top = fmaxf(top, fabsf(f[e]));
            }
#pragma unroll
            for (int d = 1; d < IP; d <<= 1) top = fmaxf(top, __shfl_xor_sync(ln.mask, top, d));
          }
          const int ex = scale_exponent(top);
          const float down = power_of(-ex);
          uint32_t c[2 * E / 4];
#pragma unroll
          for (int e = 0; e < 2 * E; e += 4) c[e / 4] = e4m3x4(f + e, down);
          unsigned char* to = page + h * head_bytes;
          constexpr int W = E / 4;  // words of a vector's codes
          if constexpr (W == 2) {
            reinterpret_cast<uint2*>(to)[at0] = make_uint2(c[0], c[1]);
            reinterpret_cast<uint2*>(to)[at1] = make_uint2(c[2], c[3]);
          } else {
            reinterpret_cast<uint32_t*>(to)[at0] = c[0];
            reinterpret_cast<uint32_t*>(to)[at1] = c[1];
          }
          if (ln.j == 0) scale[h * head_scale] = (unsigned char)(ex + kScaleBias);
          if (row != nullptr) {
            const float up = power_of(ex);
#pragma unroll
            for (int e = 0; e < 2 * E; e += 4) e4m3x4_values(c[e / 4], up, f + e);
          }
        }
        ya = V::pack(f);
        yb = V::pack(f + E);
      }
      if (!E4M3 && KIND != KIND_Q) {
        uint4* to = reinterpret_cast<uint4*>(page + h * head_bytes);
        to[at0] = ya;
        to[at1] = yb;
      }
      if (row != nullptr) {
        uint4* to = reinterpret_cast<uint4*>(row + (size_t)h * D);
        to[at0] = ya;
        to[at1] = yb;
      }
    }
  }
}

// split: groups that share out a token's heads, a power of two
template <typename T, bool E4M3, int D>
__global__ void __launch_bounds__(kNormThreads, kNormCtas)
    kv_append_norm_kernel(const __grid_constant__ AppendParams p, int split) {
  using L = NormLane<T, D>;
  constexpr int E = L::E, IP = L::IP;
  constexpr int GROUPS = kNormThreads / IP, TOKEN = D * (E4M3 ? 1 : (int)sizeof(T));
  __shared__ TokenPlace places[GROUPS];
  const int tid = threadIdx.x, tokens = GROUPS / split, tok0 = blockIdx.x * tokens;
  __shared__ int32_t offsets[kNormThreads];
  const int32_t* cu = copy_offsets<kNormThreads>(p.cu, p.B, offsets, tid);
  if (p.cu != nullptr) __syncthreads();
  if (tid < tokens && tok0 + tid < p.N) places[tid] = place_of(p, cu, tok0 + tid, TOKEN);
  if (p.cu != nullptr && blockIdx.x == 0) {
    for (int r = tid; r < p.B; r += kNormThreads) {
      if (p.cu[r] < 0 || p.cu[r + 1] < p.cu[r] || p.cu[r + 1] > p.N) atomicOr(p.err, DEVERR_SEQLEN);
    }
  }
  const int grp = tid / IP, part = grp % split, t = grp / split;
  const int np = p.P / E;  // vectors that turn, of each half
  L ln;
  ln.j = tid % IP;
  ln.turn = ln.j < np;
  ln.v0 = ln.turn ? ln.j : 2 * ln.j;
  ln.v1 = ln.turn ? ln.j + np : 2 * ln.j + 1;  // np + np + 2 (j - np) = 2 j
  ln.mask = IP == 32 ? kFull : ((1u << IP % 32) - 1u) << ((tid & 31) & ~(IP - 1));
  __syncthreads();
  const long long tok = tok0 + t;
  if (tok >= p.N || !places[t].live) return;  // a group's lanes together
  const size_t off = places[t].off;
  if (ln.turn) {
    auto axis_of = [&](int pair) {
      if (p.interleaved) {
        const int x = pair % p.axes;
        return pair < p.axes * p.sec[x] ? x : 0;
      }
      return pair < p.sec[0] ? 0 : pair < p.sec[0] + p.sec[1] ? 1 : 2;
    };
    const int first_axis = axis_of(ln.j * E);
    if (p.axes == 1 || (!p.interleaved && first_axis == axis_of(ln.j * E + E - 1))) {
      const float4* row = reinterpret_cast<const float4*>(
          p.rope + (size_t)places[t].pos[first_axis] * 2 * p.P + ln.j * E);
#pragma unroll
      for (int e = 0; e < E; e += 4) {
        const float4 c4 = __ldg(row + e / 4), s4 = __ldg(row + (p.P + e) / 4);
        ln.cs[e / 2] = f2(c4.x, c4.y), ln.cs[e / 2 + 1] = f2(c4.z, c4.w);
        ln.sn[e / 2] = f2(s4.x, s4.y), ln.sn[e / 2 + 1] = f2(s4.z, s4.w);
      }
    } else {
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        float c2[2], s2[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int pair = ln.j * E + e + k;
          const float* row = p.rope + (size_t)places[t].pos[axis_of(pair)] * 2 * p.P + pair;
          c2[k] = __ldg(row);
          s2[k] = __ldg(row + p.P);
        }
        ln.cs[e / 2] = f2(c2[0], c2[1]);
        ln.sn[e / 2] = f2(s2[0], s2[1]);
      }
    }
  }
  // the heads of all kinds are dealt out one after the other
  const int hq = p.q != nullptr ? p.HQ : 0;
  const size_t head_bytes = (size_t)TOKEN << p.shift, head_scale = (size_t)2 << p.shift;
  const size_t row = (size_t)tok * p.HKV * D;
  unsigned char* scale = E4M3 ? p.scales + 2 * (off / D) : nullptr;  // D bytes in the pages, two here
  if (hq > 0)
    write_heads<T, E4M3, D, KIND_Q>(ln, static_cast<const T*>(p.q) + tok * p.qs,
                                    static_cast<T*>(p.q_out) + (size_t)tok * hq * D, nullptr, 0,
                                    nullptr, 0, part, hq, split, p.q_weight, p.eps);
  write_heads<T, E4M3, D, KIND_K>(
      ln, static_cast<const T*>(p.k) + tok * p.ks,
      p.k_out != nullptr ? static_cast<T*>(p.k_out) + row : nullptr, p.kp + off, head_bytes, scale,
      head_scale, (part - hq) & (split - 1), p.HKV, split, p.k_weight, p.eps);
  write_heads<T, E4M3, D, KIND_V>(
      ln, static_cast<const T*>(p.v) + tok * p.vs,
      p.v_out != nullptr ? static_cast<T*>(p.v_out) + row : nullptr, p.vp + off, head_bytes,
      E4M3 ? scale + 1 : nullptr, head_scale, (part - hq - p.HKV) & (split - 1), p.HKV, split,
      nullptr, p.eps);
}

template <typename T, bool E4M3>
cudaError_t launch(const AppendParams& p, int split, int grid, cudaStream_t st) {
  if (p.D == 64) kv_append_norm_kernel<T, E4M3, 64><<<grid, kNormThreads, 0, st>>>(p, split);
  else if (p.D == 128) kv_append_norm_kernel<T, E4M3, 128><<<grid, kNormThreads, 0, st>>>(p, split);
  else kv_append_norm_kernel<T, E4M3, 256><<<grid, kNormThreads, 0, st>>>(p, split);
  return cudaGetLastError();
}

}  // namespace

cudaError_t kv_append_norm_launch(const AppendParams& p, cudaStream_t st) {
  const int ip = p.D * dtype_bytes(p.dt) / 32, groups = kNormThreads / ip;
  // groups share out a token's heads as long as the SMs take all CTAs at once
  int split = 1;
  while (2 * split <= groups && (long long)p.N * 2 * split <= (long long)kMaxSms * kNormCtas * groups)
    split *= 2;
  const int tokens = groups / split;
  const int grid = (p.N + tokens - 1) / tokens;
  if (p.dt == DT_F32) return launch<float, false>(p, split, grid, st);
  if (p.dt == DT_BF16)
    return p.scales != nullptr ? launch<__nv_bfloat16, true>(p, split, grid, st)
                               : launch<__nv_bfloat16, false>(p, split, grid, st);
  return p.scales != nullptr ? launch<__half, true>(p, split, grid, st)
                             : launch<__half, false>(p, split, grid, st);
}

}  // namespace rssm
