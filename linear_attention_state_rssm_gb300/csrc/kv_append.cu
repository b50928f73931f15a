// New tokens of one layer: rotary positions on q and k, and the append of k
// and v to the slots' pages, in one pass over the projection's output.
//
//     pair i < P of a head:  y_i     = x_i cos a - x_{i+P} sin a
//                            y_{i+P} = x_{i+P} cos a + x_i sin a,
//     a = position[axis(i)] * frequency_i (cosines and sines from a table);
//     dimensions from 2 P on, and v, are copied.
// With several axes (time, height, width) each pair turns by the position of
// its own axis. Angles are looked up, not computed: a position times a
// frequency in fp32 is off by 2^-24 of the angle, 0.06 rad at position 10^6.
//
// Every value is read once and written once: HBM-bound. A token's row, slot,
// length, page and positions are trips to memory one behind the other, so a CTA
// takes up to eight tokens and looks them up side by side, one thread each; a
// thread then keeps its pairs' cosines and sines in registers over the heads it
// serves and has the loads of two heads on their way at a time. 16168 tokens of
// 32/8 heads of 128, positions of three axes: 75 us, 80% of the copy rate (four
// heads at a time and four warps 78 us; one token to a CTA 89 us).
#include "kv_common.cuh"
#include "kv_tokens.cuh"

namespace rssm {

namespace {

constexpr int kAppendThreads = 192;
constexpr int kHeadsAhead = 2;

constexpr int kMaxTokens = 8;  // of a CTA

struct TokenPlace {
  size_t off;             // bytes of its first head within the layer's pages
  int pos[kMaxRopeAxes];
  int live;
};

// Row, page and positions of token `tok`; token_bytes: of one head in the pages.
__device__ __forceinline__ TokenPlace place_of(const AppendParams& p, int tok, int token_bytes) {
  TokenPlace t{};
  int r, i;  // the token's row and place in its window
  if (!token_row(p.cu, p.B, p.T, p.N, tok, r, i)) return t;
  const int s = p.slot[r];
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
      t.pos[a] = len + i;
      if (p.positions != nullptr && a < p.axes) t.pos[a] = p.positions[(size_t)a * p.N + tok];
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

// One head of one token, two vectors of it a lane (a and b; the ip lanes of the
// head are head_lanes): norm, rotation, and the stores.
template <typename T, bool E4M3>
__device__ __forceinline__ void write_head(const AppendParams& p, long long tok, int h, int hq,
                                           size_t off, size_t head_bytes, const uint4& a,
                                           const uint4& b, int v0, int v1, int j, int ip,
                                           bool turn, const float* cs, const float* sn,
                                           unsigned head_lanes) {
  using V = Vec16<T>;
  constexpr int E = V::E;
  const bool query = h < hq, val = h >= hq + p.HKV;
  const int at0 = val ? 2 * j : v0, at1 = val ? 2 * j + 1 : v1;  // the vectors' places
  float x[2 * E];
  V::unpack(a, x);
  V::unpack(b, x + E);
  const float* w = query ? p.q_weight : val ? nullptr : p.k_weight;
  if (w != nullptr) {
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 2 * E; ++e) ss = fmaf(x[e], x[e], ss);
    for (int d = 1; d < ip; d <<= 1) ss += __shfl_xor_sync(head_lanes, ss, d);
    float inv = __frsqrt_rn(ss / (float)p.D + p.eps);
    if (!(ss <= 3.4028235e38f)) {
      // squares past fp32: the same of x 2^-70 (an infinity or NaN among x stays one)
      constexpr float kDown = 8.470329472543003e-22f;  // 2^-70
      ss = 0.f;
#pragma unroll
      for (int e = 0; e < 2 * E; ++e) ss = fmaf(x[e] * kDown, x[e] * kDown, ss);
      for (int d = 1; d < ip; d <<= 1) ss += __shfl_xor_sync(head_lanes, ss, d);
      inv = __frsqrt_rn(ss / (float)p.D) * kDown;
    }
#pragma unroll
    for (int e = 0; e < E; e += 4) {
      const float4 w0 = __ldg(reinterpret_cast<const float4*>(w + at0 * E + e));
      const float4 w1 = __ldg(reinterpret_cast<const float4*>(w + at1 * E + e));
      const float wa[4] = {w0.x, w0.y, w0.z, w0.w}, wb[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[e + i] = x[e + i] * inv * wa[i];
        x[E + e + i] = x[E + e + i] * inv * wb[i];
      }
    }
  }
  if (turn && !val) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float xa = x[e], xb = x[E + e];
      x[e] = fmaf(xa, cs[e], -xb * sn[e]);
      x[E + e] = fmaf(xb, cs[e], xa * sn[e]);
    }
  }
  const int kvh = val ? h - hq - p.HKV : h - hq;  // of keys and values
  if constexpr (E4M3) {
    if (!query) {
      float top = 0.f;
#pragma unroll
      for (int e = 0; e < 2 * E; ++e) {
        const float y = fabsf(x[e]);
        top = fmaxf(top, y < INFINITY ? y : 0.f);
      }
      for (int d = 1; d < ip; d <<= 1) top = fmaxf(top, __shfl_xor_sync(head_lanes, top, d));
      const int ex = scale_exponent(top);
      const float down = power_of(-ex), up = power_of(ex);
      uint32_t c[2 * E / 4];
#pragma unroll
      for (int e = 0; e < 2 * E; e += 4) c[e / 4] = e4m3x4(x + e, down);
      unsigned char* to = (val ? p.vp : p.kp) + off + kvh * head_bytes;
      constexpr int W = E / 4;  // words of a vector's codes
      static_assert(W == 1 || W == 2, "four or eight values a vector");
      if constexpr (W == 2) {
        reinterpret_cast<uint2*>(to)[at0] = make_uint2(c[0], c[1]);
        reinterpret_cast<uint2*>(to)[at1] = make_uint2(c[2], c[3]);
      } else {
        reinterpret_cast<uint32_t*>(to)[at0] = c[0];
        reinterpret_cast<uint32_t*>(to)[at1] = c[1];
      }
      if (j == 0)  // a token and head has D bytes in the pages and two here
        p.scales[2 * ((off + kvh * head_bytes) / (size_t)p.D) + (val ? 1 : 0)] =
            (unsigned char)(ex + kScaleBias);
#pragma unroll
      for (int e = 0; e < 2 * E; e += 4) e4m3x4_values(c[e / 4], up, x + e);
    }
  }
  const uint4 ya = V::pack(x), yb = V::pack(x + E);
  if (!E4M3 || query) {
    uint4* to = query ? reinterpret_cast<uint4*>(static_cast<T*>(p.q_out) +
                                                 ((size_t)tok * p.HQ + h) * p.D)
                      : reinterpret_cast<uint4*>((val ? p.vp : p.kp) + off + kvh * head_bytes);
    to[at0] = ya;
    to[at1] = yb;
  }
  void* row = query ? nullptr : val ? p.v_out : p.k_out;
  if (row != nullptr) {
    uint4* to = reinterpret_cast<uint4*>(static_cast<T*>(row) +
                                         ((size_t)tok * p.HKV + kvh) * p.D);
    to[at0] = ya;
    to[at1] = yb;
  }
}

// MORE: norms of q and k, values in a row; E4M3: quantised pages (and MORE).
template <typename T, bool MORE, bool E4M3>
__global__ void __launch_bounds__(kAppendThreads, MORE ? 4 : 5)
    kv_append_kernel(const __grid_constant__ AppendParams p, int tokens) {
  using V = Vec16<T>;
  constexpr int E = V::E;
  __shared__ TokenPlace places[kMaxTokens];
  const int tok0 = blockIdx.x * tokens, tid = threadIdx.x;
  const int token_bytes = p.D * (E4M3 ? 1 : (int)sizeof(T));  // of one head
  if (tid < tokens && tok0 + tid < p.N) places[tid] = place_of(p, tok0 + tid, token_bytes);
  if (p.cu != nullptr && blockIdx.x == 0) {
    for (int r = tid; r < p.B; r += kAppendThreads) {
      if (p.cu[r] < 0 || p.cu[r + 1] < p.cu[r] || p.cu[r + 1] > p.N) atomicOr(p.err, DEVERR_SEQLEN);
    }
  }
  const int ip = p.D / (2 * E);  // items of a head: two vectors each
  const int np = p.P / E;        // of which turned
  const int j = tid % ip, y0 = tid / ip, ny = kAppendThreads / ip;
  const bool turn = j < np;
  const int v0 = turn ? j : 2 * j, v1 = turn ? j + np : 2 * j + 1;  // np + np + 2 (j - np) = 2 j
  const int hq = p.q != nullptr ? p.HQ : 0, heads = hq + 2 * p.HKV;
  const size_t head_bytes = (size_t)token_bytes << p.shift;
  auto axis_of = [&](int pair) {
    if (p.interleaved) {
      const int x = pair % p.axes;
      return pair < p.axes * p.sec[x] ? x : 0;
    }
    return pair < p.sec[0] ? 0 : pair < p.sec[0] + p.sec[1] ? 1 : 2;
  };
  // the lanes of a head: ip is a power of two, at most 32
  const unsigned head_lanes =
      ip >= 32 ? kFull : ((1u << ip) - 1u) << ((tid & 31) & ~(ip - 1));
  const int first_axis = turn ? axis_of(j * E) : 0;
  // the thread's pairs all go by one axis: its angles are whole vectors
  const bool one_axis =
      p.axes == 1 || (!p.interleaved && turn && first_axis == axis_of(j * E + E - 1));
  __syncthreads();

  for (int t = 0; t < tokens && tok0 + t < p.N; ++t) {
    if (!places[t].live) continue;
    const long long tok = tok0 + t;
    const size_t off = places[t].off;
    for (int y = y0; y < heads; y += ny * kHeadsAhead) {
      uint4 a[kHeadsAhead], b[kHeadsAhead];
#pragma unroll
      for (int k = 0; k < kHeadsAhead; ++k) {
        const int h = y + k * ny;
        if (h < heads) {
          const bool val = h >= hq + p.HKV;
          const T* x = h < hq ? static_cast<const T*>(p.q) + tok * p.qs + (long long)h * p.D
                       : !val ? static_cast<const T*>(p.k) + tok * p.ks + (long long)(h - hq) * p.D
                              : static_cast<const T*>(p.v) + tok * p.vs +
                                    (long long)(h - hq - p.HKV) * p.D;
          a[k] = reinterpret_cast<const uint4*>(x)[val ? 2 * j : v0];
          b[k] = reinterpret_cast<const uint4*>(x)[val ? 2 * j + 1 : v1];
        }
      }
      float cs[E], sn[E];
      if (turn) {
        if (one_axis) {
          const float4* row = reinterpret_cast<const float4*>(
              p.rope + (size_t)places[t].pos[first_axis] * 2 * p.P + j * E);
#pragma unroll
          for (int e = 0; e < E; e += 4) {
            const float4 c4 = __ldg(row + e / 4), s4 = __ldg(row + (p.P + e) / 4);
            cs[e] = c4.x, cs[e + 1] = c4.y, cs[e + 2] = c4.z, cs[e + 3] = c4.w;
            sn[e] = s4.x, sn[e + 1] = s4.y, sn[e + 2] = s4.z, sn[e + 3] = s4.w;
          }
        } else {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const float* row =
                p.rope + (size_t)places[t].pos[axis_of(j * E + e)] * 2 * p.P + j * E + e;
            cs[e] = __ldg(row);
            sn[e] = __ldg(row + p.P);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < kHeadsAhead; ++k) {
        const int h = y + k * ny;
        if (h < heads) {
          const bool val = h >= hq + p.HKV;
          if constexpr (!MORE) {
            if (turn && !val) {
              float xa[E], xb[E], ya[E], yb[E];
              V::unpack(a[k], xa);
              V::unpack(b[k], xb);
#pragma unroll
              for (int e = 0; e < E; ++e) {
                ya[e] = fmaf(xa[e], cs[e], -xb[e] * sn[e]);
                yb[e] = fmaf(xb[e], cs[e], xa[e] * sn[e]);
              }
              a[k] = V::pack(ya);
              b[k] = V::pack(yb);
            }
            uint4* to = h < hq ? reinterpret_cast<uint4*>(static_cast<T*>(p.q_out) +
                                                          ((size_t)tok * p.HQ + h) * p.D)
                        : !val ? reinterpret_cast<uint4*>(p.kp + off + (h - hq) * head_bytes)
                               : reinterpret_cast<uint4*>(p.vp + off + (h - hq - p.HKV) * head_bytes);
            to[val ? 2 * j : v0] = a[k];
            to[val ? 2 * j + 1 : v1] = b[k];
            if (p.k_out != nullptr && h >= hq && !val) {
              uint4* out = reinterpret_cast<uint4*>(static_cast<T*>(p.k_out) +
                                                    ((size_t)tok * p.HKV + h - hq) * p.D);
              out[v0] = a[k];
              out[v1] = b[k];
            }
          } else {
            write_head<T, E4M3>(p, tok, h, hq, off, head_bytes, a[k], b[k], v0, v1, j, ip, turn,
                                cs, sn, head_lanes);
          }
        }
      }
    }
  }
}

}  // namespace

cudaError_t kv_append_launch(const AppendParams& p, cudaStream_t st) {
  // a token to a CTA until the SMs have several each, then up to eight
  const int per = p.N / (kMaxSms * 8);
  const int tokens = per < 1 ? 1 : per < kMaxTokens ? per : kMaxTokens;
  const int grid = (p.N + tokens - 1) / tokens;
  const bool more = p.q_weight != nullptr || p.k_weight != nullptr || p.v_out != nullptr;
  auto run = [&](auto kernel) { kernel<<<grid, kAppendThreads, 0, st>>>(p, tokens); };
  if (p.dt == DT_F32) {
    if (more) run(kv_append_kernel<float, true, false>);
    else run(kv_append_kernel<float, false, false>);
  } else if (p.dt == DT_BF16) {
    if (p.scales != nullptr) run(kv_append_kernel<__nv_bfloat16, true, true>);
    else if (more) run(kv_append_kernel<__nv_bfloat16, true, false>);
    else run(kv_append_kernel<__nv_bfloat16, false, false>);
  } else {
    if (p.scales != nullptr) run(kv_append_kernel<__half, true, true>);
    else if (more) run(kv_append_kernel<__half, true, false>);
    else run(kv_append_kernel<__half, false, false>);
  }
  return cudaGetLastError();
}

}  // namespace rssm
