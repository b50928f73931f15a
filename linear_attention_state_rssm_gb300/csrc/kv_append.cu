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
#include "attn_core.cuh"
#include "kv_common.cuh"

namespace rssm {

namespace {

constexpr int kAppendThreads = 192;
constexpr int kHeadsAhead = 2;

template <typename T>
struct Vec16 {
  static constexpr int E = 16 / (int)sizeof(T);
  static __device__ __forceinline__ void unpack(const uint4& u, float (&v)[E]) {
    const T* t = reinterpret_cast<const T*>(&u);
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = attn_f32(t[i]);
  }
  static __device__ __forceinline__ uint4 pack(const float (&v)[E]) {
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

constexpr int kMaxTokens = 8;  // of a CTA

struct TokenPlace {
  size_t off;             // bytes of its first head within the layer's pages
  int pos[kMaxRopeAxes];
  int live;
};

// Row, page and positions of token `tok`.
__device__ __forceinline__ TokenPlace place_of(const AppendParams& p, int tok, int token_bytes) {
  TokenPlace t{};
  int r, i;  // the token's row and place in its window
  if (p.cu == nullptr) {
    r = tok / p.T;
    i = tok - r * p.T;
  } else {
    int lo = 0, hi = p.B;  // last row that begins at or before the token
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.cu[mid] <= tok) lo = mid; else hi = mid;
    }
    r = lo;
    const int first = p.cu[r], end = p.cu[r + 1];
    // outside every window, or in one that is refused
    if (first < 0 || tok < first || tok >= end || end > p.N) return t;
    i = tok - first;
  }
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

template <typename T>
__global__ void __launch_bounds__(kAppendThreads, 5)
    kv_append_kernel(const __grid_constant__ AppendParams p, int tokens) {
  using V = Vec16<T>;
  constexpr int E = V::E;
  __shared__ TokenPlace places[kMaxTokens];
  const int tok0 = blockIdx.x * tokens, tid = threadIdx.x;
  const int token_bytes = p.D * (int)sizeof(T);  // of one head
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
  if (p.dt == DT_F32) {
    kv_append_kernel<float><<<grid, kAppendThreads, 0, st>>>(p, tokens);
  } else if (p.dt == DT_BF16) {
    kv_append_kernel<__nv_bfloat16><<<grid, kAppendThreads, 0, st>>>(p, tokens);
  } else {
    kv_append_kernel<__half><<<grid, kAppendThreads, 0, st>>>(p, tokens);
  }
  return cudaGetLastError();
}

}  // namespace rssm
