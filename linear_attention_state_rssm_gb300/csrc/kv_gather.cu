// Keys and values of cached tokens, read back from the slots' pages in a row:
//     out[cu[r] + i] = page value of token first[r] + i of slot[r],
// e4m3 pages as code 2^e in the output's type (one rounding; exact in bf16 and,
// between 2^-15 and 65504, in fp16). That is what the attention of a prompt
// takes for the part of its keys that the cache holds already.
//
// Bytes bound it. A page keeps a head's tokens side by side, the row a token's
// heads: a CTA takes a block of tokens and all heads, so both sides see runs of
// D values, and its threads have kAhead loads each on their way.
#include "kv_common.cuh"
#include "kv_tokens.cuh"

namespace rssm {

namespace {

constexpr int kGatherThreads = 256;
constexpr int kGatherTokens = 16;  // of a CTA at most
constexpr int kAhead = 4;

// Where token `tok` begins in the layer's pages (its first head), in units of D
// values; -1 where it is not read.
__device__ __forceinline__ long long gather_place(const GatherParams& p, int tok) {
  int r, i;
  if (!token_row(p.cu, p.B, p.T, p.N, tok, r, i)) return -1;
  const int s = p.slot[r];
  if (s < 0) return -1;
  uint32_t bad = 0;
  long long at = -1;
  if (s >= p.n_slots) {
    bad = DEVERR_SLOT;
  } else {
    const int first = p.first != nullptr ? p.first[r] : 0, held = p.held[s];
    const long long tok_at = (long long)first + i;
    if (first < 0 || held < 0 || held > p.max_pages || tok_at >= ((long long)held << p.shift)) {
      bad = DEVERR_PAGES;
    } else {
      const int page = p.table[(size_t)s * p.max_pages + (tok_at >> p.shift)];
      if (page < 0 || page >= p.n_pages) {
        bad = DEVERR_PAGES;
      } else {
        at = ((long long)page * p.HKV << p.shift) + (tok_at & ((1 << p.shift) - 1));
      }
    }
  }
  if (bad) atomicOr(p.err, bad);
  return at;
}

template <typename T, bool E4M3>
__global__ void __launch_bounds__(kGatherThreads)
    kv_gather_kernel(const __grid_constant__ GatherParams p, int tokens) {
  using V = Vec16<T>;
  constexpr int E = V::E;
  __shared__ long long places[kGatherTokens];
  const int tid = threadIdx.x;
  if (p.cu != nullptr && blockIdx.x == 0) {
    for (int r = tid; r < p.B; r += kGatherThreads) {
      if (p.cu[r] < 0 || p.cu[r + 1] < p.cu[r] || p.cu[r + 1] > p.N) atomicOr(p.err, DEVERR_SEQLEN);
    }
  }
  const int tok0 = blockIdx.x * tokens;
  const int n = min(tokens, p.N - tok0);
  if (tid < n) places[tid] = gather_place(p, tok0 + tid);
  __syncthreads();
  // 16 bytes of the output a thread: [which][token][head][unit]
  const int units = p.D / E, row = p.HKV * units, all = n * row;
  for (int which = 0; which < 2; ++which) {
    T* out = static_cast<T*>(which ? p.v_out : p.k_out);
    if (out == nullptr) continue;
    const unsigned char* pages = which ? p.vp : p.kp;
    uint4* to = reinterpret_cast<uint4*>(out + (size_t)tok0 * p.HKV * p.D);
    for (int i0 = tid; i0 < all; i0 += kGatherThreads * kAhead) {
      uint4 x[kAhead];
      unsigned char sc[kAhead];
      bool live[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int i = i0 + k * kGatherThreads;
        live[k] = i < all && places[i / row] >= 0;
        if (live[k]) {
          const int h = i % row / units, u = i % units;
          const size_t at = (size_t)places[i / row] + ((size_t)h << p.shift);
          if constexpr (E4M3) {
            const uint2 c = __ldg(reinterpret_cast<const uint2*>(pages + at * p.D) + u);
            x[k].x = c.x, x[k].y = c.y;
            sc[k] = __ldg(p.scales + 2 * at + which);
          } else {
            x[k] = __ldg(reinterpret_cast<const uint4*>(pages + at * p.D * sizeof(T)) + u);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int i = i0 + k * kGatherThreads;
        if (live[k]) {
          if constexpr (E4M3) {
            static_assert(!E4M3 || E == 8, "sixteen-bit outputs");
            float v[8];
            const float up = __uint_as_float((uint32_t)sc[k] << 23);
            e4m3x4_values(x[k].x, up, v);
            e4m3x4_values(x[k].y, up, v + 4);
            x[k] = V::pack(v);
          }
          to[i] = x[k];
        }
      }
    }
  }
}

}  // namespace

cudaError_t kv_gather_launch(const GatherParams& p, int num_sms, cudaStream_t st) {
  // a token to a CTA until the SMs have several each
  const int per = p.N / (num_sms * 4);
  const int tokens = per < 1 ? 1 : per < kGatherTokens ? per : kGatherTokens;
  const int grid = (p.N + tokens - 1) / tokens;
  auto run = [&](auto kernel) { kernel<<<grid, kGatherThreads, 0, st>>>(p, tokens); };
  if (p.dt == DT_F32) run(kv_gather_kernel<float, false>);
  else if (p.dt == DT_BF16 && p.scales == nullptr) run(kv_gather_kernel<__nv_bfloat16, false>);
  else if (p.dt == DT_BF16) run(kv_gather_kernel<__nv_bfloat16, true>);
  else if (p.scales == nullptr) run(kv_gather_kernel<__half, false>);
  else run(kv_gather_kernel<__half, true>);
  return cudaGetLastError();
}

}  // namespace rssm
