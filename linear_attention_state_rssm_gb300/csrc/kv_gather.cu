// Keys and values of cached tokens, read back from the slots' pages in a row:
//     out[cu[r] + i] = page value of token first[r] + i of slot[r],
// e4m3 pages as code 2^e in the output's type (one rounding; exact in bf16 and,
// between 2^-15 and 65504, in fp16). That is what the attention of a prompt
// takes for the part of its keys that the cache holds already.
//
// Bytes are all there is to it. A page keeps a head's tokens side by side, the row a token's
// heads: a CTA takes a block of tokens and all heads, so both sides see runs of
// D values, and its threads have kAhead loads of keys and of values each on their
// way. Measured (GB300): 12 rows of 0.5 to 16 k tokens, 8 heads of 128, e4m3 to bf16:
// 53 us, 4.8 TB/s (71% of the copy rate): sixteen codes are two stores of 16 bytes a lane,
// so a warp's store covers every second 16 bytes of a kilobyte, and L1 (73% busy, DRAM 45%)
// comes first. One load ahead 57, cached ones 63. 49.7 k tokens in 11 rows, bf16 pages 69 us,
// 5.9 TB/s; fp32 129 us, 6.3 TB/s.
#include "kv_common.cuh"
#include "kv_tokens.cuh"

namespace rssm {

namespace {

constexpr int kGatherThreads = 128;
constexpr int kGatherTokens = 16;  // of a CTA at most
constexpr int kAhead = 2;

// Where token `tok` begins in the layer's pages (its first head), in units of D
// values; -1 where it is not read.
__device__ __forceinline__ long long gather_place(const GatherParams& p, const int32_t* cu,
                                                  int tok) {
  int r, i;
  if (!token_row(cu, p.B, p.T, p.N, tok, r, i)) return -1;
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
  constexpr int SIZE = E4M3 ? 1 : (int)sizeof(T);  // of a page's value
  constexpr int E = 16 / SIZE;                     // values of a load
  __shared__ long long places[kGatherTokens];
  const int tid = threadIdx.x;
  if (p.cu != nullptr && blockIdx.x == 0) {
    for (int r = tid; r < p.B; r += kGatherThreads) {
      if (p.cu[r] < 0 || p.cu[r + 1] < p.cu[r] || p.cu[r + 1] > p.N) atomicOr(p.err, DEVERR_SEQLEN);
    }
  }
  const int tok0 = blockIdx.x * tokens;
  const int n = min(tokens, p.N - tok0);
  __shared__ int32_t offsets[kGatherThreads];
  const int32_t* cu = copy_offsets<kGatherThreads>(p.cu, p.B, offsets, tid);
  if (p.cu != nullptr) __syncthreads();
  if (tid < n) places[tid] = gather_place(p, cu, tok0 + tid);
  __syncthreads();
  // a thread has one place in the heads and goes from (token, head) to the next
  const int units = p.D / E;  // a power of two, at most 64
  const int u = tid & (units - 1), step = kGatherThreads / units;
  const int dt = step / p.HKV, dh = step % p.HKV;
  int t = tid / units / p.HKV, h = tid / units % p.HKV;
  const bool want_k = p.k_out != nullptr, want_v = p.v_out != nullptr;
  while (t < n) {
    uint4 k[kAhead], v[kAhead];
    uint32_t sc[kAhead];
    long long to[kAhead];  // of the outputs, in heads; -1: nothing
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      to[i] = -1;
      if (t < n && places[t] >= 0) {
        const size_t at = (size_t)places[t] + ((size_t)h << p.shift);
        to[i] = (long long)(tok0 + t) * p.HKV + h;
        const size_t from = at * p.D * SIZE;
        if (want_k) k[i] = __ldcs(reinterpret_cast<const uint4*>(p.kp + from) + u);
        if (want_v) v[i] = __ldcs(reinterpret_cast<const uint4*>(p.vp + from) + u);
        if constexpr (E4M3) sc[i] = __ldg(reinterpret_cast<const uint16_t*>(p.scales) + at);
      }
      t += dt;
      h += dh;
      if (h >= p.HKV) h -= p.HKV, ++t;
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (to[i] < 0) continue;
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        if (!(which ? want_v : want_k)) continue;
        uint4* out = reinterpret_cast<uint4*>(static_cast<T*>(which ? p.v_out : p.k_out) +
                                              to[i] * p.D + u * E);
        const uint4 x = which ? v[i] : k[i];
        if constexpr (E4M3) {
          const uint32_t w[4] = {x.x, x.y, x.z, x.w};
          const float up = __uint_as_float((sc[i] >> (8 * which) & 0xffu) << 23);
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            float f[8];
            e4m3x4_values(w[2 * y], up, f);
            e4m3x4_values(w[2 * y + 1], up, f + 4);
            out[y] = V::pack(f);
          }
        } else {
          out[0] = x;
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
