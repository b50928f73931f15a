// Which sequence and query tile a CTA of a packed prompt launch works on: the
// lengths are on the device, so each CTA finds its place by itself.
#pragma once

#include "attn_core.cuh"
#include "kv_common.cuh"

namespace rssm {

struct PromptTile {
  int tile;        // query tile of the sequence
  int q0, k0;      // the sequence's first query token and key
  int lq, lk;
};

// Offsets of sequence r; false for a null slot or offsets out of order.
__device__ __forceinline__ bool prompt_span(const PromptParams& p, int r, bool tell, int& q0,
                                            int& lq, int& k0, int& lk) {
  const int s = p.slot != nullptr ? p.slot[r] : 0;
  if (s < 0) return false;
  uint32_t bad = 0;
  if (s >= p.n_slots) bad = DEVERR_SLOT;
  q0 = p.cu[r];
  const int q1 = p.cu[r + 1];
  if (q0 < 0 || q1 < q0 || q1 > p.N) bad |= DEVERR_SEQLEN;
  k0 = q0;
  int k1 = q1;
  if (p.cuk != nullptr) {
    k0 = p.cuk[r];
    k1 = p.cuk[r + 1];
  }
  if (k0 < 0 || k1 < k0 || k1 > p.M) bad |= DEVERR_SEQLEN;
  if (bad) {
    if (tell) atomicOr(p.err, bad);
    return false;
  }
  lq = q1 - q0;
  lk = k1 - k0;
  return true;
}

// Tile `index` of the launch (tiles of `rows` query rows, a row being a token
// and one of the G query heads of a key head; sequences in order, a sequence's last tile first: it sees the most keys). Each warp finds
// it by itself; false when the launch has fewer tiles.
__device__ __forceinline__ bool find_tile(const PromptParams& p, int rows, int index, bool tell,
                                          PromptTile& out) {
  const int lane = threadIdx.x & 31;
  int before = 0;
  bool found = false;
  for (int r0 = 0; r0 < p.B; r0 += 32) {
    const int r = r0 + lane;
    int q0 = 0, k0 = 0, lq = 0, lk = 0, n = 0;
    if (r < p.B && prompt_span(p, r, tell && index == 0, q0, lq, k0, lk))
      n = (int)(((long long)lq * p.G + rows - 1) / rows);
    int incl = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(kFull, incl, d);
      if (lane >= d) incl += y;
    }
    const int at = before + incl - n;
    const unsigned has = __ballot_sync(kFull, at <= index && index < at + n);
    if (has != 0) {
      const int src = __ffs(has) - 1;
      out.tile = __shfl_sync(kFull, at + n - 1 - index, src);
      out.q0 = __shfl_sync(kFull, q0, src);
      out.k0 = __shfl_sync(kFull, k0, src);
      out.lq = __shfl_sync(kFull, lq, src);
      out.lk = __shfl_sync(kFull, lk, src);
      found = true;
      if (index != 0) return true;  // tile 0's warps look every sequence over
    }
    before += __shfl_sync(kFull, incl, 31);
  }
  // the launch has room for every tile unless sequences share query tokens
  if (tell && index == 0 && lane == 0 && before > (int)(gridDim.x / (unsigned)p.HKV))
    atomicOr(p.err, DEVERR_SEQLEN);
  return found;
}

}  // namespace rssm
