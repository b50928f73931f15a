// Pages of the key-value cache: handing them out, sharing them between forked
// slots, taking them back, moving them to the front of the pool, and the slots'
// lengths.
//
// The cache's state is whole numbers: table[slot][i] the page of the slot's
// tokens [i p, (i + 1) p), held[slot] how many pages it has, length[slot] its
// committed tokens, refs[page] how many tables name the page (0: free). One CTA
// plans a call: it scans the rows' needs and the reference counts, so free
// pages are given lowest first and in row order, and the same call on the same
// state always gives the same pages. Copies are listed as (from, to) pairs for
// a second launch that moves the bytes of every layer (HBM-bound; the plan is
// latency-bound and costs a few microseconds).
#include "kv_common.cuh"

namespace rssm {

namespace {

constexpr int kPlanThreads = 1024;

// Sum of one value per thread over the CTA before this thread (exclusive),
// and the total.
__device__ __forceinline__ int cta_scan(int x, int* sums, int tid, int& total) {
  const int warp = tid >> 5, lane = tid & 31;
  int incl = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(kFull, incl, d);
    if (lane >= d) incl += y;
  }
  __syncthreads();  // the last call's sums have been read
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  int s = sums[lane];
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(kFull, s, d);
    if (lane >= d) s += y;
  }
  total = __shfl_sync(kFull, s, 31);
  const int before = __shfl_sync(kFull, s, warp > 0 ? warp - 1 : 0);
  return incl - x + (warp > 0 ? before : 0);
}

// The lowest `want` pages with refs == 0, in order, into list; how many there are.
__device__ __forceinline__ int free_pages(const PageParams& p, int32_t* list, int want, int* sums,
                                          int tid) {
  int got = 0;
  for (int b = 0; b < p.n_pages && got < want; b += kPlanThreads) {
    const int i = b + tid;
    const int f = i < p.n_pages && __ldcg(p.refs + i) == 0;
    int n;
    const int at = got + cta_scan(f, sums, tid, n);
    if (f && at < want) list[at] = i;
    got += n;
  }
  __syncthreads();
  return got < want ? got : want;
}

__device__ __forceinline__ bool page_ok(const PageParams& p, int page) {
  if (page >= 0 && page < p.n_pages) return true;
  atomicOr(p.err, DEVERR_PAGES);
  return false;
}

// One reference less to each page of the rows' slots; the slots end empty. A
// warp per row.
__device__ __forceinline__ void release_rows(const PageParams& p, int tid) {
  const int warp = tid >> 5, lane = tid & 31;
  for (int r = warp; r < p.B; r += kPlanThreads / 32) {
    const int s = p.slot[r];
    if (s < 0 || (p.parent != nullptr && p.parent[r] < 0)) continue;
    if (s >= p.n_slots || (p.parent != nullptr && (p.parent[r] >= p.n_slots || p.parent[r] == s))) {
      if (lane == 0) atomicOr(p.err, DEVERR_SLOT);
      continue;
    }
    int32_t* row = p.table + (size_t)s * p.max_pages;
    const int held = min(max(p.held[s], 0), p.max_pages);
    for (int i = lane; i < held; i += 32) {
      const int page = row[i];
      if (page_ok(p, page) && atomicSub(p.refs + page, 1) <= 0) {
        atomicAdd(p.refs + page, 1);  // never below zero
        atomicOr(p.err, DEVERR_PAGES);
      }
      row[i] = -1;
    }
    __syncwarp();
    if (lane == 0) p.held[s] = 0, p.length[s] = 0;
  }
}

__global__ void __launch_bounds__(kPlanThreads) plan_reserve_kernel(const PageParams p) {
  __shared__ int sums[32];
  const int tid = threadIdx.x;
  // first free page of each row (p.rows) and the pages wanted in all
  int total = 0;
  for (int b = 0; b < p.B; b += kPlanThreads) {
    const int r = b + tid;
    int need = 0;
    if (r < p.B) {
      const int s = p.slot[r];
      uint32_t bad = 0;
      if (s >= p.n_slots) {
        bad = DEVERR_SLOT;
      } else if (s >= 0) {
        int n = p.T;
        if (p.cu != nullptr) {
          n = p.cu[r + 1] - p.cu[r];
          if (p.cu[r] < 0 || n < 0) bad = DEVERR_SEQLEN, n = 0;
        }
        const int len = p.length[s], held = p.held[s];
        if (len < 0 || held < 0 || held > p.max_pages) {
          bad |= len < 0 ? DEVERR_CURSOR : DEVERR_PAGES;
        } else if (bad == 0) {
          const long long pages = ((long long)len + n + (1 << p.shift) - 1) >> p.shift;
          if (pages > p.max_pages) {
            bad = DEVERR_PAGES;
          } else {
            need = pages > held ? (int)pages - held : 0;
          }
        }
      }
      if (bad) atomicOr(p.err, bad);
    }
    int n;
    const int at = total + cta_scan(need, sums, tid, n);
    if (r < p.B) p.rows[r] = at;
    total += n;
  }
  if (tid == 0) p.rows[p.B] = total;
  __syncthreads();
  if (total == 0) return;
  const int got = free_pages(p, p.dst, min(total, p.n_pages), sums, tid);
  for (int r = tid; r < p.B; r += kPlanThreads) {
    const int at = p.rows[r], n = p.rows[r + 1] - at;
    if (n == 0) continue;
    if (at + n > got) {
      atomicOr(p.err, DEVERR_PAGES);
      continue;
    }
    const int s = p.slot[r], held = p.held[s];
    for (int i = 0; i < n; ++i) {
      const int page = p.dst[at + i];
      p.table[(size_t)s * p.max_pages + held + i] = page;
      p.refs[page] = 1;
    }
    p.held[s] = held + n;
  }
}

__global__ void __launch_bounds__(kPlanThreads) plan_release_kernel(const PageParams p) {
  release_rows(p, threadIdx.x);
}

__global__ void __launch_bounds__(kPlanThreads) plan_fork_kernel(const PageParams p) {
  __shared__ int sums[32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int page = 1 << p.shift;
  release_rows(p, tid);
  __syncthreads();
  // what each row shares and what it needs new
  auto row_of = [&](int r, int& s, int& d, int& len, int& whole, int& need) {
    s = p.parent[r];
    d = p.slot[r];
    if (s < 0 || d < 0 || s >= p.n_slots || d >= p.n_slots || s == d) return false;
    len = p.length[s];
    if (len < 0 || len > ((long long)min(max(p.held[s], 0), p.max_pages) << p.shift)) {
      atomicOr(p.err, len < 0 ? DEVERR_CURSOR : DEVERR_PAGES);
      return false;
    }
    const int pages = (int)(((long long)len + page - 1) >> p.shift);
    whole = p.deep ? 0 : len >> p.shift;
    need = pages - whole;
    return true;
  };
  int total = 0;
  for (int b = 0; b < p.B; b += kPlanThreads) {
    const int r = b + tid;
    int s, d, len, whole, need = 0;
    if (r < p.B && !row_of(r, s, d, len, whole, need)) need = 0;
    int n;
    const int at = total + cta_scan(need, sums, tid, n);
    if (r < p.B) p.rows[r] = at;
    total += n;
  }
  if (tid == 0) p.rows[p.B] = total;
  __syncthreads();
  for (int r = warp; r < p.B; r += kPlanThreads / 32) {
    int s, d, len, whole, need;
    if (p.deep || !row_of(r, s, d, len, whole, need)) continue;
    for (int i = lane; i < whole; i += 32) {
      const int pg = p.table[(size_t)s * p.max_pages + i];
      if (page_ok(p, pg)) atomicAdd(p.refs + pg, 1);
    }
  }
  __syncthreads();
  const int got = total > 0 ? free_pages(p, p.dst, min(total, p.n_pages), sums, tid) : 0;
  __syncthreads();
  int moves = 0;
  for (int b = 0; b < p.B; b += kPlanThreads / 32) {
    const int r = b + warp;
    int s, d, len, whole, need;
    if (r >= p.B || !row_of(r, s, d, len, whole, need)) continue;
    const int at = p.rows[r];
    const int32_t* from = p.table + (size_t)s * p.max_pages;
    int32_t* to = p.table + (size_t)d * p.max_pages;
    if (at + need > got) {  // not enough pages: the row shares nothing after all
      for (int i = lane; i < whole; i += 32) {
        if (from[i] >= 0 && from[i] < p.n_pages) atomicSub(p.refs + from[i], 1);
      }
      if (lane == 0) atomicOr(p.err, DEVERR_PAGES);
      continue;
    }
    for (int i = lane; i < whole + need; i += 32) {
      const int pg = from[i];
      if (i < whole) {
        to[i] = pg;
      } else {
        const int at_i = at + i - whole, fresh = p.dst[at_i];
        to[i] = fresh;
        p.refs[fresh] = 1;
        p.src[at_i] = page_ok(p, pg) ? pg : fresh;
      }
    }
    if (lane == 0) p.held[d] = whole + need, p.length[d] = len;
    moves = max(moves, at + need);
  }
  if (lane == 0) sums[warp] = moves;
  __syncthreads();
  if (tid == 0) {
    for (int w = 0; w < kPlanThreads / 32; ++w) moves = max(moves, sums[w]);
    *p.moves = moves;
  }
}

// Pages in use move to the front: the n-th used page behind the first U places
// (U pages are in use) to the n-th free place within them.
__global__ void __launch_bounds__(kPlanThreads) plan_compact_kernel(const PageParams p) {
  __shared__ int sums[32];
  const int tid = threadIdx.x;
  int used = 0;
  for (int b = 0; b < p.n_pages; b += kPlanThreads) {
    const int i = b + tid;
    used += __syncthreads_count(i < p.n_pages && p.refs[i] > 0);
  }
  int holes = 0, movers = 0;
  for (int b = 0; b < p.n_pages; b += kPlanThreads) {
    const int i = b + tid;
    const bool in = i < p.n_pages;
    const bool live = in && p.refs[i] > 0;
    const int h = in && i < used && !live, m = in && i >= used && live;
    int nh, nm;
    const int ah = holes + cta_scan(h, sums, tid, nh);
    const int am = movers + cta_scan(m, sums, tid, nm);
    if (h) p.dst[ah] = i;
    if (m) p.src[am] = i;
    if (in) p.map[i] = i;
    holes += nh;
    movers += nm;
  }
  __syncthreads();
  for (int i = tid; i < movers; i += kPlanThreads) {
    const int s = p.src[i], d = p.dst[i];
    p.map[s] = d;
    p.refs[d] = p.refs[s];
    p.refs[s] = 0;
  }
  if (tid == 0) *p.moves = movers;
}

// Copies of whole pages, every layer's keys and values, 16 KB of a page per
// CTA step; with a map, the tables take the pages' new places too.
constexpr int kCopyThreads = 256;
constexpr int kCopyVecs = 4;

__global__ void __launch_bounds__(kCopyThreads) page_copy_kernel(const CopyParams p) {
  const int moves = *p.moves;
  constexpr size_t step = (size_t)kCopyThreads * kCopyVecs * 16;
  const size_t chunks = (p.page_bytes + step - 1) / step;
  const size_t units = (size_t)moves * chunks * p.n_layers * 2;
  for (size_t u = blockIdx.x; u < units; u += gridDim.x) {
    const size_t mv = u / (chunks * p.n_layers * 2), rest = u % (chunks * p.n_layers * 2);
    const size_t lay = rest / (chunks * 2), which = rest / chunks % 2, chunk = rest % chunks;
    unsigned char* base = (which ? p.v : p.k) + lay * p.layer_bytes;
    const uint4* s = reinterpret_cast<const uint4*>(base + p.src[mv] * p.page_bytes);
    uint4* d = reinterpret_cast<uint4*>(base + p.dst[mv] * p.page_bytes);
    const size_t at = chunk * step / 16 + threadIdx.x, end = p.page_bytes / 16;
    uint4 v[kCopyVecs];
#pragma unroll
    for (int i = 0; i < kCopyVecs; ++i) {
      if (at + i * kCopyThreads < end) v[i] = s[at + i * kCopyThreads];
    }
#pragma unroll
    for (int i = 0; i < kCopyVecs; ++i) {
      if (at + i * kCopyThreads < end) d[at + i * kCopyThreads] = v[i];
    }
  }
  if (p.map != nullptr && moves > 0) {
    for (size_t i = (size_t)blockIdx.x * kCopyThreads + threadIdx.x; i < p.table_size;
         i += (size_t)gridDim.x * kCopyThreads) {
      const int page = p.table[i];
      if (page >= 0 && page < p.n_pages) p.table[i] = p.map[page];
    }
  }
}

__global__ void __launch_bounds__(256) length_kernel(const LengthParams p) {
  const int r = blockIdx.x * 256 + threadIdx.x;
  if (r >= p.B) return;
  const int s = p.slot[r];
  if (s < 0) return;
  int n = p.T;
  uint32_t bad = 0;
  if (s >= p.n_slots) {
    bad = DEVERR_SLOT;
  } else {
    if (p.cu != nullptr) {
      n = p.cu[r + 1] - p.cu[r];
      if (p.cu[r] < 0 || n < 0) bad = DEVERR_SEQLEN;
    }
    const int a = p.accept != nullptr ? p.accept[r] : n;
    if (bad == 0 && (a < 0 || a > n)) bad = DEVERR_ACCEPT;
    if (bad == 0) {
      const long long to = (long long)p.length[s] + a;
      if (p.length[s] < 0) {
        bad = DEVERR_CURSOR;
      } else if (to > ((long long)p.held[s] << p.shift)) {
        bad = DEVERR_PAGES;
      } else {
        p.length[s] = (int)to;
      }
    }
  }
  if (bad) atomicOr(p.err, bad);
}

}  // namespace

cudaError_t kv_plan_launch(int mode, const PageParams& p, cudaStream_t st) {
  switch (mode) {
    case PLAN_RESERVE: plan_reserve_kernel<<<1, kPlanThreads, 0, st>>>(p); break;
    case PLAN_FORK: plan_fork_kernel<<<1, kPlanThreads, 0, st>>>(p); break;
    case PLAN_RELEASE: plan_release_kernel<<<1, kPlanThreads, 0, st>>>(p); break;
    case PLAN_COMPACT: plan_compact_kernel<<<1, kPlanThreads, 0, st>>>(p); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

cudaError_t kv_copy_launch(const CopyParams& p, int num_sms, cudaStream_t st) {
  page_copy_kernel<<<num_sms * 8, kCopyThreads, 0, st>>>(p);
  return cudaGetLastError();
}

cudaError_t kv_length_launch(const LengthParams& p, cudaStream_t st) {
  length_kernel<<<(p.B + 255) / 256, 256, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace rssm
