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
// a second launch that moves the bytes of every layer (HBM-bound: 510 MB
// moved in 157 us, 96% of the copy rate). The plan is bound by its trips to memory, one behind
// the other: 10.6 us for a fork of 96 slots (16 to 19 with a warp per row), 7.5 us
// for a compaction of 3899 pages; the copies are launched beside it.
#include "kv_common.cuh"

namespace rssm {

namespace {

constexpr int kPlanThreads = 1024;
// Where the sum of a call's needs stops: more pages than any pool has (2^28), and
// with a block's rows behind it (1024 of at most 2^20 pages) still below 2^31.
constexpr int kPlenty = 1 << 29;

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

// Eight neighbouring pages' reference counts per thread: a block of 8192 pages
// costs one trip to memory and one scan. Pages outside the pool count as used.
constexpr int kPerThread = 8;
constexpr int kPlanBlock = kPlanThreads * kPerThread;
__device__ __forceinline__ void load_refs(const PageParams& p, int first, int (&r)[kPerThread]) {
#pragma unroll
  for (int i = 0; i < kPerThread; ++i)
    r[i] = first + i < p.n_pages ? __ldcg(p.refs + first + i) : 1;
}

// The lowest `want` pages with refs == 0, in order, into list; how many there are.
__device__ __forceinline__ int free_pages(const PageParams& p, int32_t* list, int want, int* sums,
                                          int tid) {
  int got = 0;
  for (int b = 0; b < p.n_pages && got < want; b += kPlanBlock) {
    const int first = b + tid * kPerThread;
    int r[kPerThread], n = 0, all;
    load_refs(p, first, r);
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) n += r[i] == 0;
    int at = got + cta_scan(n, sums, tid, all);
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      if (r[i] == 0) {
        if (at < want) list[at] = first + i;
        ++at;
      }
    }
    got += all;
  }
  __syncthreads();
  return got < want ? got : want;
}

__device__ __forceinline__ bool page_ok(const PageParams& p, int page) {
  if (page >= 0 && page < p.n_pages) return true;
  atomicOr(p.err, DEVERR_PAGES);
  return false;
}

// Eight lanes to a row: 128 rows at a time, so that a plan for a batch is a few
// trips to memory long, not a few per row.
constexpr int kRowLanes = 8;
constexpr int kRowsAtOnce = kPlanThreads / kRowLanes;

// One reference less to each page of the rows' slots; the slots end empty.
__global__ void __launch_bounds__(kPlanThreads) plan_release_kernel(const PageParams p) {
  const int sub = threadIdx.x % kRowLanes;
  for (int r = threadIdx.x / kRowLanes; r < p.B; r += kRowsAtOnce) {
    const int s = p.slot[r];
    if (s < 0) continue;
    if (s >= p.n_slots) {
      if (sub == 0) atomicOr(p.err, DEVERR_SLOT);
      continue;
    }
    int32_t* row = p.table + (size_t)s * p.max_pages;
    const int held = min(max(p.held[s], 0), p.max_pages);
#pragma unroll 4
    for (int i = sub; i < held; i += kRowLanes) {
      const int page = row[i];
      if (page_ok(p, page)) atomicSub(p.refs + page, 1);
      row[i] = -1;
    }
    __syncwarp(0xffu << (threadIdx.x & 24));  // the row's lanes have read held
    if (sub == 0) p.held[s] = 0, p.length[s] = 0;
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
    total = min(total + n, kPlenty);
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

// What a row of a fork takes: `whole` shared pages, `need` new ones.
struct ForkRow {
  int s, d, held, len, whole, need;
};
__device__ __forceinline__ ForkRow fork_row(const PageParams& p, int r, bool tell) {
  ForkRow f{-1, -1, 0, 0, 0, 0};
  if (r >= p.B) return f;
  const int s = p.parent[r], d = p.slot[r];
  if (s < 0 || d < 0) return f;
  if (s >= p.n_slots || d >= p.n_slots || s == d) {
    if (tell) atomicOr(p.err, DEVERR_SLOT);
    return f;
  }
  const int len = p.length[s], held = p.held[s];
  f.d = d;
  f.held = min(max(p.held[d], 0), p.max_pages);
  if (len < 0 || len > ((long long)min(max(held, 0), p.max_pages) << p.shift)) {
    if (tell) atomicOr(p.err, len < 0 ? DEVERR_CURSOR : DEVERR_PAGES);
    return f;  // the destination ends empty
  }
  f.s = s;
  f.len = len;
  f.whole = p.deep ? 0 : len >> p.shift;
  f.need = (int)(((long long)len + (1 << p.shift) - 1) >> p.shift) - f.whole;
  return f;
}

__global__ void __launch_bounds__(kPlanThreads) plan_fork_kernel(const PageParams p) {
  __shared__ int sums[32];
  asm volatile("griddepcontrol.launch_dependents;");  // the copies' launch
  __shared__ ForkRow rows[kPlanThreads];
  const int tid = threadIdx.x, sub = tid % kRowLanes;
  // every row's needs before any length is changed (p.rows: first new page)
  int total = 0;
  for (int b = 0; b < p.B; b += kPlanThreads) {
    const ForkRow f = fork_row(p, b + tid, true);
    if (b == 0) rows[tid] = f;
    int n;
    const int at = total + cta_scan(f.need, sums, tid, n);
    if (b + tid < p.B) p.rows[b + tid] = at;
    total = min(total + n, kPlenty);
  }
  if (tid == 0) p.rows[p.B] = total;
  __syncthreads();
  // the destinations give back what they hold and share the sources' full
  // pages (no page is handed out in between, so none is lost by the order)
  for (int b = 0; b < p.B; b += kRowsAtOnce) {
    const int r = b + tid / kRowLanes;
    const ForkRow f = r < kPlanThreads ? rows[r] : fork_row(p, r, false);
    if (f.d < 0) continue;
    int32_t* to = p.table + (size_t)f.d * p.max_pages;
    const int32_t* from = p.table + (size_t)max(f.s, 0) * p.max_pages;
#pragma unroll 4
    for (int i = sub; i < max(f.held, f.whole); i += kRowLanes) {
      const int old = i < f.held ? to[i] : -1, pg = i < f.whole ? from[i] : -1;
      if (i < f.held && page_ok(p, old)) atomicSub(p.refs + old, 1);
      if (i < f.whole && page_ok(p, pg)) atomicAdd(p.refs + pg, 1);
      to[i] = pg;
    }
  }
  __syncthreads();
  const int got = total > 0 ? free_pages(p, p.dst, min(total, p.n_pages), sums, tid) : 0;
  int moves = 0;
  for (int b = 0; b < p.B; b += kRowsAtOnce) {
    const int r = b + tid / kRowLanes;
    // lengths and pages held of sources are as they were: none is a destination
    const ForkRow f = r < kPlanThreads ? rows[r] : fork_row(p, r, false);
    if (f.d < 0) continue;
    int32_t* to = p.table + (size_t)f.d * p.max_pages;
    const int32_t* from = p.table + (size_t)max(f.s, 0) * p.max_pages;
    const int at = p.rows[r];
    const bool fits = f.s >= 0 && (f.need == 0 || at + f.need <= got);
    if (f.s >= 0 && !fits) {  // not enough pages: the row shares nothing after all
      for (int i = sub; i < f.whole; i += kRowLanes) {
        if (from[i] >= 0 && from[i] < p.n_pages) atomicSub(p.refs + from[i], 1);
        to[i] = -1;
      }
      if (sub == 0) atomicOr(p.err, DEVERR_PAGES);
    }
    if (fits) {
      for (int i = sub; i < f.need; i += kRowLanes) {
        const int pg = from[f.whole + i], fresh = p.dst[at + i];
        to[f.whole + i] = fresh;
        p.refs[fresh] = 1;
        p.src[at + i] = page_ok(p, pg) ? pg : fresh;
      }
      moves = max(moves, at + f.need);
    }
    if (sub == 0) {
      p.held[f.d] = fits ? f.whole + f.need : 0;
      p.length[f.d] = fits ? f.len : 0;
    }
  }
  moves = __reduce_max_sync(kFull, moves);
  __syncthreads();
  if (tid % 32 == 0) sums[tid / 32] = moves;
  __syncthreads();
  if (tid < 32) {
    moves = __reduce_max_sync(kFull, sums[tid]);
    if (tid == 0) *p.moves = moves;
  }
}

// Pages in use move to the front: the n-th used page behind the first U places
// (U pages are in use) to the n-th free place within them.
__global__ void __launch_bounds__(kPlanThreads) plan_compact_kernel(const PageParams p) {
  __shared__ int sums[32];
  asm volatile("griddepcontrol.launch_dependents;");  // the copies' launch
  const int tid = threadIdx.x;
  int r[kPerThread], used = 0, n = 0;
  for (int b = 0; b < p.n_pages; b += kPlanBlock) {
    const int first = b + tid * kPerThread;
    load_refs(p, first, r);
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) n += first + i < p.n_pages && r[i] > 0;
  }
  cta_scan(n, sums, tid, used);
  int holes = 0, movers = 0;
  for (int b = 0; b < p.n_pages; b += kPlanBlock) {
    const int first = b + tid * kPerThread;
    if (p.n_pages > kPlanBlock) load_refs(p, first, r);  // else they are at hand
    int both = 0, all;  // free places in the low half word, pages to move in the high one
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      if (first + i < p.n_pages) {
        both += first + i < used ? r[i] <= 0 : (r[i] > 0) << 16;
        p.map[first + i] = first + i;
      }
    }
    const int before = cta_scan(both, sums, tid, all);
    int ah = holes + (before & 0xffff), am = movers + (before >> 16);
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      if (first + i < p.n_pages) {
        if (first + i < used) {
          if (r[i] <= 0) p.dst[ah++] = first + i;
        } else if (r[i] > 0) {
          p.src[am++] = first + i;
        }
      }
    }
    holes += all & 0xffff;
    movers += all >> 16;
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

// Copies of whole pages, every layer's keys and values (and scales), 16 KB of a
// page per CTA step; with a map, the tables take the pages' new places too.
constexpr int kCopyThreads = 256;
constexpr int kCopyVecs = 4;

__global__ void __launch_bounds__(kCopyThreads) page_copy_kernel(const CopyParams p) {
  // launched while the plan runs (its CTA leaves the other SMs idle); waits
  // here until the plan has ended and its list can be seen
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int moves = *p.moves;
  constexpr size_t step = (size_t)kCopyThreads * kCopyVecs * 16;
  const size_t chunks = (p.page_bytes + step - 1) / step;
  const int kinds = p.scales != nullptr ? 3 : 2;  // keys, values, scales of quantised pages
  const size_t units = (size_t)moves * chunks * p.n_layers * kinds;
  for (size_t u = blockIdx.x; u < units; u += gridDim.x) {
    const size_t mv = u / (chunks * p.n_layers * kinds), rest = u % (chunks * p.n_layers * kinds);
    const size_t lay = rest / (chunks * kinds), which = rest / chunks % kinds, chunk = rest % chunks;
    const size_t bytes = which == 2 ? p.scale_page_bytes : p.page_bytes;
    unsigned char* base = (which == 0 ? p.k : which == 1 ? p.v : p.scales) +
                          lay * (which == 2 ? p.scale_layer_bytes : p.layer_bytes);
    const uint4* s = reinterpret_cast<const uint4*>(base + p.src[mv] * bytes);
    uint4* d = reinterpret_cast<uint4*>(base + p.dst[mv] * bytes);
    const size_t at = chunk * step / 16 + threadIdx.x, end = bytes / 16;
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
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)num_sms * 8);
  cfg.blockDim = dim3(kCopyThreads);
  cfg.stream = st;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, page_copy_kernel, p);
}

cudaError_t kv_length_launch(const LengthParams& p, cudaStream_t st) {
  length_kernel<<<(p.B + 255) / 256, 256, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace rssm
