// Prefixes that rows of a batch share: the plan of a step, made from the page
// tables once for all layers, and the attention that reads each prefix once for
// all its rows.
//
// A fork leaves a prompt's full pages named by several tables. Rows whose tables
// begin with the same page form a group; its prefix is as many pages as all of
// them begin with, among those that every one has committed whole, so all of it
// is seen by all of the group's query tokens. The softmax of a row is then taken
// in two parts of its keys, which meet in the running maximum, sum and output
// (attn_decode.cuh): what the second launch begins with is what the first left.
//
// It is bound by trips to memory: one CTA, seven phases one after the other, 11 us
// for 64 rows of 130 pages. Once a step, so beside all layers' attention it is small;
// more CTAs would need waits over the grid.
//
// The plan says which rows and how many keys, not which pages: pages may move
// (all tables follow) and slots grow. Where a table no longer begins with its
// group's pages the attention sees that, and skips the row.
#include <climits>

#include "kv_common.cuh"

namespace rssm {

namespace {

constexpr int kShareThreads = 1024;
// Keys that a CTA takes of one row's own at most, if it has one row; longer ones are
// cut. 64 rows with four heads of 128 behind one prefix, four layers with the plan:
// 600 keys of their own 139 us an item to a CTA, 163 cut; 1500 keys 210 and 184, but
// over quantised pages 161 and 184.
constexpr int kMostOwn = 1024, kMostOwnQuant = 2048;
// Steps of 128 keys: a stretch at least, but for a prefix's last. 64 rows behind 8200
// keys: 2 or 4 116 us, 8 124.
constexpr int kLeastSteps = 4;

struct PlanShareParams {
  ShareView v;
  const int32_t* slot;
  const int32_t* table;
  const int32_t* held;
  const int32_t* length;
  int32_t* map;  // [n_pages] of the cache's work buffer
  int B, T, n_slots, n_pages, max_pages, shift;
  int HKV, rows, split;  // key heads; query rows of a row and key head; stretches at most, about
  int most_own;
};

__device__ __forceinline__ int scan_of(int x, int* sums, int tid, int& total) {
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
  return incl - x + (warp > 0 ? __shfl_sync(kFull, s, warp - 1) : 0);
}

// One CTA. Groups are numbered in the order of their first rows, so that the
// same tables give the same stretches, and sums, in the attention. Counters are
// read past the L1 cache, which atomics do not write.
__global__ void __launch_bounds__(kShareThreads)
    plan_share_kernel(const __grid_constant__ PlanShareParams p) {
  __shared__ int sums[32];
  __shared__ int all_cut, all_whole, longest;
  __shared__ unsigned long long work;  // steps of 128 keys of all blocks
  const int tid = threadIdx.x;
  int32_t* full = p.v.order;                // whole committed pages, until phase 3
  int32_t* count = p.v.scratch;             // of a lead: members; then its group
  int32_t* common = p.v.scratch + p.B;      // of a lead: pages; then its group's next place
  if (tid == 0) {
    p.v.of[0] = p.B;
    p.v.of[1] = p.T;
    *p.v.made_for = p.v.stamp;
    *p.v.lost = 0;
    work = 0;
    longest = 0;
  }
  // ---- 1: each row's whole pages, and the first row that begins with its page
  auto first_page = [&](int r) {
    const int s = p.slot[r];
    if (s < 0 || s >= p.n_slots || full[r] < 1) return -1;
    const int page = p.table[(size_t)s * p.max_pages];
    return page >= 0 && page < p.n_pages ? page : -1;
  };
  for (int r = tid; r < p.B; r += kShareThreads) {
    const int s = p.slot[r];
    int n = 0;
    if (s >= 0 && s < p.n_slots) {
      const int len = p.length[s], held = p.held[s];
      if (len >= 0 && held >= 0 && held <= p.max_pages &&
          (long long)len + p.T <= ((long long)held << p.shift))
        n = len >> p.shift;
    }
    full[r] = n;
    count[r] = 0;
    common[r] = INT_MAX;
    p.v.prefix[r] = 0;
    const int page = first_page(r);
    if (page >= 0) p.map[page] = INT_MAX;
  }
  __syncthreads();
  for (int r = tid; r < p.B; r += kShareThreads) {
    const int page = first_page(r);
    if (page >= 0) atomicMin(p.map + page, r);
  }
  __syncthreads();
  // ---- 2: pages in common with the lead, a warp to a row
  for (int r = tid >> 5; r < p.B; r += kShareThreads / 32) {
    const int lane = tid & 31, page = first_page(r);
    const int lead = page >= 0 ? __ldcg(p.map + page) : r;
    int same = full[r];
    if (lead != r) {
      const int n = min(same, full[lead]);
      const int32_t* a = p.table + (size_t)p.slot[r] * p.max_pages;
      const int32_t* b = p.table + (size_t)p.slot[lead] * p.max_pages;
      same = n;
      for (int i0 = 0; i0 < n; i0 += 128) {
        bool eq[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int i = i0 + 32 * k + lane;
          eq[k] = i >= n || a[i] == b[i];
        }
        int at = n;
#pragma unroll
        for (int k = 3; k >= 0; --k) {
          const unsigned off = __ballot_sync(kFull, !eq[k]);
          if (off) at = i0 + 32 * k + __ffs(off) - 1;
        }
        if (at < n) {
          same = at;
          break;
        }
      }
    }
    if (lane == 0) {
      p.v.group[r] = lead;  // until phase 5
      if (page >= 0) {
        atomicMin(common + lead, same);
        atomicAdd(count + lead, 1);
      }
    }
  }
  __syncthreads();
  // ---- 3: the groups, and the stretches that their prefixes are cut into
  auto group_of = [&](int r, int& n, int& keys) {  // whether r leads one; members, keys
    n = r < p.B ? __ldcg(count + r) : 0;
    const int pages = r < p.B ? __ldcg(common + r) : 0;
    keys = n >= 2 ? pages << p.shift : 0;
    return keys > 0;
  };
  auto blocks_of = [&](int n) { return (int)(((long long)n * p.rows + 127) / 128) * p.HKV; };
  unsigned long long mine = 0;
  for (int r = tid; r < p.B; r += kShareThreads) {
    int n, keys;
    if (group_of(r, n, keys))
      mine += (unsigned long long)blocks_of(n) * (unsigned)((keys + 127) / 128);
  }
  if (mine > 0) atomicAdd(&work, mine);
  __syncthreads();
  const unsigned long long even = (work + p.split - 1) / p.split;
  int per = even < kLeastSteps ? kLeastSteps : even > (1 << 24) ? 1 << 24 : (int)even;
  // a second turn of a few CTAs costs as much as the first: longer stretches where
  // that leaves one for each SM at most (20 groups of 4 rows of 700 to 5000 keys, four
  // heads: four layers 193 us, without this 230)
  for (int turn = 0; turn < 6; ++turn) {
    int cut = 0, whole = 0;  // stretches, blocks
    for (int r = tid; r < p.B; r += kShareThreads) {
      int n, keys;
      if (group_of(r, n, keys)) {
        const int b = blocks_of(n);
        whole += b;
        cut += b * (((keys + 127) / 128 + per - 1) / per);
      }
    }
    if (tid == 0) all_cut = all_whole = 0;
    __syncthreads();
    if (whole > 0) atomicAdd(&all_cut, cut), atomicAdd(&all_whole, whole);
    __syncthreads();
    const int n = all_cut, blocks = all_whole;
    __syncthreads();
    if (n <= p.split || blocks > p.split) break;
    per += max(1, (int)((long long)per * (n - p.split) / p.split));
  }
  int groups = 0, rows = 0, segs = 0, slots = 0;
  for (int r0 = 0; r0 < p.B; r0 += kShareThreads) {
    const int r = r0 + tid;
    int n, keys;
    const bool on = group_of(r, n, keys);
    const int parts = on ? ((keys + 127) / 128 + per - 1) / per : 0;
    const int here = on ? blocks_of(n) * parts : 0;
    int all_groups, all_rows, all_segs, all_slots;
    const int g = groups + scan_of(on, sums, tid, all_groups);
    const int at = rows + scan_of(on ? n : 0, sums, tid, all_rows);
    const int seg = segs + scan_of(here, sums, tid, all_segs);
    const int slot = slots + scan_of(parts > 1 ? here : 0, sums, tid, all_slots);
    if (r < p.B) {
      if (on) {
        p.v.begin[g] = at;
        p.v.group_keys[g] = keys;
        p.v.seg[g] = seg;
        p.v.parts[g] = parts;
        p.v.part0[g] = slot;
        p.v.order[at] = r;
        common[r] = 1;
        count[r] = g;
      } else {
        count[r] = -1;
      }
    }
    groups += all_groups;
    rows += all_rows;
    segs += all_segs;
    slots += all_slots;
  }
  if (tid == 0) {
    *p.v.groups = groups;
    *p.v.steps = per;
    *p.v.segments = segs;
    p.v.begin[groups] = rows;
    p.v.seg[groups] = segs;
  }
  __syncthreads();
  // ---- 4: a record of each stretch, so that a CTA that takes it has one look-up
  for (int i = tid; i < segs; i += kShareThreads) {
    int lo = 0, hi = groups;  // the last group whose first stretch is not behind i
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.v.seg[mid] <= i) lo = mid; else hi = mid;
    }
    const int parts = p.v.parts[lo], within = i - p.v.seg[lo];
    ShareSeg s;
    s.begin = p.v.begin[lo];
    s.lead = p.v.order[s.begin];
    s.group = lo;
    s.keys = p.v.group_keys[lo];
    s.rows = (p.v.begin[lo + 1] - s.begin) * p.rows;
    s.at = within / parts;
    s.part = within % parts;
    s.out = parts > 1 ? p.v.part0[lo] + within : -1;
    p.v.segs[i] = s;
  }
  // ---- 5: their members
  for (int r = tid; r < p.B; r += kShareThreads) {
    const int lead = p.v.group[r], g = __ldcg(count + lead);
    if (g < 0) continue;
    const int at = lead == r ? 0 : atomicAdd(common + lead, 1);
    const int begin = p.v.begin[g];
    if (at > 0) p.v.order[begin + at] = r;
    ShareRow x{};
    x.group = g;
    x.lead = lead;
    x.first = at * p.rows;
    x.parts = p.v.parts[g];
    x.part0 = p.v.part0[g];
    x.blocks = ((p.v.begin[g + 1] - begin) * p.rows + 127) / 128;
    p.v.rows[r] = x;
    p.v.prefix[r] = p.v.group_keys[g];
    p.v.group[r] = g;
  }
  // ---- 6: whether a CTA for each row and key head is the better split of the rows'
  // own keys. Slots grow: the answer is a matter of speed alone.
  for (int r = tid; r < p.B; r += kShareThreads) {
    const int s = p.slot[r];
    if (s >= 0 && s < p.n_slots) atomicMax(&longest, p.length[s] + p.T - p.v.prefix[r]);
  }
  __syncthreads();
  if (tid == 0) *p.v.direct = longest <= p.most_own;
}

}  // namespace

cudaError_t kv_share_launch(const ShareView& v, const PageParams& p, int HKV, int G,
                            bool quant, cudaStream_t st) {
  PlanShareParams s{};
  s.v = v;
  s.slot = p.slot;
  s.table = p.table;
  s.held = p.held;
  s.length = p.length;
  s.map = p.map;
  s.B = p.B;
  s.T = p.T;
  s.n_slots = p.n_slots;
  s.n_pages = p.n_pages;
  s.max_pages = p.max_pages;
  s.shift = p.shift;
  s.HKV = HKV;
  s.rows = p.T * G;
  s.most_own = quant ? kMostOwnQuant : kMostOwn;
  // Blocks that are cut leave fewer than 2 kShareSplit parts: an even split, and the
  // last stretch of each, which has another before it.
  s.split = kShareSplit;
  plan_share_kernel<<<1, kShareThreads, 0, st>>>(s);
  return cudaGetLastError();
}

}  // namespace rssm
