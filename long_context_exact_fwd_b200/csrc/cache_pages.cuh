// Pages of the cache: reserving (with copies of shared pages before they are written), forking,
// trimming and compacting.
//
// A page is free when its reference count is 0.  Decisions need the whole batch and the whole
// count array at once, in one order, so each operator is a plan by ONE block (prefix sums over the
// batch and over `refs`, 16 pages a thread per sweep: a pool of 16K pages is one sweep) followed,
// where data or long tables move, by a launch over all SMs that carries the plan out.  The plan is
// bound by latency (a handful of dependent loads and barriers), the copies by memory.
// Results do not depend on timing: the only atomics add and subtract whole numbers.
#pragma once
#include "cache.cuh"

namespace ra {
namespace cache {

constexpr int PLAN_THREADS = 1024;
constexpr int SWEEP = 16;            // pages a thread looks at per sweep
constexpr int COPY_THREADS = 256;
constexpr int COPY_BYTES = 16384;    // bytes of one copy unit: 4 x 16 bytes a thread

// What a plan leaves in the workspace for the launch that follows.
struct Plan {
  int pairs;       // page copies
  int rows;        // fork: entries
  int items;       // fork: table entries to copy
};

// Exclusive prefix sum over the block's threads; `total` to all.  `warp_sum` holds 33 ints.
__device__ __forceinline__ int block_scan(int x, int* warp_sum, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, s, d);
    if (lane >= d) s += y;
  }
  if (lane == 31) warp_sum[warp] = s;
  __syncthreads();
  if (warp == 0) {
    const int w = lane < static_cast<int>(blockDim.x >> 5) ? warp_sum[lane] : 0;
    int t = w;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, t, d);
      if (lane >= d) t += y;
    }
    warp_sum[lane] = t - w;
    if (lane == 31) warp_sum[32] = t;
  }
  __syncthreads();
  total = warp_sum[32];
  const int r = warp_sum[warp] + s - x;
  __syncthreads();
  return r;
}

// Pages with refs == 0 (want_free) or > 0, in ascending order from page `from`, into list[0 ..
// limit); returns how many were written.
__device__ __forceinline__ int list_pages(const int* refs, int from, int to, bool want_free, int limit, int* list,
                                          int* warp_sum) {
  int found = 0;
  for (int base = from; base < to && found < limit; base += PLAN_THREADS * SWEEP) {
    const int p0 = base + threadIdx.x * SWEEP;
    unsigned hit = 0;
#pragma unroll
    for (int i = 0; i < SWEEP; ++i)
      if (p0 + i < to && ((refs[p0 + i] == 0) == want_free)) hit |= 1u << i;
    int total;
    int at = found + block_scan(__popc(hit), warp_sum, total);
    for (; hit; hit &= hit - 1, ++at)
      if (at < limit) list[at] = p0 + __ffs(hit) - 1;
    found += total;
  }
  return found < limit ? found : limit;
}

// Pages for positions len .. len + n_new - 1 of every entry; len += n_new.  All or nothing: with
// too few free pages nothing changes.  granted (or null; may be n_new itself): n_new of the entries that were given
// room, 0 of the others.
__global__ void __launch_bounds__(PLAN_THREADS)
    reserve_plan_kernel(Pool c, const int* slots, const int* n_new, int B, int* granted, Plan* plan, int* pairs,
                        int* free_list) {
  behind_last();
  __shared__ int s_slot[MAX_BATCH], s_last[MAX_BATCH], s_first[MAX_BATCH], s_have[MAX_BATCH], warp_sum[33];
  const int b = threadIdx.x;
  const int slot = b < B ? slots[b] : -1;
  s_slot[b] = slot;
  __syncthreads();
  bool active = slot >= 0 && slot < c.slots;
  bool bad = slot < -1 || slot >= c.slots;
  int len = 0, n = 0, have = 0, need = 0, last = -1;
  if (active) {
    for (int i = 0; i < b; ++i) bad |= s_slot[i] == slot;
    len = c.lens[slot];
    n = n_new[b];
    bad |= len < 0 || n < 0 || len > c.max_pages * static_cast<long long>(c.page) ||
           static_cast<long long>(len) + n > c.max_pages * static_cast<long long>(c.page);
    active = !bad && n > 0;
  }
  if (active) {
    have = (len + c.page - 1) / c.page;
    need = (len + n + c.page - 1) / c.page - have;
    if (len % c.page) {
      last = c.table[static_cast<long long>(slot) * c.max_pages + have - 1];
      if (last < 0 || last >= c.pages) {
        bad = true;
        active = false;
        need = 0;
        last = -1;
      }
    }
  }
  if (bad) record_pages();
  s_last[b] = last;
  __syncthreads();
  // Entries that share a partly filled last page copy it, in batch order, until one holder is left.
  bool copied = false;
  if (last >= 0) {
    const int holders = c.refs[last];
    if (holders > 1) {
      int before = 0;
      for (int i = 0; i < b; ++i) before += s_last[i] == last;
      copied = holders - before > 1;
    }
  }
  int total, n_copies;
  const int first = block_scan(need + (copied ? 1 : 0), warp_sum, total);
  const int copy_at = block_scan(copied ? 1 : 0, warp_sum, n_copies);
  s_first[b] = first;
  s_have[b] = copied ? have - 1 : have;   // the first table column that gets a page
  const int found = list_pages(c.refs, 0, c.pages, true, total, free_list, warp_sum);
  if (found < total) {
    if (threadIdx.x == 0) {
      record_pages();
      plan->pairs = 0;
    }
    if (granted && b < B) granted[b] = 0;
    return;
  }
  __syncthreads();   // the list is complete, every count has been read
  if (copied) {
    pairs[2 * copy_at] = last;
    pairs[2 * copy_at + 1] = free_list[first];
    atomicSub(c.refs + last, 1);
  }
  for (int i = threadIdx.x; i < total; i += PLAN_THREADS) {
    const int r = find_row(s_first, B, i);
    const int pid = free_list[i];
    c.refs[pid] = 1;
    c.table[static_cast<long long>(s_slot[r]) * c.max_pages + s_have[r] + (i - s_first[r])] = pid;
  }
  if (active) c.lens[slot] = len + n;
  if (granted && b < B) granted[b] = active ? n : 0;
  if (threadIdx.x == 0) plan->pairs = n_copies;
}

// dst takes src's pages (references + 1) and length.  Sources are read as they were before the
// call; a destination has to be empty, and the first entry that names it has it.
__global__ void __launch_bounds__(PLAN_THREADS)
    fork_plan_kernel(Pool c, const int* src, const int* dst, int B, Plan* plan, int* first) {
  behind_last();
  __shared__ int s_dst[MAX_BATCH], warp_sum[33];
  const int b = threadIdx.x;
  const int s = b < B ? src[b] : -1, d = b < B ? dst[b] : -1;
  s_dst[b] = d;
  __syncthreads();
  bool active = !(s == -1 && d == -1);
  int len = 0;
  if (active) {
    bool ok = s >= 0 && s < c.slots && d >= 0 && d < c.slots && s != d;
    for (int i = 0; ok && i < b; ++i) ok = s_dst[i] != d;
    if (ok) {
      len = c.lens[s];
      ok = c.lens[d] == 0 && len >= 0 && len <= c.max_pages * static_cast<long long>(c.page);
    }
    if (!ok) record_pages();
    active = ok;
  }
  const int n = active ? (len + c.page - 1) / c.page : 0;
  int total;
  const int at = block_scan(n, warp_sum, total);   // barriers: every length has been read
  if (b < B) first[b] = at;
  if (active) c.lens[d] = len;
  if (b == 0) {
    plan->rows = B;
    plan->items = total;
  }
}

__global__ void __launch_bounds__(COPY_THREADS)
    fork_apply_kernel(Pool c, const int* src, const int* dst, const Plan* plan, const int* first) {
  behind_last();
  const int rows = plan->rows, items = plan->items;
  for (int i = blockIdx.x * COPY_THREADS + threadIdx.x; i < items; i += gridDim.x * COPY_THREADS) {
    const int r = find_row(first, rows, i);
    const int col = i - first[r];
    const int pid = c.table[static_cast<long long>(src[r]) * c.max_pages + col];
    if (pid < 0 || pid >= c.pages) {
      record_pages();
      continue;
    }
    c.table[static_cast<long long>(dst[r]) * c.max_pages + col] = pid;
    atomicAdd(c.refs + pid, 1);
  }
}

// Pages behind the first keep[b] tokens lose one reference (free at 0); len = min(len, keep).
__global__ void __launch_bounds__(COPY_THREADS) trim_kernel(Pool c, const int* slots, const int* keep, int B) {
  behind_last();
  const int b = blockIdx.x;
  const int slot = slots[b];
  if (slot == -1) return;
  const bool dup = named_before(slots, b, slot);
  if (slot < 0 || slot >= c.slots || dup) {
    if (threadIdx.x == 0) record_pages();
    return;
  }
  const int len = c.lens[slot], kept = keep ? keep[b] : 0;
  if (len < 0 || kept < 0 || len > c.max_pages * static_cast<long long>(c.page)) {
    if (threadIdx.x == 0) record_pages();
    return;
  }
  if (kept >= len) return;
  __syncthreads();   // every thread has read the length
  const int have = (len + c.page - 1) / c.page, stay = (kept + c.page - 1) / c.page;
  int* row = c.table + static_cast<long long>(slot) * c.max_pages;
  for (int j = stay + threadIdx.x; j < have; j += COPY_THREADS) {
    const int pid = row[j];
    row[j] = -1;
    if (pid < 0 || pid >= c.pages || atomicSub(c.refs + pid, 1) <= 0) record_pages();
  }
  if (threadIdx.x == 0) c.lens[slot] = kept;
}

// Live pages at or above n_live (the number of live pages), in order, go to the holes below it.
__global__ void __launch_bounds__(PLAN_THREADS)
    compact_plan_kernel(Pool c, Plan* plan, int* holes, int* movers, int* moved_to) {
  behind_last();
  __shared__ int warp_sum[33];
  int live = 0;
  for (int base = threadIdx.x * SWEEP; base < c.pages; base += PLAN_THREADS * SWEEP)
#pragma unroll
    for (int i = 0; i < SWEEP; ++i) live += base + i < c.pages && c.refs[base + i] != 0;
  int n_live;
  block_scan(live, warp_sum, n_live);
  const int n = list_pages(c.refs, 0, n_live, true, c.pages, holes, warp_sum);
  list_pages(c.refs, n_live, c.pages, false, n, movers, warp_sum);
  __syncthreads();
  for (int p = threadIdx.x; p < c.pages; p += PLAN_THREADS) moved_to[p] = p < n_live ? p : -1;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += PLAN_THREADS) {
    const int from = movers[i], to = holes[i];
    moved_to[from] = to;
    c.refs[to] = c.refs[from];
    c.refs[from] = 0;
  }
  if (threadIdx.x == 0) plan->pairs = n;
}

// Copies pages src -> dst of the plan's pairs in all layers, keys, values and scales, in units of
// COPY_BYTES that the blocks share out; sources and destinations are disjoint.  With moved_to, the
// page table is renumbered by it in the same launch.
__global__ void __launch_bounds__(COPY_THREADS)
    copy_pages_kernel(Pool c, const Plan* plan, const int* src, const int* dst, int stride, const int* moved_to) {
  behind_last();
  const int n_pairs = plan->pairs;
  if (moved_to && n_pairs > 0) {
    const long long n = static_cast<long long>(c.slots) * c.max_pages;
    for (long long i = static_cast<long long>(blockIdx.x) * COPY_THREADS + threadIdx.x; i < n;
         i += static_cast<long long>(gridDim.x) * COPY_THREADS) {
      const int pid = c.table[i];
      if (pid >= 0 && pid < c.pages) {
        const int to = moved_to[pid];
        if (to >= 0 && to != pid) c.table[i] = to;
      }
    }
  }
  const long long page_bytes = static_cast<long long>(c.heads) * c.page * c.Dh;
  const int chunks = static_cast<int>((page_bytes + COPY_BYTES - 1) / COPY_BYTES);
  const long long units = static_cast<long long>(n_pairs) * c.layers * 2 * chunks;
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const int chunk = static_cast<int>(u % chunks);
    const long long rest = u / chunks;
    const int kv = static_cast<int>(rest & 1);
    const long long lp = rest >> 1;
    const int layer = static_cast<int>(lp % c.layers);
    const int pair = static_cast<int>(lp / c.layers);
    const long long from = static_cast<long long>(layer) * c.pages + src[pair * stride];
    const long long to = static_cast<long long>(layer) * c.pages + dst[pair * stride];
    uint8_t* pool = kv ? c.v : c.k;
    const uint4* a = reinterpret_cast<const uint4*>(pool + from * page_bytes);
    uint4* z = reinterpret_cast<uint4*>(pool + to * page_bytes);
    const int end = static_cast<int>(min(page_bytes / 16, static_cast<long long>(chunk + 1) * (COPY_BYTES / 16)));
    const int i0 = chunk * (COPY_BYTES / 16) + threadIdx.x;
    constexpr int N = COPY_BYTES / 16 / COPY_THREADS;
    uint4 x[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i0 + i * COPY_THREADS < end) x[i] = a[i0 + i * COPY_THREADS];
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i0 + i * COPY_THREADS < end) z[i0 + i * COPY_THREADS] = x[i];
    if (chunk == 0) {
      float* sc = kv ? c.v_scale : c.k_scale;
      for (int h = threadIdx.x; h < c.heads; h += COPY_THREADS) sc[to * c.heads + h] = sc[from * c.heads + h];
    }
  }
}

}  // namespace cache
}  // namespace ra
