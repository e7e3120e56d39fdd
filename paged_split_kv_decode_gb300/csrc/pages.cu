// Pages of a paged cache: forking, freeing, compacting and copying them (the contract is in include/psd.h).
//
// Which pages are free is what their reference counts say, so there is no free list to keep: a call that
// needs n pages takes the n lowest free ids.  The tables and counts are worked on by one cluster of 8 CTAs
// in phases that its barriers divide: 65536 pages' counts are 8 a thread, and a barrier of the cluster takes
// a fraction of what a launch or a grid's barrier does.  All sums are of integers, so that the order of the
// atomics shows nowhere.  Counts are worked on in the workspace and written when the call is known to go
// through: a call that cannot writes nothing.  The pages' bytes are moved by a second kernel over all SMs.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <numeric>

#include "context.h"
#include "device.cuh"
#include "kernels.h"

namespace psd {

namespace {

constexpr int kCtas = 8, kThreads = 1024, kAll = kCtas * kThreads, kWarps = kAll / 32;
constexpr int kPoolsALaunch = 128;

// The workspace: a header, then lists of 32-bit numbers.
struct Header {
  int32_t moves;                  // entries of the list of moves
  int32_t accepted;               // 0: the call has been refused
  int32_t pad[14];
  long long totals[8][kCtas];     // one row for each exchange between the CTAs
  uint32_t faults[8][kCtas];
};
constexpr size_t kHeaderBytes = 2048;
static_assert(sizeof(Header) <= kHeaderBytes, "header");

struct Lists {
  Header *head;
  int32_t *count;   // [num_pages] the reference counts as the call leaves them
  int32_t *first;   // [num_pages] fork: the first child that may keep the page; compact: the new id
  int32_t *fresh;   // [num_pages] fork: free pages in order; compact: the counts of the pages that move
  int32_t *start;   // [num_new + 1] fork: where a child's pages begin in the new table
  int4 *rows;       // [num_new + 1] fork: a child's parent's row, pages handed down, its own row, its fresh pages
  int2 *moves;      // [max(num_new, num_pages / 2) + 1] source and destination; source < 0: none
};
size_t lists_of(Lists *l, void *base, int64_t num_pages, int64_t num_new) {
  uint8_t *at = static_cast<uint8_t *>(base);
  auto take = [&](size_t bytes) {
    uint8_t *p = at;
    at += (bytes + 255) / 256 * 256;
    return p;
  };
  Lists x;
  x.head = reinterpret_cast<Header *>(take(kHeaderBytes));
  x.count = reinterpret_cast<int32_t *>(take(size_t(num_pages) * 4));
  x.first = reinterpret_cast<int32_t *>(take(size_t(num_pages) * 4));
  x.fresh = reinterpret_cast<int32_t *>(take(size_t(num_pages) * 4));
  x.start = reinterpret_cast<int32_t *>(take(size_t(num_new + 1) * 4));
  x.rows = reinterpret_cast<int4 *>(take(size_t(num_new + 1) * 16));
  x.moves = reinterpret_cast<int2 *>(take(size_t(std::max(num_new, num_pages / 2) + 1) * 8));
  if (l) *l = x;
  return size_t(at - static_cast<uint8_t *>(base));
}

struct ForkParams {
  Lists w;
  const int32_t *parents, *indptr, *indices, *kv_len, *ref;
  int32_t *new_ref, *new_indptr, *new_indices, *new_len, *fault;
  int64_t num_indices, num_pages, capacity;
  int N, B, P, room, release;
};

// ------------------------------------------------------------------------------------- the cluster
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The cluster's threads, numbered through.
struct Team {
  Header *head;
  int id, rank, turn = 0;
  long long *sums;  // [33] shared
  __device__ Team(Header *h, long long *s) : head(h), rank(int(cluster_rank())), sums(s) { id = rank * kThreads + threadIdx.x; }
  // The sum of `v` over the threads before this one, and over all; `faults` of all are or-ed.  A barrier of
  // the cluster: what its threads wrote before is there for all behind it.
  __device__ long long scan(long long v, long long &total, uint32_t &faults) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long up = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, up, d);
      if (lane >= d) up += x;
    }
    const uint32_t warp_faults = __reduce_or_sync(0xffffffffu, faults);
    const bool any = __syncthreads_or(int(warp_faults)) != 0;  // (and `sums` is free)
    if (lane == 31) sums[warp] = up;
    uint32_t *bits = reinterpret_cast<uint32_t *>(sums + 32);
    if (any && threadIdx.x == 0) *bits = 0;
    __syncthreads();
    if (any) {
      if (lane == 0 && warp_faults) atomicOr(bits, warp_faults);
      __syncthreads();
    }
    if (warp == 0) {
      long long x = sums[lane];
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
      }
      sums[lane] = x;
      if (lane == 31) {
        head->totals[turn][rank] = x;
        head->faults[turn][rank] = any ? *bits : 0u;
      }
    }
    cluster_sync();
    long long before = 0;
    total = 0;
    faults = 0;
#pragma unroll
    for (int c = 0; c < kCtas; ++c) {
      const long long x = __ldcg(&head->totals[turn][c]);
      faults |= __ldcg(&head->faults[turn][c]);
      if (c < rank) before += x;
      total += x;
    }
    ++turn;
    return before + (warp ? sums[warp - 1] : 0) + up - v;
  }
};

// ---------------------------------------------------------------------------------------------- fork
// A child: its parent's pages that it takes over whole, whether it has a part-full one, and what it wants.
struct Child {
  int first, full, want, len;  // first: of the parent's row; want < 0: the child is refused
  bool tail;
};
__device__ __forceinline__ Child child_of(const ForkParams &p, int parent, uint32_t &faults) {
  Child c{0, 0, 0, 0, false};
  if (parent == -1) return c;
  if (parent < 0 || parent >= p.B) {
    faults |= PSD_FAULT_RANGE;
    return c;
  }
  c.first = p.indptr[parent];
  c.len = p.kv_len[parent];
  const int held = (c.len - 1) / p.P + (c.len > 0);  // pages
  const int64_t want = (int64_t(c.len) + p.room + p.P - 1) / p.P;
  if (c.len < 0 || c.first < 0 || int64_t(c.first) + held > p.indptr[parent + 1] || p.indptr[parent + 1] > p.num_indices ||
      int64_t(c.len) + p.room > 0x7fffffff) {
    faults |= PSD_FAULT_RANGE;
    return Child{0, 0, 0, 0, false};
  }
  c.full = c.len / p.P;
  c.tail = c.len % p.P != 0;
  c.want = int(want);
  return c;
}

__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads, 1) fork_kernel(const ForkParams p) {
  __shared__ long long sums[33];
  dependents_may_launch();
  Team team(p.w.head, sums);
  const int id = team.id, lane = threadIdx.x & 31, warp = id >> 5;
  // Children in runs, pages in runs: a run a thread, so that sums over the threads before give their places.
  const int run = (p.N + kAll - 1) / kAll, i0 = min(p.N, id * run), i1 = min(p.N, i0 + run);
  const int64_t stretch = (p.num_pages + kAll - 1) / kAll;
  const int64_t g0 = min(p.num_pages, id * stretch), g1 = min(p.num_pages, g0 + stretch);
  uint32_t faults = 0;
  long long total;

  // The children's wants; the counts to work on.
  long long want = 0;
  for (int i = i0; i < i1; ++i) want += child_of(p, p.parents[i], faults).want;
  const int64_t old_end = p.B > 0 ? p.indptr[p.B] : 0, old_begin = p.B > 0 ? p.indptr[0] : 0;
  if (old_begin < 0 || old_end < old_begin || old_end > p.num_indices) faults |= PSD_FAULT_RANGE;
  for (int64_t g = id; g < p.num_pages; g += kAll) {
    const int r = p.ref[g];
    if (r < 0) faults |= PSD_FAULT_RANGE;
    p.w.count[g] = r;
    p.w.first[g] = INT_MAX;
  }
  {
    long long at = team.scan(want, total, faults);
    for (int i = i0; i < i1; ++i) {
      uint32_t none = 0;
      p.w.start[i] = int(at);
      at += child_of(p, p.parents[i], none).want;
    }
  }
  if (total > p.capacity) faults |= PSD_FAULT_RANGE;
  const int pages_wanted = int(min(total, 0x7fffffffLL));

  // The old requests let go of their pages.
  if (!faults)
    for (int64_t e = old_begin + id; e < old_end; e += kAll) {
      const int g = p.indices[e];
      if (g < 0 || g >= p.num_pages) faults |= PSD_FAULT_PAGE_ID;
      else if (p.release) atomicSub(p.w.count + g, 1);
    }
  team.scan(0, total, faults);

  if (!faults)
    for (int64_t g = id; g < p.num_pages; g += kAll)
      if (__ldcg(p.w.count + g) < 0) faults |= PSD_FAULT_RANGE;  // referred to more often than counted
  team.scan(0, total, faults);

  // Pages handed down whoever else has them are counted.
  const int parts = max(1, kWarps / max(p.N, 1));  // warps a child
  if (!faults)
    for (int u = warp; u < p.N * parts; u += kWarps) {
      const Child c = child_of(p, p.parents[u / parts], faults);
      const int down = c.full + (c.tail && !p.room);
      for (int j = (u % parts) * 32 + lane; j < down; j += 32 * parts) {
        const int g = p.indices[c.first + j];
        if (g < 0 || g >= p.num_pages) faults |= PSD_FAULT_PAGE_ID;  // (behind the old table's end)
        else atomicAdd(p.w.count + g, 1);
      }
    }
  team.scan(0, total, faults);

  // A part-full page that will be written to, and that nothing else refers to (not as a full page either), goes to its first
  // child.
  if (!faults && p.room)
    for (int i = i0; i < i1; ++i) {
      const Child c = child_of(p, p.parents[i], faults);
      if (!c.tail) continue;
      const int g = p.indices[c.first + c.full];
      if (g < 0 || g >= p.num_pages) faults |= PSD_FAULT_PAGE_ID;
      else if (__ldcg(p.w.count + g) == 0) atomicMin(p.w.first + g, i);
    }
  team.scan(0, total, faults);

  // Pages to be found are numbered.
  auto keeps = [&](const Child &c, int i) {
    return c.tail && (!p.room || __ldcg(p.w.first + p.indices[c.first + c.full]) == i);
  };
  long long blanks = 0, all_blanks;
  if (!faults)
    for (int i = i0; i < i1; ++i) {
      const Child c = child_of(p, p.parents[i], faults);
      const bool kept = keeps(c, i);
      blanks += c.want - c.full - kept;
      if (p.room && kept) p.w.count[p.indices[c.first + c.full]] = 1;
    }
  {
    long long at = team.scan(blanks, all_blanks, faults);
    if (!faults)
      for (int i = i0; i < i1; ++i) {
        const Child c = child_of(p, p.parents[i], faults);
        const int kept = c.full + keeps(c, i);
        p.w.rows[i] = make_int4(c.first, kept, p.w.start[i], int(at));
        at += c.want - kept;
      }
  }

  // The free pages, lowest first.
  long long free_pages = 0;
  if (!faults)
    for (int64_t g = g0; g < g1; ++g) free_pages += __ldcg(p.w.count + g) == 0;
  {
    long long at = team.scan(free_pages, total, faults);
    if (total < all_blanks) faults |= PSD_FAULT_NO_PAGES;
    if (!faults)
      for (int64_t g = g0; g < g1; ++g) {
        const int n = __ldcg(p.w.count + g);
        const bool taken = n == 0 && at < all_blanks;
        if (taken) p.w.fresh[at] = int(g);
        at += n == 0;
        p.new_ref[g] = taken ? 1 : n;
      }
  }
  if (faults) {  // the same for all
    if (id == 0) {
      atomicOr(p.fault, int32_t(faults));
      p.w.head->moves = p.w.head->accepted = 0;
    }
    return;
  }
  cluster_sync();

  for (int i = i0; i < i1; ++i) {
    const Child c = child_of(p, p.parents[i], faults);
    const int4 r = p.w.rows[i];
    p.new_indptr[i] = r.z;
    p.new_len[i] = c.want ? c.len + p.room : 0;
    p.w.moves[i] = c.tail && r.y == c.full ? make_int2(p.indices[c.first + c.full], __ldcg(p.w.fresh + r.w)) : make_int2(-1, -1);
  }
  if (id == 0) {
    if (p.new_indptr) p.new_indptr[p.N] = pages_wanted;
    p.w.head->moves = p.N;
    p.w.head->accepted = 1;
  }
}

// The same by one CTA with the counts in shared memory, for up to kFewChildren children, kFewPages pages and
// kFewEntries new entries: its barriers and atomics take tens of cycles where the cluster's take hundreds.  Counts and the old
// table come by asynchronous copies while the children are looked up (with a load at a time the kernel took 20 us where it
// takes 11, caches cold).  It is bound by one SM's atomics, one or two a table entry and 6 to 9 cycles for 32 of them, and by
// the latency of what depends on what.  A whole call, copies included: 4 children of 40 pages 8 us against 20; 128 of some
// 150 pages each 19 us against 32.  At the border, 128 children of some 145 pages and 4 pools: 49152 pages 25 us, 49153, by the
// cluster, 37; 200000 pages 67.  Letting go of such a table alone: 8 us of 3100 pages, 15 of 49152, 27 and 58 by the cluster.
constexpr int kFewChildren = 1024, kFewPages = 49152, kFewEntries = (1 << 21) - 2;

__device__ __forceinline__ int block_scan(int v, int &total, int *sums) {  // the sum over the threads before
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int up = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, up, d);
    if (lane >= d) up += x;
  }
  __syncthreads();  // (sums are free)
  if (lane == 31) sums[warp] = up;
  __syncthreads();
  int x = sums[lane];
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  total = __shfl_sync(0xffffffffu, x, 31);
  const int before = __shfl_sync(0xffffffffu, x, warp ? warp - 1 : 0);
  return (warp ? before : 0) + up - v;
}

// Shared memory: the counts, padded to kRun, the rows, and the old table's entries where they fit.
constexpr int kRun = 128;  // pages of a warp's turn, four a lane
constexpr size_t kFewShared = 227 * 1024 - 1024;
size_t few_shared(int64_t num_pages, int num_new, int64_t num_indices) {
  const size_t least = size_t((num_pages + kRun - 1) / kRun * kRun) * 4 + size_t(num_new + 1) / 2 * 16;
  return std::min(kFewShared, least + size_t(num_indices) * 4 + 16);
}
static_assert(kFewPages % kRun == 0 && kFewPages * 4 + kFewChildren * 8 <= kFewShared, "counts and rows fit");

__device__ __forceinline__ uint32_t shared_address(const void *at) { return uint32_t(__cvta_generic_to_shared(at)); }
// n numbers to shared memory, without waiting: 16 bytes at a time where both lie so, all threads.
__device__ __forceinline__ void bring(int *dst, const int32_t *src, int n) {
  int i = threadIdx.x;
  if ((reinterpret_cast<uintptr_t>(src) & 15) == 0 && (shared_address(dst) & 15) == 0) {
    for (; i < n / 4; i += kThreads)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(shared_address(dst + 4 * i)), "l"(src + 4 * i) : "memory");
    i = n / 4 * 4 + threadIdx.x;
  }
  for (; i < n; i += kThreads)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(shared_address(dst + i)), "l"(src + i) : "memory");
}

__global__ void __launch_bounds__(kThreads, 1) fork_few_kernel(const ForkParams p, int shared_entries, int spread) {
  extern __shared__ __align__(16) int count[];  // [num_pages], then the rows, then the entries
  __shared__ int sums[32], n_moves;
  const int padded = int((p.num_pages + kRun - 1) / kRun * kRun);
  int2 *rows = reinterpret_cast<int2 *>(count + padded);
  dependents_may_launch();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n_pages = int(p.num_pages);
  uint32_t faults = 0;
  int total;
  // The counts and the old table's entries are on their way while the children are looked up.
  int old_end = p.B > 0 ? p.indptr[p.B] : 0, old_begin = p.B > 0 ? p.indptr[0] : 0;
  const int parent = tid < p.N ? p.parents[tid] : -1;
  bring(count, p.ref, n_pages);
  if (tid == 0) n_moves = 0;
  for (int g = n_pages + tid; g < padded; g += kThreads) count[g] = 1;
  const Child looked_up = child_of(p, parent, faults);
  if (old_begin < 0 || old_end < old_begin || old_end > p.num_indices) {
    faults |= PSD_FAULT_RANGE;
    old_begin = old_end = 0;
  }
  // (from the last 16-byte border before them, so that the wide copies fit)
  int before = int(reinterpret_cast<uintptr_t>(p.indices + old_begin) / 4 & 3);
  if (before > old_begin) before = 0;
  const bool staged = old_end - old_begin <= shared_entries - before;
  int *entries = reinterpret_cast<int *>(rows + (p.N + 1) / 2 * 2);
  if (staged) bring(entries, p.indices + (old_begin - before), old_end - old_begin + before);
  const int *entry0 = entries + before - old_begin;
  auto entry = [&](int e) { return staged && e >= old_begin && e < old_end ? entry0[e] : p.indices[e]; };
  Child c = looked_up;
  // (of wants that do not fit into the new table the sum only has to stay too large)
  const int start = block_scan(int(min(int64_t(c.want), p.capacity + 1)), total, sums);
  if (total > p.capacity) faults |= PSD_FAULT_RANGE;
  // Everybody's faults: from here on all go the same way.
  auto together = [&]() {
    const uint32_t x = __reduce_or_sync(0xffffffffu, faults);
    faults = uint32_t(__syncthreads_or(int(x & 1)) ? 1 : 0);
    faults |= __syncthreads_or(int(x & 2)) ? 2u : 0u;
    faults |= __syncthreads_or(int(x & 4)) ? 4u : 0u;
    faults |= __syncthreads_or(int(x & 8)) ? 8u : 0u;
    return faults != 0;
  };
  auto give_up = [&]() {
    if (tid == 0) {
      atomicOr(p.fault, int32_t(faults));
      p.w.head->moves = p.w.head->accepted = 0;
    }
  };
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  int tail = 0;
  if (c.tail) {
    tail = entry(c.first + c.full);
    if (tail < 0 || tail >= n_pages) faults |= PSD_FAULT_PAGE_ID, c.tail = false;
  }
  if (tid < p.N) rows[tid] = make_int2(c.first, c.full + (c.tail && !p.room));  // what is handed down whoever else has it
  // The old requests let go of their pages.
  auto let_go = [&](const int *at, int n) {
#pragma unroll 4
    for (uint32_t e = tid; e < uint32_t(n); e += kThreads) {
      const int g = at[e];
      if (uint32_t(g) >= uint32_t(n_pages)) faults |= PSD_FAULT_PAGE_ID;
      else if (p.release) atomicSub(count + g, 1);
    }
  };
  if (staged) let_go(entries + before, old_end - old_begin);
  else let_go(p.indices + old_begin, old_end - old_begin);
  __syncthreads();
  int4 *const count4 = reinterpret_cast<int4 *>(count);
  for (int k = tid; k < padded / 4; k += kThreads) {
    const int4 r = count4[k];
    if ((r.x | r.y | r.z | r.w) < 0) faults |= PSD_FAULT_RANGE;  // below 0, or referred to more often than counted
  }
  if (__syncthreads_or(faults != 0)) {
    together();
    give_up();
    return;
  }
  // Pages handed down are counted.
  const int parts = max(1, kThreads / 32 / max(p.N, 1));  // warps a child
  // (Children that share pages, neighbours mostly, are not taken at the same time: their atomics would meet.)
  for (int x = warp; x < p.N * parts; x += kThreads / 32) {
    const int u = parts == 1 ? x * spread % p.N : x;
    const int2 r = rows[parts == 1 ? u : u / parts];
    auto take = [&](const int *at) {  // (in shared memory a third of the instructions)
#pragma unroll 1
      for (int j = (parts == 1 ? 0 : u % parts) * 32 + lane; j < r.y; j += 32 * parts) {
        const int g = at[j];
        if (uint32_t(g) >= uint32_t(n_pages)) faults |= PSD_FAULT_PAGE_ID;  // (behind the old table's end)
        else atomicAdd(count + g, 1);
      }
    };
    if (staged && r.x >= old_begin && r.x + r.y <= old_end) take(entries + before + (r.x - old_begin));
    else take(p.indices + r.x);
  }
  __syncthreads();
  // A part-full page that will be written to, and that nothing else refers to (not as a full page either), goes to its first
  // child: the least child, below 0, stands in its count.
  const bool claims = c.tail && p.room && count[tail] == 0;
  __syncthreads();
  if (claims) atomicMin(count + tail, tid - kFewChildren);
  __syncthreads();
  const bool mine = claims && count[tail] == tid - kFewChildren;
  const bool kept_tail = c.tail && (!p.room || mine), copies = c.tail && !kept_tail;
  const int move = copies ? atomicAdd(&n_moves, 1) : 0;  // (the order of the moves shows nowhere)
  __syncthreads();
  if (mine) count[tail] = 1;
  const int kept = c.full + kept_tail;
  int all_blanks;
  const int blank = block_scan(c.want - kept, all_blanks, sums);  // (with barriers: the counts are complete)
  if (tid < p.N) p.w.rows[tid] = make_int4(c.first, kept, start, blank);
  // The free pages, lowest first: a warp has a stretch of them, kRun at a time.
  const int runs = padded / kRun, each = (runs + 31) / 32, run0 = warp * each, run1 = min(runs, run0 + each);
  int free_pages = 0;
  for (int k = run0; k < run1; ++k) {
    const int4 r = count4[32 * k + lane];
    free_pages += (r.x == 0) + (r.y == 0) + (r.z == 0) + (r.w == 0);
  }
  free_pages = __reduce_add_sync(0xffffffffu, free_pages);
  int at = block_scan(lane == 0 ? free_pages : 0, total, sums);
  at = __shfl_sync(0xffffffffu, at, 0);
  if (total < all_blanks) faults |= PSD_FAULT_NO_PAGES;
  if (__syncthreads_or(faults != 0)) {
    together();
    give_up();
    return;
  }
  const bool wide = (reinterpret_cast<uintptr_t>(p.new_ref) & 15) == 0;
  for (int k = run0; k < run1; ++k) {
    const int4 r = count4[32 * k + lane];
    const int g = kRun * k + 4 * lane;
    int of[4] = {r.x, r.y, r.z, r.w};
    uint32_t who[4];
    int rank = at, all = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      who[i] = __ballot_sync(0xffffffffu, of[i] == 0);
      rank += __popc(who[i] & ((1u << lane) - 1u));
      all += __popc(who[i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (of[i] == 0) {
        if (rank < all_blanks) p.w.fresh[rank] = g + i, of[i] = 1;
        ++rank;
      }
    at += all;
    if (wide && g + 4 <= n_pages) {
      *reinterpret_cast<int4 *>(p.new_ref + g) = make_int4(of[0], of[1], of[2], of[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (g + i < n_pages) p.new_ref[g + i] = of[i];
    }
  }
  __syncthreads();
  if (tid < p.N) {
    p.new_indptr[tid] = start;
    p.new_len[tid] = c.want ? c.len + p.room : 0;
    if (copies) p.w.moves[move] = make_int2(tail, p.w.fresh[blank]);
    if (tid == p.N - 1) p.new_indptr[p.N] = start + c.want;
  }
  if (tid == 0) {
    if (p.N == 0 && p.new_indptr) p.new_indptr[0] = 0;
    p.w.head->moves = n_moves;
    p.w.head->accepted = 1;
  }
}

// ------------------------------------------------------------------------------------------- compact
struct CompactParams {
  Lists w;
  const int32_t *indices, *ref;
  int32_t *new_indices, *new_ref, *num_live, *page_map, *fault;
  int64_t num_indices, num_pages;
};

__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads, 1) compact_kernel(const CompactParams p) {
  __shared__ long long sums[33];
  dependents_may_launch();
  Team team(p.w.head, sums);
  const int id = team.id;
  const int64_t stretch = (p.num_pages + kAll - 1) / kAll;
  const int64_t g0 = min(p.num_pages, id * stretch), g1 = min(p.num_pages, g0 + stretch);
  uint32_t faults = 0;
  long long n_live, total, mine = 0;
  for (int64_t g = g0; g < g1; ++g) {
    const int r = p.ref[g];
    if (r < 0) faults |= PSD_FAULT_RANGE;
    mine += r > 0;
  }
  for (int64_t e = id; e < p.num_indices; e += kAll) {
    const int g = p.indices[e];
    if (g < 0 || g >= p.num_pages || p.ref[g] <= 0) faults |= PSD_FAULT_PAGE_ID;
  }
  team.scan(mine, n_live, faults);
  if (faults) {
    if (id == 0) {
      atomicOr(p.fault, int32_t(faults));
      p.w.head->moves = p.w.head->accepted = 0;
    }
    return;
  }
  // Free pages among the first n_live (high half), live pages behind them: there are as many of each.
  long long both = 0;
  for (int64_t g = g0; g < g1; ++g) {
    const bool live = p.ref[g] > 0;
    both += g < n_live ? (live ? 0LL : 1LL << 32) : live;
  }
  const long long at = team.scan(both, total, faults);
  int hole = int(at >> 32), mover = int(at & 0xffffffff);
  for (int64_t g = g0; g < g1; ++g) {
    const int r = p.ref[g];
    p.w.count[g] = r;
    if (g < n_live && r == 0) p.w.moves[hole++].y = int(g);
    if (g >= n_live && r > 0) {
      p.w.fresh[mover] = r;
      p.w.first[g] = mover;
      p.w.moves[mover++].x = int(g);
    }
  }
  cluster_sync();
  hole = int(at >> 32);
  for (int64_t g = g0; g < g1; ++g) {
    const int r = p.w.count[g];
    p.new_ref[g] = g >= n_live ? 0 : r > 0 ? r : __ldcg(p.w.fresh + hole++);
    if (p.page_map) p.page_map[g] = r == 0 ? -1 : g < n_live ? int(g) : __ldcg(&p.w.moves[p.w.first[g]].y);
  }
  for (int64_t e = id; e < p.num_indices; e += kAll) {
    const int g = p.indices[e];
    p.new_indices[e] = g < n_live ? g : __ldcg(&p.w.moves[__ldcg(p.w.first + g)].y);
  }
  if (id == 0) {
    *p.num_live = int(n_live);
    p.w.head->accepted = 1;
    p.w.head->moves = int(total & 0xffffffff);
  }
}

// ---------------------------------------------------------------------------------------------- copy
struct CopyPools {
  psd_page_pool pool[kPoolsALaunch];
};
struct CopyParams {
  const Header *head;         // how many entries there are, or
  const int32_t *src, *dst;   // lists of a caller's, n long
  const int2 *moves;
  int32_t *fault;
  int64_t num_pages;
  int n, pools, parts;        // parts of a page of a pool
  // a new table to be written first, if there are children
  int children;
  const int4 *rows;
  const int32_t *new_indptr, *indices, *fresh;
  int32_t *new_indices;
};

// A CTA takes a part of a page of one pool at a time, of 16 KB so that few large pages keep all SMs busy: 16 bytes a thread and
// access, four of them on their way.  Its next part's place is added up, not divided out (a third of the instructions).  The
// last CTAs, which may have a part less, write the new table's rows first.  (Here and not in the kernel before: 152 SMs write
// them beside the copies.)  Bound by DRAM: 14700 pages of 16 KB in 75 us, 0.97 of the copy rate; 36 to 45 moves in 32 pools, 18 to 23 MB
// read, in 12 us, where the chain from the list to the last store shows.
constexpr int kPart = 16384;
__global__ void __launch_bounds__(256) copy_pages_kernel(const CopyParams p, const __grid_constant__ CopyPools pools) {
  const int per = p.pools * p.parts, first = per ? int(blockIdx.x) / per : 0;
  wait_for_prior_grid();
  // (the first move on its way beside the number of them: the list has an entry for every CTA)
  const int2 first_move = p.moves ? __ldcg(p.moves + first) : make_int2(0, 0);
  const int n = p.head ? __ldcg(&p.head->moves) : p.n;
  if (p.children > 0 && __ldcg(&p.head->accepted))
    for (int i = gridDim.x - 1 - blockIdx.x; i < p.children; i += gridDim.x) {
      const int4 r = __ldcg(p.rows + i);
      const int want = __ldcg(p.new_indptr + i + 1) - r.z;
#pragma unroll 4
      for (int j = threadIdx.x; j < want; j += 256)
        p.new_indices[r.z + j] = j < r.y ? p.indices[r.x + j] : __ldcg(p.fresh + r.w + j - r.y);
    }
  if (per == 0) return;
  const int step = int(gridDim.x) / per, step_rest = int(gridDim.x) - step * per;
  for (int i = first, rest = int(blockIdx.x) - first * per, turn = 0; i < n; ++turn) {
    const int which = p.parts == 1 ? rest : rest / p.parts, part = rest - which * p.parts;
    const psd_page_pool pool = pools.pool[which];
    int2 m = first_move;
    bool good = true;
    if (!p.moves) {
      m = make_int2(p.src[i], p.dst[i]);
      good = m.x >= 0 && m.x < p.num_pages && m.y >= 0 && m.y < p.num_pages;
      if (!good && threadIdx.x == 0) atomicOr(p.fault, PSD_FAULT_PAGE_ID);
    } else if (turn > 0) {
      m = __ldcg(p.moves + i);
    }
    if (good && m.x >= 0 && m.x != m.y) {
      const bool wide = ((reinterpret_cast<uintptr_t>(pool.base) | uint64_t(pool.page_bytes)) & 15) == 0;
      const int64_t size = wide ? pool.page_bytes / 16 : pool.page_bytes;  // words, or bytes
      const int64_t each = p.parts == 1 ? size : max(int64_t(wide ? kPart / 16 : kPart), (size + p.parts - 1) / p.parts);
      const int64_t begin = part * each;
      const int left = int(min(size - begin, each));                       // (none, where the pool's pages are smaller)
      const uint8_t *base = static_cast<const uint8_t *>(pool.base);
      if (wide) {
        const uint4 *x = reinterpret_cast<const uint4 *>(base + int64_t(m.x) * pool.page_bytes) + begin + threadIdx.x;
        uint4 *y = reinterpret_cast<uint4 *>(const_cast<uint8_t *>(base + int64_t(m.y) * pool.page_bytes)) + begin + threadIdx.x;
        int k = threadIdx.x;
        for (; k + 768 < left; k += 1024, x += 1024, y += 1024) {
          uint4 w[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) w[c] = __ldcs(x + 256 * c);
#pragma unroll
          for (int c = 0; c < 4; ++c) y[256 * c] = w[c];
        }
        for (; k < left; k += 256, x += 256, y += 256) *y = __ldcs(x);
      } else {
        const uint8_t *x = base + int64_t(m.x) * pool.page_bytes + begin;
        uint8_t *y = const_cast<uint8_t *>(base + int64_t(m.y) * pool.page_bytes) + begin;
        for (int k = threadIdx.x; k < left; k += 256) y[k] = x[k];
      }
    }
    i += step, rest += step_rest;
    if (rest >= per) ++i, rest -= per;
  }
}

// One or more launches over all pools, behind the kernel that makes the list (or not).
psd_status launch_copy(CopyParams p, const psd_page_pool *pools, int num_pools, int64_t most, bool behind, const DeviceInfo &dev,
                       cudaStream_t s) {
  for (int k = 0; (k < num_pools && most > 0) || p.children > 0; k += kPoolsALaunch) {
    CopyPools c;
    p.pools = most > 0 ? std::min(kPoolsALaunch, num_pools - k) : 0;
    std::copy(pools + k, pools + k + p.pools, c.pool);
    int64_t page = 1;
    for (int i = 0; i < p.pools; ++i) page = std::max(page, c.pool[i].page_bytes);
    p.parts = int(std::min<int64_t>((page + kPart - 1) / kPart, 1024));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(std::min<int64_t>(std::max<int64_t>(most * p.pools * p.parts, p.children), int64_t(dev.num_sms) * 8)));
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = behind && k == 0 ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, copy_pages_kernel, p, c);
    if (e != cudaSuccess) return fail(PSD_ERR_CUDA, "copy_pages launch: %s", cudaGetErrorString(e));
    p.children = 0;
  }
  return PSD_OK;
}

psd_status check_pools(const char *what, const psd_page_pool *pools, int32_t num_pools, int64_t num_pages) {
  if (num_pages < 1 || num_pages > 0x7fffffffLL) return fail(PSD_ERR_INVALID_ARG, "%s: num_pages %lld", what, (long long)num_pages);
  if (num_pools < 0 || (num_pools > 0 && !pools)) return fail(PSD_ERR_INVALID_ARG, "%s: pools", what);
  for (int32_t i = 0; i < num_pools; ++i)
    if (!pools[i].base || pools[i].page_bytes < 1 || pools[i].page_bytes > (int64_t(1) << 40))
      return fail(PSD_ERR_INVALID_ARG, "%s: pool %d", what, i);
  return PSD_OK;
}

bool overlap(const void *a, int64_t na, const void *b, int64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && na > 0 && nb > 0 && x < y + uintptr_t(nb) * 4 && y < x + uintptr_t(na) * 4;
}

}  // namespace
}  // namespace psd

using namespace psd;

extern "C" size_t psd_pages_workspace_bytes(int64_t num_pages, int32_t num_new) {
  if (num_pages < 1 || num_new < 0) return 0;
  return lists_of(nullptr, nullptr, num_pages, num_new);
}

static psd_status fork_table(const char *what, psd_ctx *ctx, const psd_fork_args *a, void *workspace, size_t workspace_bytes, psd_stream_t stream) {
  clear_error();
  if (!ctx || !a) return fail(PSD_ERR_INVALID_ARG, "%s: NULL", what);
  const psd_status st = check_pools(what, a->pools, a->num_pools, a->num_pages);
  if (st != PSD_OK) return st;
  if (a->num_new < 0 || a->batch < 0 || a->num_page_indices < 0 || a->new_capacity < 0 || a->page_size < 1 || a->room < 0)
    return fail(PSD_ERR_INVALID_ARG, "%s: bad sizes", what);
  if (a->num_new > (1 << 24) || a->num_page_indices > 0x7fffffffLL || a->new_capacity > 0x7fffffffLL)
    return fail(PSD_ERR_UNSUPPORTED, "%s: more than 2^24 new requests or 2^31 - 1 table entries", what);
  if (!workspace || !aligned16(workspace)) return fail(PSD_ERR_INVALID_ARG, "%s: workspace must be 16-byte aligned", what);
  const size_t need = psd_pages_workspace_bytes(a->num_pages, a->num_new);
  if (workspace_bytes < need) return fail(PSD_ERR_WORKSPACE_TOO_SMALL, "%s: workspace %zu < %zu bytes", what, workspace_bytes, need);
  if (!a->ref_count || !a->new_ref_count || !a->fault_dev ||
      (a->batch > 0 && (!a->page_indptr || !a->kv_len || (a->num_page_indices > 0 && !a->page_indices))) ||
      (a->num_new > 0 && (!a->parents || !a->new_indptr || !a->new_len || (a->new_capacity > 0 && !a->new_indices))))
    return fail(PSD_ERR_INVALID_ARG, "%s: NULL pointer", what);
  if (overlap(a->page_indices, a->num_page_indices, a->new_indices, a->new_capacity) ||
      overlap(a->page_indptr, int64_t(a->batch) + 1, a->new_indptr, int64_t(a->num_new) + 1) ||
      overlap(a->kv_len, a->batch, a->new_len, a->num_new) || overlap(a->parents, a->num_new, a->new_len, a->num_new) ||
      overlap(a->parents, a->num_new, a->new_indptr, int64_t(a->num_new) + 1) ||
      overlap(a->parents, a->num_new, a->new_indices, a->new_capacity))
    return fail(PSD_ERR_INVALID_ARG, "%s: the new table overlaps the old one or the parents", what);
  if (a->ref_count != a->new_ref_count && overlap(a->ref_count, a->num_pages, a->new_ref_count, a->num_pages))
    return fail(PSD_ERR_INVALID_ARG, "%s: new_ref_count is ref_count, or apart from it", what);
  DeviceGuard g(ctx->dev.device);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  ForkParams p = {};
  lists_of(&p.w, workspace, a->num_pages, a->num_new);
  p.parents = a->parents;
  p.indptr = a->page_indptr;
  p.indices = a->page_indices;
  p.kv_len = a->kv_len;
  p.ref = a->ref_count;
  p.new_ref = a->new_ref_count;
  p.new_indptr = a->new_indptr;
  p.new_indices = a->new_indices;
  p.new_len = a->new_len;
  p.fault = a->fault_dev;
  p.num_indices = a->num_page_indices;
  p.num_pages = a->num_pages;
  p.capacity = a->new_capacity;
  p.N = a->num_new;
  p.B = a->batch;
  p.P = a->page_size;
  p.room = a->room;
  p.release = a->keep_old == 0;
  cudaError_t e = cudaSuccess;
  if (a->num_new <= kFewChildren && a->num_pages <= kFewPages && a->new_capacity <= kFewEntries) {
    static std::atomic<uint64_t> ready{0};
    const uint64_t bit = ctx->dev.device < 64 ? uint64_t(1) << ctx->dev.device : 0;
    if (!(ready.load(std::memory_order_acquire) & bit)) {
      e = cudaFuncSetAttribute(fork_few_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kFewShared));
      if (e != cudaSuccess) return fail(PSD_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
      ready.fetch_or(bit, std::memory_order_release);
    }
    const size_t shared = few_shared(a->num_pages, a->num_new, a->num_page_indices), least = few_shared(a->num_pages, a->num_new, 0);
    int spread = std::max(1, a->num_new * 3 / 8);
    while (std::gcd(spread, a->num_new) > 1) ++spread;
    fork_few_kernel<<<1, kThreads, shared, s>>>(p, int((shared - least + 16) / 4), spread);
  } else {
    fork_kernel<<<kCtas, kThreads, 0, s>>>(p);
  }
  e = cudaGetLastError();
  if (e != cudaSuccess) return fail(PSD_ERR_CUDA, "fork_pages launch: %s", cudaGetErrorString(e));
  CopyParams c = {};
  c.head = p.w.head;
  c.moves = p.w.moves;
  c.fault = a->fault_dev;
  c.num_pages = a->num_pages;
  c.children = a->num_new;
  c.rows = p.w.rows;
  c.new_indptr = a->new_indptr;
  c.indices = a->page_indices;
  c.fresh = p.w.fresh;
  c.new_indices = a->new_indices;
  return launch_copy(c, a->pools, a->num_pools, a->room > 0 ? a->num_new : 0, true, ctx->dev, s);
}

extern "C" psd_status fork_pages(psd_ctx *ctx, const psd_fork_args *a, void *workspace, size_t workspace_bytes,
                                 psd_stream_t stream) {
  return fork_table("fork_pages", ctx, a, workspace, workspace_bytes, stream);
}

extern "C" psd_status free_pages(psd_ctx *ctx, const int32_t *page_indptr, const int32_t *page_indices, int64_t num_page_indices,
                                 int32_t batch, int32_t *ref_count, int64_t num_pages, int32_t *fault_dev, void *workspace,
                                 size_t workspace_bytes, psd_stream_t stream) {
  psd_fork_args a = {};
  a.page_indptr = page_indptr;
  a.page_indices = page_indices;
  a.kv_len = page_indptr;  // (of no child: not read)
  a.num_page_indices = num_page_indices;
  a.batch = batch;
  a.page_size = 1;
  a.ref_count = ref_count;
  a.new_ref_count = ref_count;
  a.num_pages = num_pages;
  a.fault_dev = fault_dev;
  return fork_table("free_pages", ctx, &a, workspace, workspace_bytes, stream);
}

extern "C" psd_status compact_pages(psd_ctx *ctx, const psd_compact_args *a, void *workspace, size_t workspace_bytes,
                                    psd_stream_t stream) {
  clear_error();
  if (!ctx || !a) return fail(PSD_ERR_INVALID_ARG, "compact_pages: NULL");
  const psd_status st = check_pools("compact_pages", a->pools, a->num_pools, a->num_pages);
  if (st != PSD_OK) return st;
  if (a->num_page_indices < 0) return fail(PSD_ERR_INVALID_ARG, "compact_pages: num_page_indices");
  if (!workspace || !aligned16(workspace)) return fail(PSD_ERR_INVALID_ARG, "compact_pages: workspace must be 16-byte aligned");
  const size_t need = psd_pages_workspace_bytes(a->num_pages, 0);
  if (workspace_bytes < need) return fail(PSD_ERR_WORKSPACE_TOO_SMALL, "workspace %zu < %zu bytes", workspace_bytes, need);
  if (!a->ref_count || !a->new_ref_count || !a->num_live || !a->fault_dev ||
      (a->num_page_indices > 0 && (!a->page_indices || !a->new_indices)))
    return fail(PSD_ERR_INVALID_ARG, "compact_pages: NULL pointer");
  const struct {
    const int32_t *at;
    int64_t n;
  } inputs[2] = {{a->page_indices, a->num_page_indices}, {a->ref_count, a->num_pages}},
    outputs[4] = {{a->new_indices, a->num_page_indices}, {a->new_ref_count, a->num_pages}, {a->page_map, a->num_pages}, {a->num_live, 1}};
  for (int i = 0; i < 4; ++i) {
    bool bad = false;
    for (int j = 0; j < 2; ++j) bad |= !(i == j && outputs[i].at == inputs[j].at) && overlap(outputs[i].at, outputs[i].n, inputs[j].at, inputs[j].n);
    for (int j = 0; j < i; ++j) bad |= overlap(outputs[i].at, outputs[i].n, outputs[j].at, outputs[j].n);
    if (bad) return fail(PSD_ERR_INVALID_ARG, "compact_pages: an output is its input, or apart from all others");
  }
  DeviceGuard g(ctx->dev.device);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  CompactParams p = {};
  lists_of(&p.w, workspace, a->num_pages, 0);
  p.indices = a->page_indices;
  p.ref = a->ref_count;
  p.new_indices = a->new_indices;
  p.new_ref = a->new_ref_count;
  p.num_live = a->num_live;
  p.page_map = a->page_map;
  p.fault = a->fault_dev;
  p.num_indices = a->num_page_indices;
  p.num_pages = a->num_pages;
  compact_kernel<<<kCtas, kThreads, 0, s>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(PSD_ERR_CUDA, "compact_pages launch: %s", cudaGetErrorString(e));
  CopyParams c = {};
  c.head = p.w.head;
  c.moves = p.w.moves;
  c.fault = a->fault_dev;
  c.num_pages = a->num_pages;
  return launch_copy(c, a->pools, a->num_pools, a->num_pages / 2, true, ctx->dev, s);
}

extern "C" psd_status copy_pages(psd_ctx *ctx, const psd_page_pool *pools, int32_t num_pools, int64_t num_pages,
                                 const int32_t *src, const int32_t *dst, int32_t n, int32_t *fault_dev, psd_stream_t stream) {
  clear_error();
  if (!ctx) return fail(PSD_ERR_INVALID_ARG, "copy_pages: NULL");
  const psd_status st = check_pools("copy_pages", pools, num_pools, num_pages);
  if (st != PSD_OK) return st;
  if (n < 0) return fail(PSD_ERR_INVALID_ARG, "copy_pages: n %d", n);
  if (n == 0 || num_pools == 0) return PSD_OK;
  if (!src || !dst || !fault_dev) return fail(PSD_ERR_INVALID_ARG, "copy_pages: NULL pointer");
  DeviceGuard g(ctx->dev.device);
  CopyParams c = {};
  c.src = src;
  c.dst = dst;
  c.n = n;
  c.fault = fault_dev;
  c.num_pages = num_pages;
  return launch_copy(c, pools, num_pools, n, false, ctx->dev, reinterpret_cast<cudaStream_t>(stream));
}
