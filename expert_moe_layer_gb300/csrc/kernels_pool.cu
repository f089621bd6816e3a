// Pages of a cache that several requests share: forking, reserving, releasing,
// compacting and copying.
//
// Whole numbers throughout, and nothing depends on the order in which threads
// run: free pages are handed out by rank (the k-th lowest free page to the k-th
// place that needs one), and counts of holders change by atomics whose order
// does not show. Reserving and compacting look through all counts once, a CTA
// per chunk, and leave behind each chunk's free pages from the front of its part
// of a list and its pages in use from the back; the CTA that comes last sums up
// the chunks and plans the call, and a second kernel carries it out on the whole
// GPU. Launch latency bounds the calls on tables; copies of pages are bound by
// memory: a warp takes 4 KB of a page, eight 16-byte loads per lane on the way.
#include <cuda_runtime.h>

#include "launch.cuh"
#include "ptx.cuh"
#include "serve.h"

namespace moe {
namespace {

constexpr int kScanThreads = 1024;
constexpr int kPer = kScan / kScanThreads;  // counts per thread and step
constexpr int kApplyThreads = 256;
constexpr int kPiece = 4096;       // bytes of a page that a warp copies at a time
constexpr int kCopyCtasPerSm = 6;  // of kApplyThreads
constexpr int kMaxApplyCtas = 2048;
constexpr int kAhead = 4;          // entries that a thread has under way

struct Item {
  int first;  // rank of its first fresh page; -1: nothing is done
  int own;    // entries that get a page of their own
};

struct Work {
  PoolHeader* head;
  int* claims;
  Item* items;
  int2* copies;  // (from, to)
  int* prefix;   // free pages before each chunk, [chunks + 1]
  int32_t* list;
  int32_t* ranks;
  long chunk;
  int chunks;
};

Work work_of(const PoolArgs& a, void* ws, const PoolLayout& L) {
  char* w = static_cast<char*>(ws);
  Work k;
  k.head = reinterpret_cast<PoolHeader*>(w);
  k.claims = reinterpret_cast<int*>(w + L.claims);
  k.items = reinterpret_cast<Item*>(w + L.items);
  k.copies = reinterpret_cast<int2*>(w + L.copies);
  k.prefix = reinterpret_cast<int*>(w + L.prefix);
  k.list = reinterpret_cast<int32_t*>(w + L.list);
  k.ranks = reinterpret_cast<int32_t*>(w + L.ranks);
  k.chunk = pool_chunk(a.pages);
  k.chunks = static_cast<int>((a.pages + k.chunk - 1) / k.chunk);
  return k;
}

// A token's entry, and the entries that so many tokens take.
__device__ __forceinline__ int entry_of(const PoolArgs& a, long token) {
  return static_cast<int>(token >> a.page_shift);
}
__device__ __forceinline__ int entries_of(const PoolArgs& a, long tokens) {
  return static_cast<int>((tokens + (1l << a.page_shift) - 1) >> a.page_shift);
}
__device__ __forceinline__ long tokens_of_row(const PoolArgs& a) {
  return static_cast<long>(a.max_pages) << a.page_shift;
}

// Sum of the values of the threads before this one in a block of kScanThreads,
// plus `base`, to which the block's sum is added.
template <typename T>
__device__ __forceinline__ T scan(T v, T* warp_sum, T& base) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T sum = v;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const T u = __shfl_up_sync(~0u, sum, d);
    if (lane >= d) sum += u;
  }
  if (lane == 31) warp_sum[warp] = sum;
  __syncthreads();
  T warps = warp_sum[lane];  // (as many warps as lanes)
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const T u = __shfl_up_sync(~0u, warps, d);
    if (lane >= d) warps += u;
  }
  const T before = base + (warp > 0 ? __shfl_sync(~0u, warps, (warp + 31) & 31) : 0);
  base += __shfl_sync(~0u, warps, 31);
  __syncthreads();
  return before + sum - v;
}

__device__ __forceinline__ void report(const PoolArgs& a, unsigned flags) {
  if (flags && a.status) atomicOr(a.status, flags);
}

// One holder of a page less. (Counts that do not fit the table stay at 0.)
__device__ __forceinline__ void drop(const PoolArgs& a, int page, unsigned& flags) {
  if (atomicSub(a.refs + page, 1) > 0) return;
  atomicAdd(a.refs + page, 1);
  flags |= MOE_DEV_BAD_PAGE;
}

// The k-th free page, or page in use, counted from 0: the last chunk that has at
// most k of them before it, then its part of the list. (What another CTA of the
// same kernel wrote is read past the L1 cache.)
template <bool kFree>
__device__ __forceinline__ int chunk_of_rank(const Work& w, long k) {
  int lo = 0, hi = w.chunks;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    const long free = __ldcg(w.prefix + mid);
    if ((kFree ? free : mid * w.chunk - free) <= k) lo = mid;
    else hi = mid;
  }
  return lo;
}
__device__ __forceinline__ int free_page(const Work& w, long k) {
  const int c = chunk_of_rank<true>(w, k);
  return __ldcg(w.list + c * w.chunk + (k - __ldcg(w.prefix + c)));
}
__device__ __forceinline__ int used_page(const Work& w, long pages, long k) {
  const int c = chunk_of_rank<false>(w, k);
  const long end = min((c + 1) * w.chunk, pages);
  return __ldcg(w.list + end - 1 - (k - (c * w.chunk - __ldcg(w.prefix + c))));
}

// A CTA's chunk: its free pages and its pages in use into the list, and with
// kRanks each page's place among its kind. Returns the free ones' number.
template <bool kRanks>
__device__ __forceinline__ int scan_chunk(const PoolArgs& a, const Work& w, int* warp_sum) {
  const long begin = blockIdx.x * w.chunk, end = min(begin + w.chunk, a.pages);
  const bool wide = reinterpret_cast<uintptr_t>(a.refs) % 16 == 0;
  int found = 0;
  for (long at = begin; at < end; at += kScan) {
    const long p0 = at + threadIdx.x * kPer;
    int refs[kPer];
    if (wide && p0 + kPer <= end) {
#pragma unroll
      for (int i = 0; i < kPer / 4; ++i) {
        const int4 v = reinterpret_cast<const int4*>(a.refs + p0)[i];
        refs[4 * i] = v.x, refs[4 * i + 1] = v.y, refs[4 * i + 2] = v.z, refs[4 * i + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i) refs[i] = p0 + i < end ? a.refs[p0 + i] : 1;
    }
    int n = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) n += refs[i] == 0;
    int f = scan(n, warp_sum, found);  // free ones before p0
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const long p = p0 + i;
      if (p >= end) continue;
      const long u = p - begin - f;  // pages in use before p
      if (refs[i] == 0) {
        w.list[begin + f] = static_cast<int32_t>(p);
        if (kRanks) w.ranks[p] = f;
        ++f;
      } else {
        w.list[end - 1 - u] = static_cast<int32_t>(p);
        if (kRanks) w.ranks[p] = static_cast<int32_t>(u);
      }
    }
  }
  return found;
}

// Puts the chunk's count behind those of the others. True in the CTA that came
// last, where prefix[] is then summed up and `total` holds all free pages.
__device__ __forceinline__ bool last_to_scan(const Work& w, int found, int* warp_sum, int& total) {
  __shared__ int s_last;
  if (w.chunks == 1) {
    if (threadIdx.x == 0) w.prefix[0] = 0, w.prefix[1] = found;
    total = found;
    __syncthreads();
    return true;
  }
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    w.prefix[blockIdx.x] = found;
    s_last = ptx::add_acq_rel(&w.head->done, 1) == w.chunks - 1;
  }
  __syncthreads();
  if (!s_last) return false;
  __threadfence();
  total = 0;
  const int c = threadIdx.x;  // kMaxChunks is the number of threads
  const int before = scan(c < w.chunks ? __ldcg(w.prefix + c) : 0, warp_sum, total);
  if (c < w.chunks) w.prefix[c] = before;
  if (threadIdx.x == 0) w.prefix[w.chunks] = total;
  __syncthreads();
  return true;
}

// Row, place and number of entries of one item of a reservation.
struct Span {
  int row, lo, hi, held;  // entries [lo, hi) are to be the row's own; it has `held`
  bool ok;
};
__device__ __forceinline__ Span span_of(const PoolArgs& a, int i, const int32_t* rows,
                                        const int32_t* start, const int32_t* end) {
  Span s = {rows ? rows[i] : i, 0, 0, 0, false};
  const long from = start[i], to = end[i];
  if (s.row < 0 || s.row >= a.rows || from < 0 || to < from ||
      to > tokens_of_row(a))
    return s;
  s.held = a.held[s.row];
  s.hi = entries_of(a, to);
  s.lo = from < to ? entry_of(a, from) : s.hi;
  s.ok = s.held >= 0 && s.held <= a.max_pages;
  return s;
}
// Entries that are to be replaced are marked in the table: page p as -2 - p.
// (What is decided here by counts that the second kernel changes.)
__device__ __forceinline__ bool is_mark(const PoolArgs& a, int entry) {
  return entry <= -2 && entry >= -1 - a.pages;
}
// Whether an entry's page has other holders. One that reads as a mark becomes -1.
__device__ __forceinline__ bool shared_page(const PoolArgs& a, int32_t* entry, int page,
                                            unsigned& flags) {
  if (page < 0 || page >= a.pages) {
    flags |= MOE_DEV_BAD_PAGE;
    if (is_mark(a, page)) *entry = -1;
    return false;
  }
  return a.refs[page] > 1;
}

__global__ void __launch_bounds__(kScanThreads)
    reserve_plan_kernel(PoolArgs a, Work w, int n, const int32_t* rows, const int32_t* start,
                        const int32_t* end) {
  __shared__ int warp_sum[kScanThreads / 32];
  pdl_enter();
  if (w.chunks == 1) {
    if (threadIdx.x == 0) *w.head = {};
    if (rows)
      for (int i = threadIdx.x; i < a.rows; i += kScanThreads) w.claims[i] = 0;
    __syncthreads();
  }
  const int found = scan_chunk<false>(a, w, warp_sum);
  int all_free;
  if (!last_to_scan(w, found, warp_sum, all_free)) return;
  __shared__ long item_sum[kScanThreads / 32];
  unsigned flags = 0;
  if (rows) {  // the first item of a row has it
    for (int i = threadIdx.x; i < n; i += kScanThreads)
      if (rows[i] >= 0 && rows[i] < a.rows) atomicMax(w.claims + rows[i], n - i);
    __threadfence();
    __syncthreads();
  }
  const int lane = threadIdx.x & 31;
  long taken = 0;  // places before these items in the low 40 bits, copies above
  for (int i0 = 0; i0 < n; i0 += kScanThreads) {
    const int i = i0 + threadIdx.x;
    Span s = {0, 0, 0, 0, false};
    int fresh = 0, marked = 0, old = -1;
    if (i < n) {
      s = span_of(a, i, rows, start, end);
      if (s.ok && rows && __ldcg(w.claims + s.row) != n - i) s.ok = false;
      if (!s.ok) flags |= MOE_DEV_BAD_ROW;
    }
    const int stop = s.ok ? min(s.hi, s.held) : 0;
    int32_t* entries = a.table + static_cast<long>(s.row) * a.max_pages;
    const bool cut = s.ok && (start[i] & ((1 << a.page_shift) - 1)) != 0;  // the first page keeps tokens
    if (s.ok && s.lo < stop) {
      const int page = entries[s.lo];
      if (shared_page(a, entries + s.lo, page, flags)) {
        marked = 1;
        entries[s.lo] = -2 - page;
        if (cut) old = page;
      }
    }
    // further entries that the row has already: the warp, a row at a time
    for (unsigned more = __ballot_sync(~0u, s.ok && s.lo + 1 < stop); more; more &= more - 1) {
      const int who = __ffs(more) - 1;
      const int lo = __shfl_sync(~0u, s.lo, who) + 1, hi = __shfl_sync(~0u, stop, who);
      int32_t* row = a.table + static_cast<long>(__shfl_sync(~0u, s.row, who)) * a.max_pages;
      int count = 0;
      for (int e = lo + lane; e < hi; e += 32) {
        const int page = row[e];
        if (!shared_page(a, row + e, page, flags)) continue;
        row[e] = -2 - page;
        ++count;
      }
      count = __reduce_add_sync(~0u, count);
      if (lane == who) marked += count;
    }
    if (s.ok) fresh = marked + max(0, s.hi - s.held);
    const long mine = fresh + (old >= 0 ? 1l << 40 : 0);
    const long before = scan(mine, item_sum, taken);
    const long first = before & ((1l << 40) - 1);
    if (i < n) {
      const bool served = fresh == 0 || first + fresh <= all_free;
      if (!served) flags |= MOE_DEV_NO_PAGE;
      w.items[i] = {s.ok && served ? static_cast<int>(first) : -1, marked};
      // a place that is served has every place before it served too, so that
      // the copies form a list without gaps
      if (old >= 0 && served)
        w.copies[before >> 40] = make_int2(old, free_page(w, first));
      if (old >= 0 && served) atomicAdd(&w.head->copies, 1);
    }
  }
  report(a, flags);
}

// The pages of a list, in every cache, cut into pieces: (page of the list, cache,
// piece). Each warp has a range of neighbouring pieces, so that it looks up a pair
// of pages once for all pieces of it (compacting, where a page is found by rank in
// two dependent loads, took 200 us with pieces dealt out in turn, the case below).
template <class Pair>
__device__ __forceinline__ void copy_units(const CacheList& from, const CacheList& to, long pairs,
                                           long warp, long warps, Pair pair) {
  const int lane = threadIdx.x & 31;
  const int pieces = static_cast<int>((from.page_bytes + kPiece - 1) / kPiece);
  const long units = pairs * from.n * pieces, per = (units + warps - 1) / warps;
  long u = warp * per;
  const long end = min(units, u + per);
  if (u >= end) return;
  long rest = u / pieces;
  int piece = static_cast<int>(u - rest * pieces);
  long j = rest / from.n;
  int c = static_cast<int>(rest - j * from.n);
  int2 ids = pair(j);
  for (; u < end; ++u) {
    if (ids.x >= 0) {
      const long at = static_cast<long>(piece) * kPiece;
      const int left = static_cast<int>(min(static_cast<long>(kPiece), from.page_bytes - at)) / 16;
      const uint4* s = reinterpret_cast<const uint4*>(from.p[c] + ids.x * from.page_bytes + at);
      uint4* d = reinterpret_cast<uint4*>(to.p[c] + ids.y * from.page_bytes + at);
      uint4 v[kPiece / 512];
#pragma unroll
      for (int i = 0; i < kPiece / 512; ++i)
        if (32 * i + lane < left) v[i] = __ldcs(s + 32 * i + lane);
#pragma unroll
      for (int i = 0; i < kPiece / 512; ++i)
        if (32 * i + lane < left) __stcs(d + 32 * i + lane, v[i]);
    }
    if (++piece == pieces) {
      piece = 0;
      if (++c == from.n) {
        c = 0;
        ++j;
        if (u + 1 < end) ids = pair(j);
      }
    }
  }
}

// CTAs below `appliers` carry out items, the others copy pages.
__global__ void __launch_bounds__(kApplyThreads)
    reserve_apply_kernel(PoolArgs a, Work w, const __grid_constant__ CacheList caches, int n,
                         int appliers, const int32_t* rows, const int32_t* start,
                         const int32_t* end) {
  pdl_enter();
  const Work f = {fresh(w.head), w.claims, fresh(w.items), fresh(w.copies), fresh(w.prefix),
                  fresh(w.list), w.ranks, w.chunk, w.chunks};
  const int lane = threadIdx.x & 31;
  if (blockIdx.x >= appliers) {
    const long warps = static_cast<long>(gridDim.x - appliers) * (kApplyThreads / 32);
    const long warp = static_cast<long>(blockIdx.x - appliers) * (kApplyThreads / 32) + (threadIdx.x >> 5);
    copy_units(caches, caches, f.head->copies, warp, warps, [&](long j) { return f.copies[j]; });
    return;
  }
  unsigned flags = 0;
  for (int i = blockIdx.x; i < n; i += appliers) {
    const Span s = span_of(a, i, rows, start, end);
    const Item it = f.items[i];
    __syncthreads();  // every thread has read `held`
    if (!s.ok) continue;
    int32_t* entries = a.table + static_cast<long>(s.row) * a.max_pages;
    const bool served = it.first >= 0;
    if (it.own > 0 && threadIdx.x < 32) {  // marked entries, in their order
      int rank = it.first;
      for (int e0 = s.lo; e0 < min(s.hi, s.held); e0 += 32) {
        const int e = e0 + lane;
        const int v = e < min(s.hi, s.held) ? entries[e] : -1;
        const bool marked = is_mark(a, v);
        const unsigned mask = __ballot_sync(~0u, marked);
        if (marked && served) {
          const int page = free_page(f, rank + __popc(mask & ((1u << lane) - 1u)));
          entries[e] = page;
          a.refs[page] = 1;
          drop(a, -2 - v, flags);
        } else if (marked) {
          entries[e] = -2 - v;
        }
        rank += __popc(mask);
      }
    }
    if (!served) continue;
    for (int e = s.held + threadIdx.x; e < s.hi; e += kApplyThreads) {
      const int page = free_page(f, it.first + it.own + (e - s.held));
      entries[e] = page;
      a.refs[page] = 1;
    }
    if (threadIdx.x == 0 && s.hi > s.held) a.held[s.row] = s.hi;
  }
  report(a, flags);
}

__global__ void __launch_bounds__(kScanThreads)
    compact_plan_kernel(PoolArgs a, Work w, int32_t* used_out) {
  __shared__ int warp_sum[kScanThreads / 32];
  pdl_enter();
  if (w.chunks == 1) {
    if (threadIdx.x == 0) *w.head = {};
    __syncthreads();
  }
  const int found = scan_chunk<true>(a, w, warp_sum);
  int all_free;
  if (!last_to_scan(w, found, warp_sum, all_free) || threadIdx.x != 0) return;
  const long used = a.pages - all_free;
  long moves = all_free;  // free pages below `used`
  if (used < a.pages) {
    const int c = static_cast<int>(used / w.chunk);
    int lo = 0, hi = w.prefix[c + 1] - w.prefix[c];
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (__ldcg(w.list + c * w.chunk + mid) < used) lo = mid + 1;
      else hi = mid;
    }
    moves = w.prefix[c] + lo;
  }
  w.head->free = static_cast<int>(all_free);
  w.head->used = static_cast<int>(used);
  w.head->moves = static_cast<int>(moves);
  if (used_out) *used_out = static_cast<int32_t>(used);
}

// The k-th page in use from `used` on goes to the k-th free page (all of which
// lie below `used`): no page is both read and written. CTAs below `appliers`
// follow the moves in the counts and the table, the others copy pages. (The rows
// are looked at where nothing moves too: their bad entries are reported.)
__global__ void __launch_bounds__(kApplyThreads)
    compact_apply_kernel(PoolArgs a, Work w, const __grid_constant__ CacheList caches, int appliers) {
  pdl_enter();
  const Work f = {fresh(w.head), w.claims, w.items, w.copies, fresh(w.prefix),
                  fresh(w.list), fresh(w.ranks), w.chunk, w.chunks};
  const long used = f.head->used, moves = f.head->moves, stay = used - moves;
  if (blockIdx.x >= appliers) {
    const long warps = static_cast<long>(gridDim.x - appliers) * (kApplyThreads / 32);
    const long warp = static_cast<long>(blockIdx.x - appliers) * (kApplyThreads / 32) + (threadIdx.x >> 5);
    copy_units(caches, caches, moves, warp, warps, [&](long j) {
      return make_int2(used_page(f, a.pages, stay + j), free_page(f, j));
    });
    return;
  }
  for (long j = static_cast<long>(blockIdx.x) * kApplyThreads + threadIdx.x; j < moves;
       j += static_cast<long>(appliers) * kApplyThreads) {
    const int src = used_page(f, a.pages, stay + j), dst = free_page(f, j);
    a.refs[dst] = a.refs[src];
    a.refs[src] = 0;
  }
  unsigned flags = 0;
  for (int row = blockIdx.x; row < a.rows; row += appliers) {
    const int held = a.held[row];
    if (held < 0 || held > a.max_pages) flags |= MOE_DEV_BAD_ROW;
    int32_t* entries = a.table + static_cast<long>(row) * a.max_pages;
    for (int e = threadIdx.x; e < min(held, a.max_pages); e += kApplyThreads) {
      const int page = entries[e];
      if (page < 0 || page >= a.pages) {
        flags |= MOE_DEV_BAD_PAGE;
      } else if (page >= used) {
        const int c = static_cast<int>(page / f.chunk);
        const int rank = f.ranks[page];
        // (a held page without a holder is free: its rank is that of another kind)
        const long k = c * f.chunk - f.prefix[c] + rank - stay;
        if (k >= 0 && k < moves && used_page(f, a.pages, stay + k) == page)
          entries[e] = free_page(f, k);
        else
          flags |= MOE_DEV_BAD_PAGE;
      }
    }
  }
  report(a, flags);
}

__global__ void clear_kernel(int* words, long n) {
  pdl_enter();
  for (long i = static_cast<long>(blockIdx.x) * blockDim.x + threadIdx.x; i < n;
       i += static_cast<long>(gridDim.x) * blockDim.x)
    words[i] = 0;
}

// Few items are carried out by the blocks of one cluster, which can agree that the
// status is cleared before any of them reports (another kernel for that takes a
// call's host time from 6 to 9 us).
constexpr int kCluster = 8;
__device__ __forceinline__ void enter_items(const PoolArgs& a, int n) {
  pdl_enter();
  if (n > kFewItems || !a.status) return;
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0;
  __syncwarp();
  ptx::cluster_sync();
}
template <typename... KArgs, typename... Args>
cudaError_t launch_items(void (*kern)(KArgs...), int n, cudaStream_t st, Args&&... args) {
  if (n > kFewItems)
    return launch_pdl(kern, dim3(n < kMaxApplyCtas ? n : kMaxApplyCtas), dim3(kApplyThreads), 0, st,
                      std::forward<Args>(args)...);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kCluster);
  cfg.blockDim = dim3(kApplyThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kCluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return counted(cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...));
}

// A block per item. A child that an earlier item names too, or that is a parent
// in this call, is refused by looking through the children: nothing that a block
// reads is written by another then. It needs no workspace, but the work grows with
// n^2: 512 items 3.2 us, 4096 11, 16384 92, 65536 1.3 ms, 131072 5.1 ms.
__global__ void __launch_bounds__(kApplyThreads)
    fork_kernel(PoolArgs a, int n, const int32_t* parents, const int32_t* children,
                const int32_t* tokens) {
  enter_items(a, n);
  unsigned flags = 0;
  for (int i = blockIdx.x; i < n; i += gridDim.x) {
    const int parent = parents[i], child = children[i];
    const long t = tokens[i];
    bool ok = parent >= 0 && parent < a.rows && child >= 0 && child < a.rows && t >= 0 &&
              t <= tokens_of_row(a);
    const int need = ok ? entries_of(a, t) : 0;
    bool clash = false;
    for (int j = threadIdx.x; j < n; j += kApplyThreads) {
      const int other = children[j];
      clash |= (j < i && other == child) || other == parent;
    }
    clash = __syncthreads_or(clash);
    // (the winner alone reads its child's count, before any of its threads writes it)
    ok = ok && !clash;
    if (ok) ok = a.held[child] == 0 && need <= a.held[parent] && a.held[parent] <= a.max_pages;
    if (!__syncthreads_and(ok)) {
      flags |= MOE_DEV_BAD_ROW;
      continue;
    }
    const int32_t* from = a.table + static_cast<long>(parent) * a.max_pages;
    int32_t* to = a.table + static_cast<long>(child) * a.max_pages;
    for (int e0 = threadIdx.x; e0 < need; e0 += kAhead * kApplyThreads) {
      int page[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int e = e0 + i * kApplyThreads;
        page[i] = e < need ? from[e] : 0;
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int e = e0 + i * kApplyThreads;
        if (e >= need) continue;
        to[e] = page[i];
        if (page[i] >= 0 && page[i] < a.pages)
          atomicAdd(a.refs + page[i], 1);
        else
          flags |= MOE_DEV_BAD_PAGE;
      }
    }
    if (threadIdx.x == 0) a.held[child] = need;
  }
  report(a, flags);
}

// A block per item takes the entries between what the row is to keep and what
// it held; of items with the same row each takes the part that it finds. A count
// is lowered by compare and swap, since one that lies outside the table has to
// stay (a minimum would have changed it before anyone saw it: what such a row
// names may be other rows' pages).
__global__ void __launch_bounds__(kApplyThreads)
    release_kernel(PoolArgs a, int n, const int32_t* rows, const int32_t* keep) {
  __shared__ int s_held;
  enter_items(a, n);
  unsigned flags = 0;
  for (int i = blockIdx.x; i < n; i += gridDim.x) {
    const int row = rows ? rows[i] : i;
    const long t = keep ? keep[i] : 0;
    if (row < 0 || row >= a.rows || t < 0) {
      flags |= MOE_DEV_BAD_ROW;
      continue;
    }
    const int left = min(entries_of(a, t), a.max_pages);
    __syncthreads();
    if (threadIdx.x == 0) {
      int held = __ldcg(a.held + row);
      while (held > left && held <= a.max_pages) {
        const int found = atomicCAS(a.held + row, held, left);
        if (found == held) break;
        held = found;
      }
      s_held = held;
    }
    __syncthreads();
    const int stop = s_held;
    if (stop < 0 || stop > a.max_pages) {
      flags |= MOE_DEV_BAD_ROW;
      continue;
    }
    int32_t* entries = a.table + static_cast<long>(row) * a.max_pages;
    for (int e0 = left + threadIdx.x; e0 < stop; e0 += kAhead * kApplyThreads) {
      int page[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int e = e0 + i * kApplyThreads;
        page[i] = e < stop ? entries[e] : 0;
      }
      int before[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int e = e0 + i * kApplyThreads;
        before[i] = 1;
        if (e >= stop) continue;
        entries[e] = -1;
        if (page[i] >= 0 && page[i] < a.pages)
          before[i] = atomicSub(a.refs + page[i], 1);
        else
          flags |= MOE_DEV_BAD_PAGE;
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (before[i] <= 0) {
          atomicAdd(a.refs + page[i], 1);
          flags |= MOE_DEV_BAD_PAGE;
        }
    }
  }
  report(a, flags);
}

__global__ void __launch_bounds__(kApplyThreads)
    copy_pages_kernel(const __grid_constant__ CacheList from, long from_pages,
                      const __grid_constant__ CacheList to, long to_pages, int n,
                      const int32_t* src, const int32_t* dst, unsigned* status) {
  pdl_enter();
  unsigned flags = 0;
  const long warp = static_cast<long>(blockIdx.x) * (kApplyThreads / 32) + (threadIdx.x >> 5);
  copy_units(from, to, n, warp, static_cast<long>(gridDim.x) * (kApplyThreads / 32), [&](long j) {
    const int s = src[j], d = dst[j];
    if (s == -1 || d == -1) return make_int2(-1, -1);
    if (s < 0 || s >= from_pages || d < 0 || d >= to_pages) {
      flags |= MOE_DEV_BAD_PAGE;
      return make_int2(-1, -1);
    }
    return make_int2(s, d);
  });
  if (flags && status) atomicOr(status, flags);
}

// CTAs that copy up to `pairs` pages in all caches.
int copy_ctas(const CacheList& caches, long pairs, int sms) {
  const long units = pairs * caches.n * ((caches.page_bytes + kPiece - 1) / kPiece);
  const long ctas = (units + kApplyThreads / 32 - 1) / (kApplyThreads / 32);
  const long most = static_cast<long>(sms) * kCopyCtasPerSm;
  return static_cast<int>(ctas < most ? ctas : most);
}

}  // namespace

// (A kernel, not a memset: it can be scheduled while the one before it ends, and
// the one after it while it runs.)
cudaError_t launch_clear(void* words, long n, cudaStream_t st) {
  const long blocks = (n + 1023) / 1024;
  return launch_pdl(&clear_kernel, dim3(static_cast<unsigned>(blocks < 64 ? blocks : 64)),
                    dim3(n < 32 ? 32 : 1024), 0, st, static_cast<int*>(words), n);
}

bool pool_clears(long pages) { return pages <= pool_chunk(pages); }

PoolLayout pool_layout(long pages, int rows, int n) {
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  PoolLayout L;
  L.claims = 256;
  L.items = up(L.claims + 4 * static_cast<size_t>(rows));
  L.copies = up(L.items + sizeof(Item) * static_cast<size_t>(n));
  L.prefix = up(L.copies + sizeof(int2) * static_cast<size_t>(n));
  L.list = up(L.prefix + 4 * (kMaxChunks + 1));
  L.ranks = up(L.list + 4 * static_cast<size_t>(pages));
  L.total = up(L.ranks + 4 * static_cast<size_t>(pages));
  return L;
}

cudaError_t launch_reserve(const PoolArgs& a, const CacheList& caches, int n, const int32_t* rows,
                           const int32_t* start, const int32_t* end, void* ws, const PoolLayout& L,
                           int sms, cudaStream_t st) {
  const Work w = work_of(a, ws, L);
  const cudaError_t e = launch_pdl(&reserve_plan_kernel, dim3(w.chunks), dim3(kScanThreads), 0, st, a,
                                   w, n, rows, start, end);
  if (e != cudaSuccess) return e;
  const int appliers = n < kMaxApplyCtas ? n : kMaxApplyCtas;
  return launch_pdl(&reserve_apply_kernel, dim3(appliers + copy_ctas(caches, n, sms)),
                    dim3(kApplyThreads), 0, st, a, w, caches, n, appliers, rows, start, end);
}

cudaError_t launch_compact(const PoolArgs& a, const CacheList& caches, int32_t* used, void* ws,
                           const PoolLayout& L, int sms, cudaStream_t st) {
  const Work w = work_of(a, ws, L);
  const cudaError_t e =
      launch_pdl(&compact_plan_kernel, dim3(w.chunks), dim3(kScanThreads), 0, st, a, w, used);
  if (e != cudaSuccess) return e;
  const int appliers = a.rows < sms ? a.rows : sms;
  return launch_pdl(&compact_apply_kernel, dim3(appliers + copy_ctas(caches, a.pages / 2, sms)),
                    dim3(kApplyThreads), 0, st, a, w, caches, appliers);
}

cudaError_t launch_fork(const PoolArgs& a, int n, const int32_t* parents, const int32_t* children,
                        const int32_t* tokens, cudaStream_t st) {
  return launch_items(&fork_kernel, n, st, a, n, parents, children, tokens);
}

cudaError_t launch_release(const PoolArgs& a, int n, const int32_t* rows, const int32_t* keep,
                           cudaStream_t st) {
  return launch_items(&release_kernel, n, st, a, n, rows, keep);
}

cudaError_t launch_copy_pages(const CacheList& from, long from_pages, const CacheList& to,
                              long to_pages, int n, const int32_t* src, const int32_t* dst,
                              unsigned* status, int sms, cudaStream_t st) {
  return launch_pdl(&copy_pages_kernel, dim3(copy_ctas(from, n, sms)), dim3(kApplyThreads), 0, st,
                    from, from_pages, to, to_pages, n, src, dst, status);
}

}  // namespace moe
