// Groups of requests that share a prefix: their rows, keys and list entries.
#pragma once

#include "attn.h"
#include "attn_dev.cuh"

namespace moe {

// A prefix is cut to whole tiles of the split kernel, so that the own keys begin
// with one.
constexpr int kPrefixCut = 32;

// Place of a row's chunk of four channels among sums over prefixes.
__device__ __forceinline__ long sums_at(long row, int chunk, int chunks) {
  return (row / 8 * chunks + chunk) * 8 + row % 8;
}

struct GroupLists {
  const int* offsets;  // [n + 1] requests
  int* limit;          // [n] shared tokens
  int* first;          // [n] first request with queries
  SeqInfo* groups;     // [n] query rows, shared tokens, and `first` as the row of the page table
  long* bases;         // [n + 1] first list entry
};
struct GroupSmem {
  long bases[kSmallGroups + 1];
  SeqInfo groups[kSmallGroups];
  int offsets[kSmallGroups + 1], limit[kSmallGroups], first[kSmallGroups];
  __device__ GroupLists lists() { return {offsets, limit, first, groups, bases}; }
};

__device__ __forceinline__ int prefix_entries(const PrefixShape& w, int tokens, bool half) {
  return w.setup + (tokens + w.tile_keys - 1) / w.tile_keys * (half ? w.half_unit : w.unit);
}
// Row tiles of a group; `half`: the last has no more than half_rows rows.
__device__ __forceinline__ int row_tiles_of(const PrefixShape& w, int rows, bool& half) {
  const int n = (rows + w.tile_rows - 1) / w.tile_rows;
  half = n > 0 && rows - (n - 1) * w.tile_rows <= w.half_rows;
  return n;
}
// a / b for values that hardly ever need 64 bits.
__device__ __forceinline__ long quotient(long a, long b) {
  return ((a | b) >> 32) == 0 ? static_cast<unsigned>(a) / static_cast<unsigned>(b) : a / b;
}
// Entries per CTA of a list.
__device__ __forceinline__ long prefix_per(const PrefixShape& w, long entries) {
  const long per = quotient(entries + w.ctas - 1, w.ctas);
  return per < w.least ? w.least : per;
}

// The last of n ascending values that is at most v (0 where there is none).
template <typename T>
__device__ __forceinline__ int last_at_most(const T* values, int n, T v) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (values[mid] <= v) lo = mid;
    else hi = mid;
  }
  return lo;
}

// A block of N threads checks the requests and groups, cuts each prefix to what
// all of its requests have before their queries, and sums up the list; returns
// its entries. `smem`: where the lists are shared memory, else nullptr.
// each(b, info, group or -1) is called for every request before the lists are
// complete; flags collects MOE_DEV_* bits.
template <int N, class Each>
__device__ __forceinline__ long plan_groups(const AttnArgs& a, const Groups& gr,
                                            const PrefixShape& w, const GroupLists& l,
                                            GroupSmem* smem, long* warp_sum, unsigned& flags,
                                            Each each) {
  auto q_at = [&](int b) { return a.q_offsets ? a.q_offsets[b] : b; };
  int b = threadIdx.x;
  SeqInfo s = {0, 0, 0, 0};
  if (b < a.B) s = seq_info(a, b, flags);  // on the way while the groups are read
  bool bad = false;
  for (int g = threadIdx.x; g < gr.n; g += N) {
    const int b0 = gr.offsets[g], b1 = gr.offsets[g + 1], p = gr.prefix[g];
    bad |= b0 < 0 || b1 < b0 || b1 > a.B;
    if (p < 0) flags |= MOE_DEV_BAD_SEGMENT;
    l.limit[g] = max(0, p);
    l.first[g] = 0x7fffffff;
    l.groups[g] = {0, 0, 0, 0};
    if (smem) {
      smem->offsets[g] = b0;
      if (g == gr.n - 1) smem->offsets[gr.n] = b1;
    }
  }
  bad = __syncthreads_or(bad);
  if (bad) flags |= MOE_DEV_BAD_SEGMENT;
  while (b < a.B) {
    int g = bad ? -1 : last_at_most(l.offsets, gr.n, b);
    if (g >= 0 && (b < l.offsets[g] || b >= l.offsets[g + 1])) g = -1;
    each(b, s, g);
    if (g >= 0) {
      const int q0 = q_at(b), q1 = q_at(b + 1);
      if (b == l.offsets[g]) l.groups[g].q0 = q0;
      if (b + 1 == l.offsets[g + 1]) l.groups[g].q_len = q1;
      if (s.q_len > 0) {
        atomicMin(l.limit + g, max(0, s.len - s.q_len));
        atomicMin(l.first + g, b);
      } else if (q1 != q0) {
        atomicMin(l.limit + g, 0);  // its offsets were refused: its group's may be wrong
      }
    }
    b += N;
    if (b < a.B) s = seq_info(a, b, flags);
  }
  __threadfence_block();
  __syncthreads();
  long entries = 0;
  for (int g0 = 0; g0 < gr.n; g0 += N) {
    const int g = g0 + threadIdx.x;
    long n = 0;
    if (g < gr.n) {
      SeqInfo s = l.groups[g];
      s.q_len -= s.q0;
      int p = bad ? 0 : *const_cast<volatile int*>(l.limit + g) / kPrefixCut * kPrefixCut;
      // whatever is left of its prefix (offsets that were refused set this flag anyway)
      if (s.q_len > gr.max_len) flags |= MOE_DEV_BAD_SEGMENT;
      if (p > 0) {
        s.first_key = *const_cast<volatile int*>(l.first + g);
        // (a group of one token, or of one request, has nothing to share)
        if (l.offsets[g + 1] - l.offsets[g] < 2 || s.q_len < 2 || s.q_len > gr.max_len) p = 0;
      }
      s.len = p;
      if (p == 0) s.q_len = 0;
      l.limit[g] = p;
      l.groups[g] = s;
      const int rows = s.q_len * (a.heads / a.kv_heads);
      bool half;
      const int tiles = row_tiles_of(w, rows, half);
      n = a.kv_heads * (static_cast<long>(tiles - half) * prefix_entries(w, p, false) +
                        (half ? prefix_entries(w, p, true) : 0));
    }
    const long before = block_scan<N>(n, warp_sum, entries);
    if (g < gr.n) l.bases[g] = before;
  }
  if (threadIdx.x == 0) l.bases[gr.n] = entries;
  __syncthreads();
  return entries;
}

}  // namespace moe
