// Attention of requests that share a prefix: the prefix once for all rows of a
// group, then each request's own keys.
//
//   m = max(m1, m2),  o = (2^(m1-m) s1 + 2^(m2-m) s2) / (2^(m1-m) l1 + 2^(m2-m) l2)
//
// with s, l, m the sums of P V and of P and the base of the scores over the
// prefix (1) and over the own keys (2). Rows of all requests of a group form row
// tiles over the prefix as if they were one request whose queries see every key:
// the prompt kernel from kPromptRows rows on (bf16), else the split kernel. It
// leaves its pieces' sums in fp32 and joins nothing. The split kernel over the
// own keys then adds them to each row as it stores it: that join is spread over
// all CTAs, where the last CTA of a segment would do it for a whole row tile.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>

#include "attn_prompt.cuh"
#include "attn_split.cuh"
#include "internal.h"
#include "launch.cuh"

namespace moe {

MOE_WAIT_LIMIT_SETTER(set_wait_limit_attn_shared)

namespace {

// A block of 256: with 1024 threads the sums over the block alone took 2 of 9.5 us.
constexpr int kPlanThreads = 256;
// A prefix is cut to whole tiles of the split kernel, so that the own keys begin
// with one.
constexpr int kCut = split::kTile;

struct Groups {
  int n;
  const int32_t* offsets;  // [n + 1] requests
  const int32_t* prefix;   // [n] tokens
  int max_len;             // query tokens
};

// Up to so many requests and groups the plan keeps its lists in shared memory.
constexpr int kSmallSeqs = 1024, kSmallGroups = 256;
// Smallest range of a CTA over a prefix: pieces of two tiles.
constexpr int kMinPrefix = prompt::kSetup + 2;
static_assert(kMinPrefix > prompt::kSetup + prompt::kPrefixSnap, "cuts do not cross");

// The list of the prefix kernel: its tiles, and what the plan writes.
struct PrefixList {
  int tile_rows, tile_keys, setup, min_tiles, ctas;
  bool by_prompt;   // the prompt kernel's list is by row tile, the split kernel's by group
  int* limit;       // [n] shared tokens
  int* first;       // [n] first request with queries
  SeqInfo* groups;  // [n]
  long* bases;      // [n + 1] first entry of each group
  int* firsts;      // [n + 1] first row tile of each group
  PrefixTile* tiles;
  PrefixHead* head;
  int* begins;      // [ctas]
};
// The list of the own kernel.
struct OwnList {
  int rows, ctas;
  SeqInfo* info;   // [B]
  OwnPrefix* own;  // [B]
  long* starts;    // [B + 1]
  int* begins;     // [ctas]
};

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

// Checks requests and groups, cuts each prefix to what all of its requests have
// before their queries, and sums up both work lists. One block: a chain of a few
// loads, sums over the block and stores, all in shared memory in between.
__global__ void __launch_bounds__(kPlanThreads)
    shared_plan_kernel(AttnArgs a, Groups gr, PrefixList w, OwnList o, unsigned* status,
                       int* counters, int n_counters) {
  __shared__ long warp_sum[kPlanThreads / 32];
  __shared__ SeqInfo s_info[kSmallSeqs], s_groups[kSmallGroups];
  __shared__ long s_starts[kSmallSeqs + 1], s_bases[kSmallGroups + 1];
  __shared__ int s_group[kSmallSeqs], s_limit[kSmallGroups], s_first[kSmallGroups],
      s_firsts[kSmallGroups + 1], s_offsets[kSmallGroups + 1];
  __shared__ int s_longest;
  __shared__ unsigned long long s_tiles;
  if (threadIdx.x == 0) s_longest = 0, s_tiles = 0;
  pdl_enter();
  const bool few_seqs = a.B <= kSmallSeqs, few_groups = gr.n <= kSmallGroups;
  SeqInfo* info = few_seqs ? s_info : o.info;
  long* starts = few_seqs ? s_starts : o.starts;
  SeqInfo* groups = few_groups ? s_groups : w.groups;
  long* bases = few_groups ? s_bases : w.bases;
  int* limit = few_groups ? s_limit : w.limit;
  int* first = few_groups ? s_first : w.first;
  int* firsts = few_groups ? s_firsts : w.firsts;
  const int* offsets = few_groups ? s_offsets : gr.offsets;
  const int heads = a.heads / a.kv_heads;
  unsigned flags = 0;
  bool bad = false;
  if (threadIdx.x == 0) *status = 0;
  for (int g = threadIdx.x; g < gr.n; g += kPlanThreads) {
    const int b0 = gr.offsets[g], b1 = gr.offsets[g + 1], p = gr.prefix[g];
    bad |= b0 < 0 || b1 < b0 || b1 > a.B;
    if (p < 0) flags |= MOE_DEV_BAD_SEGMENT;
    limit[g] = max(0, p);
    first[g] = 0x7fffffff;
    if (few_groups) {
      s_offsets[g] = b0;
      if (g == gr.n - 1) s_offsets[gr.n] = b1;
    }
  }
  for (int b = threadIdx.x; b < a.B; b += kPlanThreads) info[b] = seq_info(a, b, flags);
  for (int i = threadIdx.x; i < n_counters; i += kPlanThreads) counters[i] = 0;
  bad = __syncthreads_or(bad);
  if (bad) flags |= MOE_DEV_BAD_SEGMENT;
  auto q_at = [&](int b) { return a.q_offsets ? a.q_offsets[b] : b; };
  for (int b = threadIdx.x; b < a.B; b += kPlanThreads) {
    const SeqInfo s = info[b];
    int g = bad || gr.n == 0 ? -1 : last_at_most(offsets, gr.n, b);
    if (g >= 0 && (b < offsets[g] || b >= offsets[g + 1])) g = -1;
    if (few_seqs) s_group[b] = g;
    else o.own[b].len = g;
    if (g < 0) continue;
    if (s.q_len > 0) {
      atomicMin(limit + g, max(0, s.len - s.q_len));
      atomicMin(first + g, b);
    } else if (q_at(b + 1) != q_at(b)) {
      atomicMin(limit + g, 0);  // its offsets were refused: its group's may be wrong
    }
  }
  __threadfence_block();
  __syncthreads();
  auto entries_of = [&](int p) { return w.setup + (p + w.tile_keys - 1) / w.tile_keys; };
  long entries = 0, tiles = 0;
  for (int g0 = 0; g0 < gr.n; g0 += kPlanThreads) {
    const int g = g0 + threadIdx.x;
    long n = 0, row_tiles = 0;
    if (g < gr.n) {
      SeqInfo s = {0, 0, 0, 0};
      int p = bad ? 0 : *const_cast<volatile int*>(limit + g) / kCut * kCut;
      if (p > 0) {
        const int b0 = offsets[g], b1 = offsets[g + 1];
        s.q0 = q_at(b0);
        s.q_len = q_at(b1) - s.q0;
        s.first_key = *const_cast<volatile int*>(first + g);
        if (s.q_len > gr.max_len) flags |= MOE_DEV_BAD_SEGMENT;
        if (b1 - b0 < 2 || s.q_len < 2 || s.q_len > gr.max_len) p = 0;  // nothing to share
      }
      s.len = p;
      if (p == 0) s.q_len = 0;
      limit[g] = p;
      groups[g] = s;
      if (few_groups) w.groups[g] = s;
      row_tiles = (static_cast<long>(s.q_len) * heads + w.tile_rows - 1) / w.tile_rows;
      n = row_tiles * a.kv_heads * entries_of(p);
    }
    const long before = block_scan<kPlanThreads>(n, warp_sum, entries);
    const long tiles_before = block_scan<kPlanThreads>(row_tiles, warp_sum, tiles);
    if (g < gr.n) {
      bases[g] = before;
      firsts[g] = static_cast<int>(tiles_before);
      if (few_groups) w.bases[g] = bases[g];
    }
  }
  long per = (entries + w.ctas - 1) / w.ctas;
  if (per < w.min_tiles) per = w.min_tiles;
  if (threadIdx.x == 0) {
    bases[gr.n] = entries;
    firsts[gr.n] = static_cast<int>(tiles);
    if (few_groups) w.bases[gr.n] = entries;
    w.head->total = entries;
    w.head->per = per;
  }
  __syncthreads();
  if (w.by_prompt)
    for (int r = threadIdx.x; r <= tiles; r += kPlanThreads) {
      if (r == tiles) {
        w.tiles[r] = {{0, 0, 0, 0}, entries, 0, 0};
        continue;
      }
      const int g = last_at_most(firsts, gr.n, r), i = r - firsts[g];
      const long start = bases[g] + static_cast<long>(i) * a.kv_heads * entries_of(limit[g]);
      w.tiles[r] = {groups[g], start, i * w.tile_rows, 0};
    }
  for (int c = threadIdx.x; c < w.ctas; c += kPlanThreads) {
    const long at = c * per;
    int begin = 0;
    if (at < entries) {
      begin = last_at_most(bases, gr.n, at);
      if (w.by_prompt)
        begin = firsts[begin] + static_cast<int>((at - bases[begin]) /
                                                 (a.kv_heads * entries_of(limit[begin])));
    }
    w.begins[c] = begin;
  }
  // The own kernel's segments: their number, and the tiles of the longest.
  long segs = 0, longest = 0, sum = 0;
  auto segments = [&](int q_len) {
    return (static_cast<long>(q_len) * heads + o.rows - 1) / o.rows * a.kv_heads;
  };
  auto tiles_of = [&](const SeqInfo& s) {
    return max(0, (s.len + split::kTile - 1) / split::kTile - s.first_key / split::kTile);
  };
  for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
    const int b = b0 + threadIdx.x;
    long n = 0, own_tiles = 0;
    if (b < a.B) {
      const int g = few_seqs ? s_group[b] : o.own[b].len, p = g >= 0 ? limit[g] : 0;
      SeqInfo s = info[b];
      s.first_key = p;
      info[b] = s;
      if (few_seqs) o.info[b] = s;
      o.own[b] = p > 0 ? OwnPrefix{bases[g], s.q0 - groups[g].q0, entries_of(p)} : OwnPrefix{0, 0, 0};
      n = segments(s.q_len);
      own_tiles = n > 0 ? tiles_of(s) : 0;
    }
    const long before = block_scan<kPlanThreads>(n, warp_sum, segs);
    if (b < a.B) {
      starts[b] = before;
      atomicMax(&s_longest, static_cast<int>(own_tiles));
      atomicAdd(&s_tiles, static_cast<unsigned long long>(n * own_tiles));
    }
  }
  __syncthreads();
  longest = split::kSetup + s_longest;
  sum = segs * split::kSetup + static_cast<long>(s_tiles);
  // Segments of one length, cut into the same number of pieces, one to a CTA, as
  // long as the longest does not hold up the others: a CTA with parts of two
  // segments takes about twice as long as with one, whatever its tiles.
  const long cuts = segs > 0 ? o.ctas / segs : 0;
  long own_per = cuts > 0 ? (longest + cuts - 1) / cuts : 0;
  const bool same = cuts > 0 && own_per <= sum / o.ctas + 2 * split::kSetup;
  if (same) {
    if (own_per < split::kMinTiles + split::kSetup) own_per = min(longest, static_cast<long>(split::kMinTiles + split::kSetup));
    const long len = (longest + own_per - 1) / own_per * own_per;
    for (int b = threadIdx.x; b <= a.B; b += kPlanThreads) {
      const long at = (b < a.B ? starts[b] : segs) * len;
      o.starts[b] = at;
      if (b < a.B && few_seqs) starts[b] = at;
    }
    if (threadIdx.x == 0) w.head->own_len = static_cast<int>(len);
  } else {
    long at = 0;
    for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
      const int b = b0 + threadIdx.x;
      long n = 0;
      if (b < a.B) n = segments(info[b].q_len) * (split::kSetup + tiles_of(info[b]));
      const long before = block_scan<kPlanThreads>(n, warp_sum, at);
      if (b < a.B) {
        starts[b] = before;
        if (few_seqs) o.starts[b] = before;
      }
    }
    own_per = split::range_len(at, o.ctas);
    if (threadIdx.x == 0) o.starts[a.B] = at, w.head->own_len = 0;
  }
  if (threadIdx.x == 0) w.head->own_per = own_per;
  __syncthreads();
  for (int c = threadIdx.x; c < o.ctas; c += kPlanThreads)
    o.begins[c] = last_at_most(starts, a.B, c * own_per);
  if (flags) atomicOr(status, flags);
}

struct Launch {
  AttnArgs a;       // the requests
  Groups gr;
  PrefixList list;
  OwnList own;
  PrefixSums sums;
  SharedLayout L;
  char* ws;
  cudaStream_t st;
  template <typename P>
  P* at(size_t off) const {
    return reinterpret_cast<P*>(ws + off);
  }
  int page_shift() const {
    int n = 0;
    while ((1 << n) < a.page_size) ++n;
    return n;
  }
  AttnArgs group_args() const {
    AttnArgs g = a;
    g.B = gr.n;
    return g;
  }
};

cudaError_t launch_plan(const Launch& l) {
  return launch_pdl(&shared_plan_kernel, dim3(1), dim3(kPlanThreads), 0, l.st, l.a, l.gr, l.list,
                    l.own, l.at<unsigned>(l.L.status), l.at<int>(l.L.counters), l.own.ctas);
}

template <typename T, int D, int kRows, int kTerms>
cudaError_t launch_own(const Launch& l) {
  auto* kern = &split::attn_split_kernel<T, D, kRows, kTerms, false, kOwn>;
  constexpr int smem = split::split_smem<D, kRows>();
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = opt_in_smem(reinterpret_cast<const void*>(kern), smem, done);
  if (e != cudaSuccess) return e;
  PrefixSums sums = l.sums;
  sums.begins = l.own.begins;
  return launch_pdl(kern, dim3(l.own.ctas), dim3(split::kThreads), smem, l.st, l.a,
                    l.at<unsigned>(l.L.status), l.at<int>(l.L.counters),
                    const_cast<const SeqInfo*>(l.own.info),
                    const_cast<const long*>(l.own.starts), l.at<float>(l.L.stats),
                    l.at<float>(l.L.partial), l.page_shift(), PartArgs<kOwn>{sums});
}

template <typename T, int D, int kRows, int kTerms>
cudaError_t launch_prefix_split(const Launch& l) {
  auto* kern = &split::attn_split_kernel<T, D, kRows, kTerms, false, kPrefix>;
  constexpr int smem = split::split_smem<D, kRows>();
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = opt_in_smem(reinterpret_cast<const void*>(kern), smem, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(l.list.ctas), dim3(split::kThreads), smem, l.st, l.group_args(),
                    l.at<unsigned>(l.L.status), static_cast<int*>(nullptr),
                    const_cast<const SeqInfo*>(l.list.groups),
                    const_cast<const long*>(l.list.bases), l.at<float>(l.L.prefix_stats),
                    l.at<float>(l.L.prefix_partial), l.page_shift(), PartArgs<kPrefix>{l.sums});
}

template <int D>
cudaError_t launch_prefix_prompt(const Launch& l) {
  auto* kern = &prompt::attn_prompt_kernel<D, kPrefix>;
  constexpr int smem = prompt::Shape<D>::kBytes;
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = opt_in_smem(reinterpret_cast<const void*>(kern), smem, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(l.list.ctas), dim3(prompt::kThreads), smem, l.st, l.group_args(),
                    l.at<unsigned>(l.L.status), static_cast<int*>(nullptr),
                    static_cast<const SeqInfo*>(nullptr), static_cast<const int*>(nullptr),
                    static_cast<const prompt::RowTile*>(nullptr),
                    static_cast<const long*>(nullptr), l.at<float2>(l.L.prefix_stats),
                    l.at<float4>(l.L.prefix_partial), PartArgs<kPrefix>{l.sums});
}

// Rows of a row tile of the split kernel over a prefix.
constexpr int prefix_rows(bool bf16) { return bf16 ? 16 : 8; }

bool prefix_by_prompt(const moe_attn_config* c, int max_group) {
  return c->act_dtype == MOE_BF16 &&
         static_cast<long>(max_group) * (c->num_heads / c->num_kv_heads) >= kPromptRows;
}

template <int D>
cudaError_t launch_dim(const moe_attn_config* c, Launch& l) {
  const bool bf16 = c->act_dtype == MOE_BF16, by_prompt = prefix_by_prompt(c, l.gr.max_len);
  const long rows = static_cast<long>(l.a.max_q) * (c->num_heads / c->num_kv_heads);
  PrefixList& w = l.list;
  w.by_prompt = by_prompt;
  if (by_prompt) {
    using H = prompt::Shape<D>;
    w.tile_rows = H::kTile, w.tile_keys = H::kKeys;
    w.setup = prompt::kSetup, w.min_tiles = kMinPrefix, w.ctas = l.a.sms;
    l.sums.lo = prompt::kSetup, l.sums.hi = prompt::kPrefixSnap + 1;
  } else {
    w.tile_rows = prefix_rows(bf16), w.tile_keys = split::kTile;
    w.setup = split::kSetup, w.min_tiles = split::kMinTiles;
    w.ctas = l.a.sms * (bf16 ? split::ctas_per_sm<D, prefix_rows(true), 1>()
                             : split::ctas_per_sm<D, prefix_rows(false), 2>());
    l.sums.lo = split::kSetup - 1, l.sums.hi = 1;
  }
  l.sums.tile_rows = w.tile_rows;
  // the kernels: (type, rows of a row tile)
  auto own = [&](auto launch, int ctas_per_sm) {
    l.own.ctas = l.a.sms * ctas_per_sm;
    cudaError_t e = launch_plan(l);
    if (e != cudaSuccess) return e;
    e = by_prompt ? launch_prefix_prompt<D>(l)
        : bf16    ? launch_prefix_split<__nv_bfloat16, D, prefix_rows(true), 1>(l)
                  : launch_prefix_split<float, D, prefix_rows(false), 2>(l);
    return e == cudaSuccess ? launch(l) : e;
  };
  l.own.rows = rows <= 4 ? 4 : rows <= 8 || !bf16 ? 8 : 16;
  if (!bf16)
    return l.own.rows == 4 ? own(launch_own<float, D, 4, 2>, split::ctas_per_sm<D, 4, 2>())
                           : own(launch_own<float, D, 8, 2>, split::ctas_per_sm<D, 8, 2>());
  return l.own.rows == 4
             ? own(launch_own<__nv_bfloat16, D, 4, 1>, split::ctas_per_sm<D, 4, 1>())
         : l.own.rows == 8
             ? own(launch_own<__nv_bfloat16, D, 8, 1>, split::ctas_per_sm<D, 8, 1>())
             : own(launch_own<__nv_bfloat16, D, 16, 1>, split::ctas_per_sm<D, 16, 1>());
}

}  // namespace

// Requests of that many rows fill half a row tile of the prompt kernel by
// themselves: its matrix work is no longer shared then, and their own keys are
// better off there than with the split kernel, which goes through them once per
// 16 rows. A window ends the sharing too: it begins elsewhere for each request.
bool shares_prefix(const moe_attn_config* c, int max_q, int groups) {
  if (groups == 0 || c->window > 0) return false;
  return c->act_dtype != MOE_BF16 ||
         static_cast<long>(max_q) * (c->num_heads / c->num_kv_heads) < kSharedRows;
}

SharedLayout shared_layout(const moe_attn_config* c, int B, int T, int groups, int max_group) {
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  const bool by_prompt = prefix_by_prompt(c, max_group);
  const size_t D = c->head_dim, heads = c->num_heads / c->num_kv_heads, b = B, g = groups;
  const size_t ctas = static_cast<size_t>(kAttnMaxSms) * split::kMaxCtasPerSm;
  const size_t own_rows = 2 * ctas * 16;  // two pieces per CTA
  const size_t prefix_rows = by_prompt ? 2 * static_cast<size_t>(kAttnMaxSms) * prompt_tile(c->head_dim)
                                       : own_rows;
  const size_t row_tiles = by_prompt ? T * heads / prompt_tile(c->head_dim) + g : 0;
  const size_t rows = static_cast<size_t>(T) * c->num_heads;
  SharedLayout L;
  L.status = 0;
  L.head = 64;
  L.counters = 256;
  L.own_begins = up(L.counters + 4 * ctas);
  L.prefix_begins = up(L.own_begins + 4 * ctas);
  L.info = up(L.prefix_begins + 4 * ctas);
  L.own = up(L.info + sizeof(SeqInfo) * b);
  L.starts = up(L.own + sizeof(OwnPrefix) * b);
  L.limit = up(L.starts + 8 * (b + 1));
  L.first = up(L.limit + 4 * g);
  L.groups = up(L.first + 4 * g);
  L.bases = up(L.groups + sizeof(SeqInfo) * g);
  L.firsts = up(L.bases + 8 * (g + 1));
  L.tiles = up(L.firsts + 4 * (g + 1));
  L.stats = up(L.tiles + sizeof(PrefixTile) * (row_tiles + 1));
  L.partial = up(L.stats + 8 * own_rows);
  L.prefix_stats = up(L.partial + 4 * D * own_rows);
  L.prefix_partial = up(L.prefix_stats + 8 * prefix_rows);
  L.row_stats = up(L.prefix_partial + 4 * D * prefix_rows);
  L.row_sums = up(L.row_stats + 8 * rows);
  L.total = up(L.row_sums + 4 * D * rows);
  return L;
}

cudaError_t launch_kv_attention_shared(const moe_attn_config* c, const AttnArgs& a, int groups,
                                       const int32_t* group_offsets, const int32_t* prefix_lens,
                                       int max_group, void* ws, const SharedLayout& L,
                                       cudaStream_t st) {
  Launch l;
  l.a = a;
  l.gr = {groups, group_offsets, prefix_lens, max_group};
  l.L = L, l.ws = static_cast<char*>(ws), l.st = st;
  l.list.limit = l.at<int>(L.limit), l.list.first = l.at<int>(L.first);
  l.list.groups = l.at<SeqInfo>(L.groups), l.list.bases = l.at<long>(L.bases);
  l.list.firsts = l.at<int>(L.firsts), l.list.tiles = l.at<PrefixTile>(L.tiles);
  l.list.head = l.at<PrefixHead>(L.head), l.list.begins = l.at<int>(L.prefix_begins);
  l.own.info = l.at<SeqInfo>(L.info), l.own.own = l.at<OwnPrefix>(L.own);
  l.own.starts = l.at<long>(L.starts), l.own.begins = l.at<int>(L.own_begins);
  l.sums.row_stats = l.at<float2>(L.row_stats), l.sums.row_sums = l.at<float4>(L.row_sums);
  l.sums.stats = l.at<float2>(L.prefix_stats), l.sums.sums = l.at<float4>(L.prefix_partial);
  l.sums.own = l.own.own, l.sums.head = l.list.head, l.sums.tiles = l.list.tiles;
  l.sums.begins = l.list.begins;
  switch (a.D) {
    case 64:
      return launch_dim<64>(c, l);
    case 128:
      return launch_dim<128>(c, l);
    default:
      return launch_dim<256>(c, l);
  }
}

}  // namespace moe
