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

constexpr int kPlanThreads = 1024;
// A prefix is cut to whole tiles of the split kernel, so that the own keys begin
// with one.
constexpr int kCut = split::kTile;

struct Groups {
  int n;
  const int32_t* offsets;  // [n + 1] requests
  const int32_t* prefix;   // [n] tokens
  int max_len;             // query tokens
};

// The list of the prefix kernel: its tiles, and what the plan writes.
struct PrefixList {
  int tile_rows, tile_keys, setup, min_tiles, ctas;
  int max_row_tiles;  // 0: the split kernel, whose list is by group
  int* limit;         // [n] shared tokens
  int* first;         // [n] first request with queries
  SeqInfo* groups;    // [n]
  long* bases;        // [n + 1] first entry of each group
  int* firsts;        // prompt: [n + 1] first row tile of each group
  prompt::RowTile* row_tiles;
  long* starts;       // prompt: first entry of each row tile
  long* per;
};

// Checks requests and groups, cuts each prefix to what all of its requests have
// before their queries, and sums up both work lists.
__global__ void __launch_bounds__(kPlanThreads)
    shared_plan_kernel(AttnArgs a, Groups gr, PrefixList w, int own_rows, unsigned* status,
                       int* counters, int n_counters, SeqInfo* info, OwnPrefix* own, long* starts) {
  __shared__ long warp_sum[kPlanThreads / 32];
  pdl_enter();
  if (threadIdx.x == 0) *status = 0;
  for (int i = threadIdx.x; i < n_counters; i += kPlanThreads) counters[i] = 0;
  const int heads = a.heads / a.kv_heads;
  unsigned flags = 0;
  bool bad = false;
  for (int g = threadIdx.x; g < gr.n; g += kPlanThreads) {
    const int b0 = gr.offsets[g], b1 = gr.offsets[g + 1], p = gr.prefix[g];
    bad |= b0 < 0 || b1 < b0 || b1 > a.B;
    if (p < 0) flags |= MOE_DEV_BAD_SEGMENT;
    w.limit[g] = max(0, p);
    w.first[g] = 0x7fffffff;
  }
  bad = __syncthreads_or(bad);
  if (bad) flags |= MOE_DEV_BAD_SEGMENT;
  for (int b = threadIdx.x; b < a.B; b += kPlanThreads) {
    unsigned wrong = 0;
    const SeqInfo s = seq_info(a, b, wrong);
    flags |= wrong;
    info[b] = s;
    int lo = 0, hi = bad ? 0 : gr.n;  // the last group that begins at b or before
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (gr.offsets[mid] <= b) lo = mid;
      else hi = mid;
    }
    const bool in = hi > 0 && gr.offsets[lo] <= b && b < gr.offsets[lo + 1];
    own[b] = {0, 0, in ? lo : -1};
    if (!in) continue;
    if (wrong & MOE_DEV_BAD_SEGMENT) {
      atomicMin(w.limit + lo, 0);
    } else if (s.q_len > 0) {
      atomicMin(w.limit + lo, max(0, s.len - s.q_len));
      atomicMin(w.first + lo, b);
    }
  }
  __threadfence();
  __syncthreads();
  auto q_at = [&](int b) { return a.q_offsets ? a.q_offsets[b] : b; };
  auto entries_of = [&](int p) { return w.setup + (p + w.tile_keys - 1) / w.tile_keys; };
  long entries = 0, tiles = 0;
  for (int g0 = 0; g0 < gr.n; g0 += kPlanThreads) {
    const int g = g0 + threadIdx.x;
    long n = 0, row_tiles = 0;
    if (g < gr.n) {
      SeqInfo s = {0, 0, 0, 0};
      int p = bad ? 0 : __ldcg(w.limit + g) / kCut * kCut;
      if (p > 0) {
        const int b0 = gr.offsets[g], b1 = gr.offsets[g + 1];
        s.q0 = q_at(b0);
        s.q_len = q_at(b1) - s.q0;
        s.first_key = __ldcg(w.first + g);
        if (s.q_len > gr.max_len) flags |= MOE_DEV_BAD_SEGMENT;
        if (b1 - b0 < 2 || s.q_len < 2 || s.q_len > gr.max_len) p = 0;  // nothing to share
      }
      s.len = p;
      if (p == 0) s.q_len = 0;
      w.limit[g] = p;
      w.groups[g] = s;
      row_tiles = (static_cast<long>(s.q_len) * heads + w.tile_rows - 1) / w.tile_rows;
      n = row_tiles * a.kv_heads * entries_of(p);
    }
    const long before = block_scan<kPlanThreads>(n, warp_sum, entries);
    const long first = block_scan<kPlanThreads>(row_tiles, warp_sum, tiles);
    if (g < gr.n) {
      w.bases[g] = before;
      if (w.max_row_tiles > 0) w.firsts[g] = static_cast<int>(first);
    }
  }
  if (threadIdx.x == 0) {
    w.bases[gr.n] = entries;
    if (w.max_row_tiles > 0) w.firsts[gr.n] = static_cast<int>(tiles), w.starts[tiles] = entries;
    const long per = (entries + w.ctas - 1) / w.ctas;
    *w.per = per < w.min_tiles ? w.min_tiles : per;
  }
  __syncthreads();
  if (w.max_row_tiles > 0) {
    for (int r = threadIdx.x; r < tiles; r += kPlanThreads) {
      int lo = 0, hi = gr.n;  // the last group whose first row tile is at most r
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (w.firsts[mid] <= r) lo = mid;
        else hi = mid;
      }
      const int i = r - w.firsts[lo];
      w.row_tiles[r] = {lo, i * w.tile_rows};
      w.starts[r] = w.bases[lo] + static_cast<long>(i) * a.kv_heads * entries_of(w.limit[lo]);
    }
  }
  long sum = 0;
  for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
    const int b = b0 + threadIdx.x;
    long n = 0;
    if (b < a.B) {
      const int g = own[b].len, p = g >= 0 ? w.limit[g] : 0;
      const SeqInfo s = info[b];
      info[b].first_key = p;
      own[b] = p > 0 ? OwnPrefix{w.bases[g], s.q0 - w.groups[g].q0, entries_of(p)} : OwnPrefix{0, 0, 0};
      const long row_tiles = (static_cast<long>(s.q_len) * heads + own_rows - 1) / own_rows;
      const int per = (s.len + split::kTile - 1) / split::kTile - p / split::kTile;
      n = row_tiles * a.kv_heads * (split::kSetup + max(0, per));
    }
    const long before = block_scan<kPlanThreads>(n, warp_sum, sum);
    if (b < a.B) starts[b] = before;
  }
  if (threadIdx.x == 0) starts[a.B] = sum;
  if (flags) atomicOr(status, flags);
}

struct Launch {
  AttnArgs a;       // the requests
  Groups gr;
  PrefixList list;
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

cudaError_t launch_plan(const Launch& l, int own_rows, int counters) {
  return launch_pdl(&shared_plan_kernel, dim3(1), dim3(kPlanThreads), 0, l.st, l.a, l.gr, l.list,
                    own_rows, l.at<unsigned>(l.L.status), l.at<int>(l.L.counters), counters,
                    l.at<SeqInfo>(l.L.info), l.at<OwnPrefix>(l.L.own), l.at<long>(l.L.starts));
}

template <typename T, int D, int kRows, int kTerms>
cudaError_t launch_own(const Launch& l) {
  auto* kern = &split::attn_split_kernel<T, D, kRows, kTerms, false, kOwn>;
  constexpr int smem = split::split_smem<D, kRows>();
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = opt_in_smem(reinterpret_cast<const void*>(kern), smem, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(l.a.sms * split::ctas_per_sm<D, kRows, kTerms>()),
                    dim3(split::kThreads), smem, l.st, l.a, l.at<unsigned>(l.L.status),
                    l.at<int>(l.L.counters), const_cast<const SeqInfo*>(l.at<SeqInfo>(l.L.info)),
                    const_cast<const long*>(l.at<long>(l.L.starts)), l.at<float>(l.L.stats),
                    l.at<float>(l.L.partial), l.page_shift(), PartArgs<kOwn>{l.sums});
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
                    const_cast<const SeqInfo*>(l.list.groups),
                    const_cast<const int*>(l.list.firsts),
                    const_cast<const prompt::RowTile*>(l.list.row_tiles),
                    const_cast<const long*>(l.list.starts), l.at<float2>(l.L.prefix_stats),
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
  const int own_rows = rows <= 4 ? 4 : rows <= 8 || !bf16 ? 8 : 16;
  PrefixList& w = l.list;
  if (by_prompt) {
    using H = prompt::Shape<D>;
    w.tile_rows = H::kTile, w.tile_keys = H::kKeys;
    w.setup = prompt::kSetup, w.min_tiles = prompt::kMinTiles, w.ctas = l.a.sms;
    l.sums.chunk = prompt::kHalf, l.sums.lo = prompt::kSnap, l.sums.hi = prompt::kSnap + 1;
  } else {
    w.tile_rows = prefix_rows(bf16), w.tile_keys = split::kTile;
    w.setup = split::kSetup, w.min_tiles = split::kMinTiles;
    w.ctas = l.a.sms * (bf16 ? split::ctas_per_sm<D, prefix_rows(true), 1>()
                             : split::ctas_per_sm<D, prefix_rows(false), 2>());
    l.sums.chunk = 1, l.sums.lo = split::kSetup - 1, l.sums.hi = 1;
  }
  l.sums.tile_rows = w.tile_rows;
  cudaError_t e = launch_plan(l, own_rows, l.a.sms * split::kMaxCtasPerSm);
  if (e != cudaSuccess) return e;
  e = by_prompt ? launch_prefix_prompt<D>(l)
      : bf16    ? launch_prefix_split<__nv_bfloat16, D, prefix_rows(true), 1>(l)
                : launch_prefix_split<float, D, prefix_rows(false), 2>(l);
  if (e != cudaSuccess) return e;
  if (!bf16) return own_rows == 4 ? launch_own<float, D, 4, 2>(l) : launch_own<float, D, 8, 2>(l);
  return own_rows == 4   ? launch_own<__nv_bfloat16, D, 4, 1>(l)
         : own_rows == 8 ? launch_own<__nv_bfloat16, D, 8, 1>(l)
                         : launch_own<__nv_bfloat16, D, 16, 1>(l);
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
  L.per = 16;
  L.counters = 256;
  L.info = up(L.counters + 4 * ctas);
  L.own = up(L.info + sizeof(SeqInfo) * b);
  L.starts = up(L.own + sizeof(OwnPrefix) * b);
  L.limit = up(L.starts + 8 * (b + 1));
  L.first = up(L.limit + 4 * g);
  L.groups = up(L.first + 4 * g);
  L.bases = up(L.groups + sizeof(SeqInfo) * g);
  L.firsts = up(L.bases + 8 * (g + 1));
  L.row_tiles = up(L.firsts + 4 * (g + 1));
  L.row_starts = up(L.row_tiles + 8 * row_tiles);
  L.stats = up(L.row_starts + 8 * (row_tiles + 1));
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
  const size_t heads = c->num_heads / c->num_kv_heads;
  l.list.max_row_tiles =
      prefix_by_prompt(c, max_group)
          ? static_cast<int>(a.T * heads / prompt_tile(c->head_dim)) + groups
          : 0;
  l.list.limit = l.at<int>(L.limit), l.list.first = l.at<int>(L.first);
  l.list.groups = l.at<SeqInfo>(L.groups), l.list.bases = l.at<long>(L.bases);
  l.list.firsts = l.at<int>(L.firsts), l.list.row_tiles = l.at<prompt::RowTile>(L.row_tiles);
  l.list.starts = l.at<long>(L.row_starts), l.list.per = l.at<long>(L.per);
  l.sums.row_stats = l.at<float2>(L.row_stats), l.sums.row_sums = l.at<float4>(L.row_sums);
  l.sums.stats = l.at<float2>(L.prefix_stats), l.sums.sums = l.at<float4>(L.prefix_partial);
  l.sums.own = l.at<OwnPrefix>(L.own), l.sums.per = l.at<long>(L.per);
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
