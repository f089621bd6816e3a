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
//
// Three kernels: the plan (one block, the lists of the own kernel), the prefix kernel,
// which sums up its own list in every CTA and so begins beside the plan, and the own
// kernel, which goes through its keys before it waits for the prefix sums.
//
// Measured, 32 query and 8 kv heads of 128: 64 requests behind 32768 tokens with up
// to 1024 of their own 56 us, from a kernel's start: lists 2.3, first product at 9,
// 13.5 tiles of 1.9 us, sums out 2.4, own keys 5 to 11, sums in 4. Three groups of 48
// requests with 2 query tokens behind 20000 to 65535 tokens 249 us, 0.71 PFLOP/s, 37 %
// of the measured matrix rate (every other row tile there is half empty).
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
// Up to so many requests the plan keeps its lists in shared memory.
constexpr int kSmallSeqs = 1024;
static_assert(kPrefixCut == split::kTile, "own keys begin with a tile");

// Pieces are not cut below kShortPiece tiles, and not taken where they are longer
// than a CTA's share of all entries and kPieceSlack more. Equal ranges and pieces,
// prefixes of 4096 tokens, heads as above: 64 requests of up to 1024 own tokens 39
// and 32 us, 4 of up to 4096 25 and 22; 64 of up to 4096 39 and 46, so ranges there.
constexpr int kPieceSlack = 8, kShortPiece = 12;
// The list of the own kernel.
struct OwnList {
  int rows, ctas;
  SeqInfo* info;   // [B]
  OwnPrefix* own;  // [B]
  long* starts;    // [B + 1]
  int* begins;     // [ctas]
};

// The lists of the own kernel, and of more than kSmallGroups groups also that of
// the prefix kernel. One block: a chain of a few loads, sums over the block and
// stores, in shared memory in between.
__global__ void __launch_bounds__(kPlanThreads)
    shared_plan_kernel(AttnArgs a, Groups gr, PrefixShape w, GroupLists lists, PrefixHead* head,
                       OwnList o, unsigned* status, int* counters, int n_counters) {
  __shared__ long warp_sum[kPlanThreads / 32];
  __shared__ GroupSmem s_groups;
  __shared__ SeqInfo s_info[kSmallSeqs];
  __shared__ long s_starts[kSmallSeqs];
  __shared__ int s_group[kSmallSeqs], s_longest, s_enough[kPlanThreads / 32];
  if (threadIdx.x == 0) s_longest = 0;
  // the prefix kernel may report before this one ends: the status first
  pdl_wait();
  if (threadIdx.x == 0) {
    *status = 0;
    __threadfence();
  }
  __syncthreads();
  pdl_launch_dependents();
  const bool few_seqs = a.B <= kSmallSeqs, few_groups = gr.n <= kSmallGroups;
  SeqInfo* info = few_seqs ? s_info : o.info;
  long* starts = few_seqs ? s_starts : o.starts;
  const GroupLists l = few_groups ? s_groups.lists() : lists;
  const int heads = a.heads / a.kv_heads;
  unsigned flags = 0;
  const long entries = plan_groups<kPlanThreads>(
      a, gr, w, l, few_groups ? &s_groups : nullptr, warp_sum, flags,
      [&](int b, const SeqInfo& s, int g) {
        info[b] = s;
        if (few_seqs) s_group[b] = g;
        else o.own[b].len = g;
      });
  for (int i = threadIdx.x; i < n_counters; i += kPlanThreads) counters[i] = 0;
  if (threadIdx.x == 0) head->per = prefix_per(w, entries);
  // The own kernel's segments: their number, and the tiles of the longest.
  long segs = 0, sum = 0;
  auto segments = [&](int q_len) {  // (rows of a request: below 2^28)
    return static_cast<long>((q_len * heads + o.rows - 1) / o.rows) * a.kv_heads;
  };
  auto tiles_of = [&](const SeqInfo& s) {
    return max(0, (s.len + split::kTile - 1) / split::kTile - s.first_key / split::kTile);
  };
  for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
    const int b = b0 + threadIdx.x;
    long n = 0, own_tiles = 0;
    if (b < a.B) {
      const int g = few_seqs ? s_group[b] : o.own[b].len, p = g >= 0 ? l.limit[g] : 0;
      SeqInfo s = info[b];
      s.first_key = p;
      info[b] = s;
      if (few_seqs) o.info[b] = s;
      o.own[b] = p > 0 ? OwnPrefix{l.bases[g], s.q0 - l.groups[g].q0, prefix_entries(w, p, false),
                                   prefix_entries(w, p, true), l.groups[g].q_len * heads}
                       : OwnPrefix{0, 0, 0, 0, 0};
      n = segments(s.q_len);
      own_tiles = n > 0 ? tiles_of(s) : 0;
    }
    const long before = block_scan<kPlanThreads>(n, warp_sum, segs);
    block_scan<kPlanThreads>(n * own_tiles, warp_sum, sum);
    if (b < a.B) starts[b] = before;
    const int most = __reduce_max_sync(~0u, static_cast<int>(own_tiles));
    if (threadIdx.x % 32 == 0) atomicMax(&s_longest, most);
  }
  __syncthreads();
  // Whole pieces, one to a CTA: of as few tiles as give no more pieces than CTAs. A
  // part of a segment takes a CTA as long as 16 tiles beside its own, so that equal
  // ranges, where most CTAs have parts of two segments, pay only where there are
  // more segments than CTAs, few of them, or some much longer than the others.
  const int fours = (s_longest + 3) / 4;  // pieces of whole fours, a tile for each warp
  long own_per = 0;
  int piece = 0;
  if (few_seqs && segs <= o.ctas) {
    int hi = max(1, fours), lo = min(kShortPiece / 4 - 1, hi - 1);  // lo fours are too few, hi are enough
    while (hi - lo > 1) {            // a warp per candidate
      const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = kPlanThreads / 32;
      auto candidate = [&](int w) {
        return lo + max(1, static_cast<int>(static_cast<long>(hi - lo) * (w + 1) / (warps + 1)));
      };
      const int tiles = 4 * candidate(warp);
      long n = 0;
      for (int b = lane; b < a.B; b += 32) {
        const int t = tiles_of(info[b]);
        n += segments(info[b].q_len) * max(1, (t + tiles - 1) / tiles);
      }
#pragma unroll
      for (int d = 16; d > 0; d /= 2) n += __shfl_xor_sync(~0u, n, d);
      if (lane == 0) s_enough[warp] = n <= o.ctas;
      __syncthreads();
      int most = lo, least = hi;
      for (int w = 0; w < warps; ++w) {
        if (s_enough[w]) least = min(least, candidate(w));
        else most = max(most, candidate(w));
      }
      lo = most, hi = least;
      __syncthreads();
    }
    own_per = piece = 4 * hi;
    if (piece > kShortPiece &&
        (piece - kPieceSlack) * static_cast<long>(o.ctas) > sum + segs * split::kSetup)
      piece = 0;
  }
  if (piece > 0) {
    long at = 0;
    for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
      const int b = b0 + threadIdx.x;
      long n = 0;
      if (b < a.B) n = segments(info[b].q_len) * max(1, (tiles_of(info[b]) + piece - 1) / piece) * piece;
      const long before = block_scan<kPlanThreads>(n, warp_sum, at);
      if (b < a.B) starts[b] = o.starts[b] = before;
    }
    if (threadIdx.x == 0) o.starts[a.B] = at, head->own_piece = piece;
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
    if (threadIdx.x == 0) o.starts[a.B] = at, head->own_piece = 0;
  }
  if (threadIdx.x == 0) head->own_per = own_per;
  __syncthreads();
  for (int c = threadIdx.x; c < o.ctas; c += kPlanThreads)
    o.begins[c] = last_at_most(starts, a.B, c * own_per);
  if (flags) atomicOr(status, flags);
}

struct Launch {
  AttnArgs a;  // the requests
  GroupLists lists;
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
};

cudaError_t launch_plan(const Launch& l) {
  return launch_pdl(&shared_plan_kernel, dim3(1), dim3(kPlanThreads), 0, l.st, l.a, l.sums.gr,
                    l.sums.shape, l.lists, l.at<PrefixHead>(l.L.head), l.own,
                    l.at<unsigned>(l.L.status), l.at<int>(l.L.counters), l.own.ctas);
}

template <typename T, int D, int kRows, int kTerms>
cudaError_t launch_own(const Launch& l) {
  auto* kern = &split::attn_split_kernel<T, D, kRows, kTerms, false, kOwn>;
  constexpr int smem = split::split_smem<D, kRows>();
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = opt_in_smem(reinterpret_cast<const void*>(kern), smem, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(l.own.ctas), dim3(split::kThreads), smem, l.st, l.a,
                    l.at<unsigned>(l.L.status), l.at<int>(l.L.counters),
                    const_cast<const SeqInfo*>(l.own.info),
                    const_cast<const long*>(l.own.starts), l.at<float>(l.L.stats),
                    l.at<float>(l.L.partial), l.page_shift(), PartArgs<kOwn>{l.sums});
}

template <typename T, int D, int kRows, int kTerms>
cudaError_t launch_prefix_split(const Launch& l) {
  auto* kern = &split::attn_split_kernel<T, D, kRows, kTerms, false, kPrefix>;
  constexpr int smem = split::split_smem<D, kRows>();
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = opt_in_smem(reinterpret_cast<const void*>(kern), smem, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(l.sums.shape.ctas), dim3(split::kThreads), smem, l.st, l.a,
                    l.at<unsigned>(l.L.status), static_cast<int*>(nullptr),
                    static_cast<const SeqInfo*>(nullptr), static_cast<const long*>(nullptr),
                    l.at<float>(l.L.prefix_stats),
                    l.at<float>(l.L.prefix_partial), l.page_shift(), PartArgs<kPrefix>{l.sums});
}

template <int D>
cudaError_t launch_prefix_prompt(const Launch& l) {
  auto* kern = &prompt::attn_prompt_kernel<D, kPrefix>;
  constexpr int smem = prompt::Shape<D>::kPrefixBytes;
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = opt_in_smem(reinterpret_cast<const void*>(kern), smem, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(l.sums.shape.ctas), dim3(prompt::kThreads), smem, l.st, l.a,
                    l.at<unsigned>(l.L.status), static_cast<int*>(nullptr),
                    static_cast<const SeqInfo*>(nullptr), static_cast<const int*>(nullptr),
                    static_cast<const prompt::RowTile*>(nullptr),
                    static_cast<const long*>(nullptr), l.at<float2>(l.L.prefix_stats),
                    l.at<float4>(l.L.prefix_partial), PartArgs<kPrefix>{l.sums});
}

// Rows of a row tile of the split kernel over a prefix.
constexpr int prefix_rows(bool bf16) { return bf16 ? 16 : 8; }

// One kernel for all prefixes of a call, by the caller's bound on a group's tokens: a
// small group's rows then fill a row tile of 128 rows in part. 32 query and 8 kv
// heads of 128, split and prompt kernel (and unshared): ten groups of 2 requests
// behind 16384 tokens 69 and 117 us (80), of 8 127 and 126 (282), four of 12 behind
// 32768 142 and 100 (334), one of 4 26 and 41 (39), one of 12 46 and 42 (92).
bool prefix_by_prompt(const moe_attn_config* c, int max_group) {
  return c->act_dtype == MOE_BF16 &&
         static_cast<long>(max_group) * (c->num_heads / c->num_kv_heads) >= kPromptRows;
}

template <int D>
cudaError_t launch_dim(const moe_attn_config* c, Launch& l) {
  const bool bf16 = c->act_dtype == MOE_BF16, by_prompt = prefix_by_prompt(c, l.sums.gr.max_len);
  const long rows = static_cast<long>(l.a.max_q) * (c->num_heads / c->num_kv_heads);
  PrefixShape& w = l.sums.shape;
  if (by_prompt) {
    using H = prompt::Shape<D>;
    w.tile_rows = H::kTile, w.tile_keys = H::kKeys;
    w.setup = prompt::kPrefixSetup, w.least = prompt::kMinPrefix, w.ctas = l.a.sms;
    w.unit = prompt::kUnit, w.half_unit = prompt::kHalfUnit;
    w.half_rows = H::kHalves == 2 ? prompt::kHalf : 0;
    l.sums.lo = prompt::kPrefixSetup, l.sums.hi = prompt::kPrefixSnap + 1;
  } else {
    w.tile_rows = prefix_rows(bf16), w.tile_keys = split::kTile;
    w.setup = split::kSetup, w.least = split::kMinTiles;
    w.ctas = l.a.sms * (bf16 ? split::ctas_per_sm<D, prefix_rows(true), 1>()
                             : split::ctas_per_sm<D, prefix_rows(false), 2>());
    l.sums.lo = split::kSetup - 1, l.sums.hi = 1;
  }
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

// Requests of so many rows (bf16) fill half a row tile of the prompt kernel by
// themselves: its matrix work is no longer shared then, and their own keys are
// better off there than with the split kernel, which goes through them once per
// 16 rows. A window ends the sharing too: it begins elsewhere for each request.
constexpr int kMostRows = 128;
bool can_share(const moe_attn_config* c, int max_q, int groups) {
  if (groups == 0 || c->window > 0) return false;
  return c->act_dtype != MOE_BF16 ||
         static_cast<long>(max_q) * (c->num_heads / c->num_kv_heads) < kMostRows;
}

// Sharing takes one kernel more, and some 4 us; reading the keys of every request
// takes as long from about 40 MB on: 4 requests of 4160 tokens (8 kv heads of 128,
// 19 MB) unshared 14.6 us and shared 16.4, of 16448 (76 MB) 25.9 and 22.1; 16 of
// 1088 (19 MB) 14.2 and 17.9, of 4160 (76 MB) 25.1 and 22.0; 64 of 320 (20 MB)
// 17.4 and 20.5, of 1088 (77 MB) 27.5 and 22.6; fp32, 32 of 2064 (37 MB) 23.5 and
// 24.0. Lengths are not known here: the page table's width bounds them. From
// kPromptRows rows a request the unshared call takes the prompt kernel, whose row
// tiles are then half empty (4 requests of 72 rows, 9 MB: 49 and 24 us).
constexpr double kShareBytes = 40e6;
bool worth_sharing(const moe_attn_config* c, int B, int max_q, int max_pages) {
  if (c->act_dtype == MOE_BF16 &&
      static_cast<long>(max_q) * (c->num_heads / c->num_kv_heads) >= kPromptRows)
    return true;
  const double tokens = static_cast<double>(B) * max_pages * c->page_size;
  return tokens * c->num_kv_heads * (c->head_dim * 9 / 8) > kShareBytes;
}

SharedLayout shared_layout(const moe_attn_config* c, int B, int T, int groups, int max_group) {
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  const bool by_prompt = prefix_by_prompt(c, max_group);
  const size_t D = c->head_dim, b = B, g = groups;
  const size_t ctas = static_cast<size_t>(kAttnMaxSms) * split::kMaxCtasPerSm;
  const size_t own_rows = 2 * ctas * 16;  // two pieces per CTA
  const size_t prefix_rows = by_prompt ? 2 * static_cast<size_t>(kAttnMaxSms) * prompt_tile(c->head_dim)
                                       : own_rows;
  const size_t rows = (static_cast<size_t>(T) * c->num_heads + 7) / 8 * 8;
  SharedLayout L;
  L.status = 0;
  L.head = 64;
  L.counters = 256;
  L.begins = up(L.counters + 4 * ctas);
  L.info = up(L.begins + 4 * ctas);
  L.own = up(L.info + sizeof(SeqInfo) * b);
  L.starts = up(L.own + sizeof(OwnPrefix) * b);
  L.limit = up(L.starts + 8 * (b + 1));
  L.first = up(L.limit + 4 * g);
  L.groups = up(L.first + 4 * g);
  L.bases = up(L.groups + sizeof(SeqInfo) * g);
  L.stats = up(L.bases + 8 * (g + 1));
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
  l.L = L, l.ws = static_cast<char*>(ws), l.st = st;
  l.lists = {group_offsets, l.at<int>(L.limit), l.at<int>(L.first), l.at<SeqInfo>(L.groups),
             l.at<long>(L.bases)};
  l.own.info = l.at<SeqInfo>(L.info), l.own.own = l.at<OwnPrefix>(L.own);
  l.own.starts = l.at<long>(L.starts), l.own.begins = l.at<int>(L.begins);
  l.sums.row_stats = l.at<float2>(L.row_stats), l.sums.row_sums = l.at<float4>(L.row_sums);
  l.sums.stats = l.at<float2>(L.prefix_stats), l.sums.sums = l.at<float4>(L.prefix_partial);
  l.sums.own = l.own.own, l.sums.head = l.at<PrefixHead>(L.head), l.sums.begins = l.own.begins;
  l.sums.gr = {groups, group_offsets, prefix_lens, max_group};
  l.sums.groups = l.lists.groups, l.sums.bases = l.lists.bases;
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
