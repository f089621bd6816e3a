// Host-side launch helpers of the attention kernels (rotary positions, the
// 4-bit paged cache, attention over it). See include/moe.h for the contracts.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "moe.h"

namespace moe {

// Rows of heads with strides in elements.
struct Rows {
  const void* p = nullptr;
  long token = 0, head = 0;
};

struct RopeArgs {
  int T = 0, D = 0, R = 0;
  int q_heads = 0, kv_heads = 0;  // either may be 0
  Rows q, k, v;
  const int32_t* positions = nullptr;
  const int64_t* slots = nullptr;
  const float* table = nullptr;
  int table_rows = 0;
  int interleaved = 0, inverse = 0;
  void* q_out = nullptr;
  uint8_t* cache = nullptr;
  long n_slots = 0;
  int page_shift = 0;  // log2 of the page size
  float k_inv = 1.0f, v_inv = 1.0f;  // 1 / k_scale, 1 / v_scale
  unsigned* status = nullptr;
};

// Rotation of q into q_out and, with kv_heads > 0, the append of k and v.
cudaError_t launch_rope(bool bf16, const RopeArgs& a, cudaStream_t st);

constexpr int kMaxPairs = 256;  // a block of the table kernel has as many threads
// Turns per position of each pair, as 64-bit fractions of a turn.
struct RopeTurns {
  unsigned long long f[kMaxPairs];
};
cudaError_t launch_rope_table(const RopeTurns& turns, int pairs, float gain, int n,
                              const int32_t* positions, float* table, cudaStream_t st);

cudaError_t launch_kv_read(bool bf16, int N, const int64_t* slots, const uint8_t* cache,
                           long n_slots, int kv_heads, int D, int page_shift, float k_scale,
                           float v_scale, void* k_out, void* v_out, unsigned* status,
                           cudaStream_t st);

struct AttnArgs {
  int B = 0, T = 0, max_q = 0;
  int heads = 0, kv_heads = 0, D = 0, page_size = 0;
  int window = 0;
  float scale_log2 = 0.0f;  // softmax_scale * k_scale * log2(e)
  float v_scale = 1.0f;
  Rows q;
  const int32_t* q_offsets = nullptr;
  const int32_t* seq_lens = nullptr;
  const int32_t* page_table = nullptr;
  int max_pages = 0;
  const uint8_t* cache = nullptr;
  long num_pages = 0;
  void* out = nullptr;
  float* lse = nullptr;
  int sms = 0;
};

// The workspace is laid out for this many SMs, so that its size does not
// depend on the device or context of the call that asks for it.
constexpr int kAttnMaxSms = 160;

struct AttnLayout {
  size_t status, counters, info, starts, row_tiles, firsts, stats, partial, total;
};
AttnLayout attn_layout(const moe_attn_config* c, int B, int T, int max_q);

// One request, checked: first query row, its tokens, cached tokens, the first
// key that one of its queries sees.
struct SeqInfo {
  int q0, q_len, len, first_key;
};

// What a kernel computes: a request's whole attention; a group's rows over the
// prefix that its requests share (all keys seen, sums left in fp32); or a
// request's own keys behind that prefix, to which those sums are added.
enum AttnPart { kWhole = 0, kPrefix = 1, kOwn = 2 };

// Groups of requests, as the caller gives them, and the shape of the list of the
// kernel over their prefixes.
struct Groups {
  int n = 0;
  const int32_t* offsets = nullptr;  // [n + 1] requests
  const int32_t* prefix = nullptr;   // [n] tokens
  int max_len = 0;                   // query tokens
};
struct PrefixShape {
  int tile_rows = 0, tile_keys = 0, ctas = 0;
  int setup = 0, least = 0, unit = 1;  // list entries of a segment's set-up, of the smallest
                                       // range of a CTA, of a key tile
  // Prompt kernel with two halves: a half's rows. In row tiles of no more rows both
  // halves take those rows, each every other tile of keys, and leave sums of their own;
  // a key tile has half_unit entries then.
  int half_rows = 0, half_unit = 1;
};
// Up to so many groups every CTA of the prefix kernel sums up the list itself, in
// shared memory, while the plan kernel still works on the own kernel's. (It goes
// through all requests for that; 64 groups, and 65 with the plan's list: 128 requests
// 20 and 28 us, 1024 53 and 64, 4096 110 and 140, 65536 1367 and 1368.)
constexpr int kSmallGroups = 64;

struct PrefixHead {
  long per;          // entries per CTA of the list over the prefixes
  long own_per;      // and of the own kernel's
  int own_piece, pad;  // tiles of a piece there, where segments are cut into whole pieces; 0: else
};

// Where a request's rows lie in the prefix kernel's list (len 0: no prefix).
struct OwnPrefix {
  long base;  // first list entry of its group
  int tok0;   // its first query token within the group's
  int len, half_len;  // list entries of a segment, and with no more than half_rows rows
  int rows;   // the group's rows
};

// The sums over shared prefixes. Segments that one CTA took leave each row in
// row_*, others leave pieces as the whole kernels do, which the own kernel joins.
// Sums lie in blocks of eight rows, [row / 8][D / 4][row % 8] of four channels, so
// that a warp with a row per lane writes whole lines, and the rows of one request
// can be read as whole sectors.
struct PrefixSums {
  float2* row_stats = nullptr;  // [T * heads]
  float4* row_sums = nullptr;   // [T * heads, rounded up to 8, D / 4]
  const float2* stats = nullptr;
  const float4* sums = nullptr;
  const OwnPrefix* own = nullptr;  // [B]
  const PrefixHead* head = nullptr;
  const int* begins = nullptr;  // request that each CTA of the own kernel begins in
  Groups gr;
  PrefixShape shape;
  const SeqInfo* groups = nullptr;  // of more than kSmallGroups: what the plan summed up
  const long* bases = nullptr;
  int lo = 0, hi = 0;              // a segment's CTAs: (begin + lo) / per .. (end - hi) / per
};
template <int kPart>
struct PartArgs {
  PrefixSums p;
};
template <>
struct PartArgs<kWhole> {};

// Rows of a row tile of the prompt kernel (query tokens times heads of a
// group), and the rows per request it is used from (uses_prompt_kernel has the
// times of both sides).
constexpr int prompt_tile(int head_dim) { return head_dim == 256 ? 128 : 256; }
constexpr int kPromptRows = 64;
cudaError_t launch_prompt(const AttnArgs& a, void* ws, const AttnLayout& L, cudaStream_t st);

// Whether a call can share prefixes at all, and whether it pays for requests whose
// rows of the page table have so many entries.
bool can_share(const moe_attn_config* c, int max_q, int groups);
bool worth_sharing(const moe_attn_config* c, int B, int max_q, int max_pages);
struct SharedLayout {
  size_t status, head, counters, begins, info, own, starts, limit, first, groups, bases, stats,
      partial, prefix_stats, prefix_partial, row_stats, row_sums, total;
};
SharedLayout shared_layout(const moe_attn_config* c, int B, int T, int groups, int max_group);
cudaError_t launch_kv_attention_shared(const moe_attn_config* c, const AttnArgs& a, int groups,
                                       const int32_t* group_offsets, const int32_t* prefix_lens,
                                       int max_group, void* ws, const SharedLayout& L,
                                       cudaStream_t st);

cudaError_t launch_kv_attention(const moe_attn_config* c, const AttnArgs& a, void* ws,
                                const AttnLayout& L, cudaStream_t st);

}  // namespace moe
