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

// Rows of a row tile of the prompt kernel (query tokens times heads of a
// group), and the rows per request it is used from (uses_prompt_kernel has the
// times of both sides).
constexpr int prompt_tile(int head_dim) { return head_dim == 256 ? 128 : 256; }
constexpr int kPromptRows = 64;
cudaError_t launch_prompt(const AttnArgs& a, void* ws, const AttnLayout& L, cudaStream_t st);

cudaError_t launch_kv_attention(const moe_attn_config* c, const AttnArgs& a, void* ws,
                                const AttnLayout& L, cudaStream_t st);

}  // namespace moe
