// Attention over the 4-bit paged cache: launches of the split kernel, and which
// kernel a call takes.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>

#include "attn_split.cuh"
#include "launch.cuh"

namespace moe {
namespace {

using namespace split;

template <typename T, int D, int kRows, int kTerms, bool kInline>
cudaError_t launch_split_as(const AttnArgs& a, void* ws, const AttnLayout& L, cudaStream_t st) {
  auto* kern = &attn_split_kernel<T, D, kRows, kTerms, kInline>;
  const int grid = a.sms * ctas_per_sm<D, kRows, kTerms>();
  char* w = static_cast<char*>(ws);
  auto* status = reinterpret_cast<unsigned*>(w + L.status);
  auto* counters = reinterpret_cast<int*>(w + L.counters);
  auto* info = reinterpret_cast<SeqInfo*>(w + L.info);
  auto* starts = reinterpret_cast<long*>(w + L.starts);
  cudaError_t e = launch_pdl(&attn_plan_kernel, dim3(1), dim3(kPlanThreads), 0, st, a, kRows, status,
                             counters, grid, kInline ? nullptr : info, starts);
  if (e != cudaSuccess) return e;
  constexpr int smem = split_smem<D, kRows>();
  static std::atomic<unsigned long long> done{0};
  e = opt_in_smem(reinterpret_cast<const void*>(kern), smem, done);
  if (e != cudaSuccess) return e;
  int log2 = 0;
  while ((1 << log2) < a.page_size) ++log2;
  return launch_pdl(kern, dim3(grid), dim3(kThreads), smem, st, a, status, counters,
                    const_cast<const SeqInfo*>(info), const_cast<const long*>(starts),
                    reinterpret_cast<float*>(w + L.stats), reinterpret_cast<float*>(w + L.partial),
                    log2, PartArgs<kWhole>());
}
template <typename T, int D, int kRows, int kTerms>
cudaError_t launch_split(const AttnArgs& a, void* ws, const AttnLayout& L, cudaStream_t st) {
  return a.B <= kInlineSeqs ? launch_split_as<T, D, kRows, kTerms, true>(a, ws, L, st)
                            : launch_split_as<T, D, kRows, kTerms, false>(a, ws, L, st);
}

template <int D>
cudaError_t launch_dim(bool bf16, const AttnArgs& a, void* ws, const AttnLayout& L,
                       cudaStream_t st) {
  const long rows = static_cast<long>(a.max_q) * (a.heads / a.kv_heads);
  if (!bf16)
    return rows <= 4 ? launch_split<float, D, 4, 2>(a, ws, L, st)
                     : launch_split<float, D, 8, 2>(a, ws, L, st);
  return rows <= 4   ? launch_split<__nv_bfloat16, D, 4, 1>(a, ws, L, st)
         : rows <= 8 ? launch_split<__nv_bfloat16, D, 8, 1>(a, ws, L, st)
                     : launch_split<__nv_bfloat16, D, 16, 1>(a, ws, L, st);
}

}  // namespace

// From kPromptRows rows per request the matrix work, not the cache's
// bandwidth, is the bound: the prompt kernel (bf16). Split and prompt kernel,
// 16 requests of 8192 tokens: 32 rows 91 and 126 us, 48 rows 133 and 127, 64 rows
// 163 and 127. 512 tokens: 22 and 31, 26 and 31, 28 and 31. One of 65536: 60 and
// 94, 80 and 94, 102 and 95.
bool uses_prompt_kernel(const moe_attn_config* c, int max_q) {
  return c->act_dtype == MOE_BF16 &&
         static_cast<long>(max_q) * (c->num_heads / c->num_kv_heads) >= kPromptRows;
}

AttnLayout attn_layout(const moe_attn_config* c, int B, int T, int max_q) {
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  const bool prompt = uses_prompt_kernel(c, max_q);
  const size_t ctas = static_cast<size_t>(kAttnMaxSms) * (prompt ? 1 : kMaxCtasPerSm);
  // each request's last row tile may be partly filled
  const size_t group = c->num_heads / c->num_kv_heads;
  const size_t row_tiles =
      prompt ? static_cast<size_t>(T) * group / prompt_tile(c->head_dim) + B : 0;
  const size_t lists = prompt ? row_tiles : static_cast<size_t>(B);
  // two pieces per CTA, of up to 16 rows or of a whole row tile
  const size_t piece_rows = 2 * ctas * (prompt ? prompt_tile(c->head_dim) : 16);
  AttnLayout L;
  L.status = 0;
  L.counters = 256;
  L.info = up(L.counters + 2 * 4 * ctas);
  L.starts = up(L.info + sizeof(SeqInfo) * static_cast<size_t>(B));
  L.row_tiles = up(L.starts + 8 * (lists + 1));
  L.firsts = up(L.row_tiles + (prompt ? 8 * row_tiles : 0));
  L.stats = up(L.firsts + (prompt ? 4 * (static_cast<size_t>(B) + 1) : 0));
  L.partial = up(L.stats + piece_rows * 8);
  L.total = up(L.partial + piece_rows * static_cast<size_t>(c->head_dim) * 4);
  return L;
}

cudaError_t launch_kv_attention(const moe_attn_config* c, const AttnArgs& a, void* ws,
                                const AttnLayout& L, cudaStream_t st) {
  if (uses_prompt_kernel(c, a.max_q)) return launch_prompt(a, ws, L, st);
  const bool bf16 = c->act_dtype == MOE_BF16;
  switch (a.D) {
    case 64:
      return launch_dim<64>(bf16, a, ws, L, st);
    case 128:
      return launch_dim<128>(bf16, a, ws, L, st);
    default:
      return launch_dim<256>(bf16, a, ws, L, st);
  }
}

}  // namespace moe
