// Attention over the 4-bit paged cache: launches of the prompt kernel.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>

#include "attn_prompt.cuh"
#include "internal.h"
#include "launch.cuh"

namespace moe {

MOE_WAIT_LIMIT_SETTER(set_wait_limit_attn)

namespace {

using namespace prompt;

template <int D>
cudaError_t launch_dim(const AttnArgs& a, void* ws, const AttnLayout& L, cudaStream_t st) {
  char* w = static_cast<char*>(ws);
  auto* status = reinterpret_cast<unsigned*>(w + L.status);
  auto* counters = reinterpret_cast<int*>(w + L.counters);
  auto* info = reinterpret_cast<SeqInfo*>(w + L.info);
  auto* firsts = reinterpret_cast<int*>(w + L.firsts);
  auto* row_tiles = reinterpret_cast<RowTile*>(w + L.row_tiles);
  auto* starts = reinterpret_cast<long*>(w + L.starts);
  const long group = a.heads / a.kv_heads;
  const int max_row_tiles = static_cast<int>(a.T * group / Shape<D>::kTile + a.B);
  cudaError_t e =
      launch_pdl(&prompt_plan_kernel<D>, dim3(1), dim3(kPlanThreads), 0, st, a, max_row_tiles,
                 status, counters, 2 * a.sms, info, firsts, row_tiles, starts);
  if (e != cudaSuccess) return e;
  static std::atomic<unsigned long long> done{0};
  e = opt_in_smem(reinterpret_cast<const void*>(&attn_prompt_kernel<D>), Shape<D>::kBytes, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(&attn_prompt_kernel<D>, dim3(a.sms), dim3(kThreads), Shape<D>::kBytes, st, a,
                    status, counters, const_cast<const SeqInfo*>(info),
                    const_cast<const int*>(firsts), const_cast<const RowTile*>(row_tiles),
                    const_cast<const long*>(starts), reinterpret_cast<float2*>(w + L.stats),
                    reinterpret_cast<float4*>(w + L.partial), PartArgs<kWhole>());
}

}  // namespace

cudaError_t launch_prompt(const AttnArgs& a, void* ws, const AttnLayout& L, cudaStream_t st) {
  return a.D == 64    ? launch_dim<64>(a, ws, L, st)
         : a.D == 128 ? launch_dim<128>(a, ws, L, st)
                      : launch_dim<256>(a, ws, L, st);
}

}  // namespace moe
