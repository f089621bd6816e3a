// Device helpers shared by the attention kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "attn.h"
#include "kv4.cuh"

namespace moe {

// P = exp2(score - maximum) is kept as f16 times 2^kLift, so that small
// probabilities keep their bits, and the running maximum may lag behind by
// kLag powers of two before sums are rescaled: P stays below 2^15. One f16 per
// weight rounds it by 2^-11 at most, an eighth of what an output's rounding to
// bf16 may be, and takes half the matrix instructions of two; the weights' sum
// takes P in fp32. Against 64 bits the outputs' error stays that of bf16 (0.0017 of
// their size, as with P in fp32). fp32 outputs need both terms.
constexpr float kLift = 6.0f, kLag = 8.0f;

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_f16(uint32_t v) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// What request b asks for, checked; flags collects MOE_DEV_* bits.
__device__ __forceinline__ SeqInfo seq_info(const AttnArgs& a, int b, unsigned& flags) {
  SeqInfo s = {0, 0, 0, 0};
  const int q0 = a.q_offsets ? a.q_offsets[b] : b;
  const int q1 = a.q_offsets ? a.q_offsets[b + 1] : b + 1;
  const int n = a.seq_lens[b];
  if (q0 < 0 || q1 < q0 || q1 > a.T || q1 - q0 > a.max_q) {
    flags |= MOE_DEV_BAD_SEGMENT;
  } else {
    s.q0 = q0;
    s.q_len = q1 - q0;
  }
  const long cap = static_cast<long>(a.max_pages) * a.page_size;
  s.len = static_cast<int>(n < 0 ? 0 : n > cap ? cap : n);
  if (s.len != n) flags |= MOE_DEV_BAD_PAGE;
  if (a.window > 0) {
    const long lo = static_cast<long>(s.len) - s.q_len - a.window + 1;
    s.first_key = lo > 0 ? static_cast<int>(lo) : 0;
  }
  return s;
}

// Sum of the values of the threads before this one in a block of N threads,
// plus `base`, to which the block's sum is added.
template <int N>
__device__ __forceinline__ long block_scan(long v, long* warp_sum, long& base) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long sum = v;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const long u = __shfl_up_sync(~0u, sum, d);
    if (lane >= d) sum += u;
  }
  if (lane == 31) warp_sum[warp] = sum;
  __syncthreads();
  long before = base;
#pragma unroll
  for (int w = 0; w < N / 32; ++w) {
    if (w < warp) before += warp_sum[w];
    base += warp_sum[w];
  }
  __syncthreads();
  return before + sum - v;
}

template <int N>
struct Words {
  uint32_t w[N];
};
template <int N>
__device__ __forceinline__ Words<N> load_words(const uint8_t* p) {
  Words<N> r;
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 v = reinterpret_cast<const uint4*>(p)[i];
      r.w[4 * i] = v.x, r.w[4 * i + 1] = v.y, r.w[4 * i + 2] = v.z, r.w[4 * i + 3] = v.w;
    }
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    r.w[0] = v.x, r.w[1] = v.y;
  } else {
    r.w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
  return r;
}

// A power of two (and its inverse) that brings a query row whose largest
// element is `top` into [128, 256): every bit of a bf16 element then survives
// in f16 unless the element is 2^-22 of the largest.
__device__ __forceinline__ void row_power(float top, float& up, float& down) {
  int e = static_cast<int>((__float_as_uint(top) >> 23) & 0xffu) - 127;
  e = max(-90, min(127, e));
  up = __uint_as_float(static_cast<uint32_t>(7 - e + 127) << 23);
  down = __uint_as_float(static_cast<uint32_t>(e - 7 + 127) << 23);
}

// What a row's scores are multiplied by: never 0, since a masked score is -inf
// and has to stay it. (Scores are below 2^28 before it: under the smallest
// normal number all of them are 0.)
__device__ __forceinline__ float score_gain(float down, float scale_log2) {
  return fmaxf(down * scale_log2, 0x1p-126f);
}

// 1 / denominator times `gain`; 0 for a query that saw no key (NaN stays NaN).
__device__ __forceinline__ float out_factor(float den, float gain) {
  return den > 0.0f || den != den ? gain / den : 0.0f;
}
__device__ __forceinline__ float log_sum(float base, float den) {
  return den > 0.0f || den != den ? (base + log2f(den)) * 0.69314718f : -INFINITY;
}

__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
  const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                                            *reinterpret_cast<const uint32_t*>(&hi));
}
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }

}  // namespace moe
