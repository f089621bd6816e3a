// Norms around a block: the block's output is normed, gated and scaled, joins
// the residual, and the sum is normed for the next block.
//
//   u = N(y; post)      r = x + scale * gate * u      h = N(r; pre)
//
// One pass: a row lives in the registers of the threads that loaded it, as fp32,
// from its loads to its stores, so that memory bounds the kernel. Means and
// variances are taken in two steps over the registers (the squares of what is
// left after the mean), where sums of squares less the mean's would cancel. h
// comes from r before r is rounded for x_out.
//
// A row belongs to a block of as many warps as give each thread kElems elements,
// rows of one warp share a block of four. A chunk is 16 bytes of the wider type:
// neighbouring lanes hold neighbouring chunks.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "launch.cuh"
#include "serve.h"

namespace moe {
namespace {

constexpr int kRowsPerBlock = 4;  // rows of one warp each

template <int V>
__device__ __forceinline__ void load_chunk(const float* p, float* x) {
  if constexpr (V == 1) {
    x[0] = *p;
  } else {
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
      const float4 v = reinterpret_cast<const float4*>(p)[i];
      x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
    }
  }
}
template <int V>
__device__ __forceinline__ void load_chunk(const __nv_bfloat16* p, float* x) {
  if constexpr (V == 1) {
    x[0] = __bfloat162float(*p);
  } else {
    uint32_t w[V / 2];
    if constexpr (V == 8) {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x, w[1] = v.y;
    }
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}
template <int V>
__device__ __forceinline__ void store_chunk(float* p, const float* x) {
  if constexpr (V == 1) {
    *p = x[0];
  } else {
#pragma unroll
    for (int i = 0; i < V / 4; ++i)
      reinterpret_cast<float4*>(p)[i] =
          make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
  }
}
template <int V>
__device__ __forceinline__ void store_chunk(__nv_bfloat16* p, const float* x) {
  if constexpr (V == 1) {
    *p = __float2bfloat16_rn(x[0]);
  } else {
    uint32_t w[V / 2];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    if constexpr (V == 8)
      *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  }
}

// The sum over the threads of a row, the same bits in each of them. `slot` is
// a place in shared memory that no other sum of this row uses.
template <bool kWarpRow>
__device__ __forceinline__ float row_sum(float v, float* slot) {
#pragma unroll
  for (int d = 16; d > 0; d /= 2) v += __shfl_xor_sync(~0u, v, d);
  if constexpr (!kWarpRow) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0) slot[warp] = v;
    __syncthreads();
    v = lane < warps ? slot[lane] : 0.0f;
#pragma unroll
    for (int d = 16; d > 0; d /= 2) v += __shfl_xor_sync(~0u, v, d);
  }
  return v;
}

// TA: block output and h, TR: residual, V: elements of a chunk (1: any alignment).
template <typename TA, typename TR, int V, int kElems, bool kWarpRow>
__global__ void __launch_bounds__(kWarpRow ? 32 * kRowsPerBlock : 1024)
    norm_kernel(NormArgs a) {
  constexpr int kChunks = kElems / V;
  __shared__ float s_sum[4][32];
  const int lane = kWarpRow ? threadIdx.x & 31 : threadIdx.x;
  const int lanes = kWarpRow ? 32 : blockDim.x;
  const long t = kWarpRow ? static_cast<long>(blockIdx.x) * kRowsPerBlock + (threadIdx.x >> 5)
                          : blockIdx.x;
  pdl_enter();
  if (kWarpRow && t >= a.T) return;
  const TA* y = static_cast<const TA*>(a.y);
  const TR* x = static_cast<const TR*>(a.x);
  const TA* gate = static_cast<const TA*>(a.gate);
  auto at = [&](int c) { return (c * lanes + lane) * V; };

  float r[kChunks][V], u[kChunks][V];
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
#pragma unroll
    for (int i = 0; i < V; ++i) r[c][i] = u[c][i] = 0.0f;
    if (at(c) < a.H) {
      load_chunk<V>(x + t * a.x_stride + at(c), r[c]);
      if (y) load_chunk<V>(y + t * a.y_stride + at(c), u[c]);
    }
  }
  const float inv = 1.0f / static_cast<float>(a.H);
  // The row v normed in place; `used` is the number of sums taken before.
  auto norm = [&](float(&v)[kChunks][V], const float* w, const float* b, int used) {
    float mean = 0.0f;
    if (a.layer) {
      float sum = 0.0f;
#pragma unroll
      for (int c = 0; c < kChunks; ++c)
#pragma unroll
        for (int i = 0; i < V; ++i) sum += v[c][i];
      mean = row_sum<kWarpRow>(sum, s_sum[used]) * inv;
    }
    float sum = 0.0f;
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
      if (at(c) < a.H) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          v[c][i] -= mean;
          sum += v[c][i] * v[c][i];
        }
      }
    const float f = 1.0f / sqrtf(row_sum<kWarpRow>(sum, s_sum[used + 1]) * inv + a.eps);
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
      if (at(c) < a.H) {
        float wv[V], bv[V];
        if (w) load_chunk<V>(w + at(c), wv);
        if (b) load_chunk<V>(b + at(c), bv);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          v[c][i] *= f;
          if (w) v[c][i] *= wv[i] + a.offset;
          if (b) v[c][i] += bv[i];
        }
      }
  };
  if (y) {
    if (a.post) norm(u, a.post_w, a.post_b, 0);
    float one = a.scale;  // of a gate with one value per token
    if (gate && a.gate_channel == 0) {
      float g;
      load_chunk<1>(gate + t * a.gate_token, &g);
      one *= a.sigmoid ? 1.0f / (1.0f + expf(-g)) : g;
    }
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
      if (at(c) < a.H) {
        float g[V];
        const bool own = gate && a.gate_channel;
        if (own) load_chunk<V>(gate + t * a.gate_token + at(c), g);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          float f = one;
          if (own) f *= a.sigmoid ? 1.0f / (1.0f + expf(-g[i])) : g[i];
          r[c][i] += f * u[c][i];
        }
        if (a.x_out) store_chunk<V>(static_cast<TR*>(a.x_out) + t * a.H + at(c), r[c]);
      }
  }
  if (!a.h) return;
  norm(r, a.pre_w, a.pre_b, 2);
#pragma unroll
  for (int c = 0; c < kChunks; ++c)
    if (at(c) < a.H) store_chunk<V>(static_cast<TA*>(a.h) + t * a.H + at(c), r[c]);
}

template <typename TA, typename TR, int V, int kElems>
cudaError_t launch_as(const NormArgs& a, cudaStream_t st) {
  const int threads = (a.H + kElems * 32 - 1) / (kElems * 32) * 32;
  if (threads == 32)
    return launch_pdl(&norm_kernel<TA, TR, V, kElems, true>,
                      dim3((a.T + kRowsPerBlock - 1) / kRowsPerBlock), dim3(32 * kRowsPerBlock), 0,
                      st, a);
  return launch_pdl(&norm_kernel<TA, TR, V, kElems, false>, dim3(a.T), dim3(threads), 0, st, a);
}

template <typename TA, typename TR>
cudaError_t launch_types(const NormArgs& a, int sms, cudaStream_t st) {
  constexpr int V = 16 / (sizeof(TA) > sizeof(TR) ? sizeof(TA) : sizeof(TR));
  auto ok = [](const void* p, size_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; };
  const bool chunks = a.H % V == 0 && ok(a.x, V * sizeof(TR)) && a.x_stride % V == 0 &&
                      ok(a.y, V * sizeof(TA)) && a.y_stride % V == 0 &&
                      (!a.gate_channel || (ok(a.gate, V * sizeof(TA)) && a.gate_token % V == 0));
  if (chunks) return launch_as<TA, TR, V, 16>(a, st);
  return launch_as<TA, TR, 1, 16>(a, st);
}

}  // namespace

cudaError_t launch_norm(bool act_bf16, bool res_bf16, const NormArgs& a, int sms, cudaStream_t st) {
  if (act_bf16)
    return res_bf16 ? launch_types<__nv_bfloat16, __nv_bfloat16>(a, sms, st)
                    : launch_types<__nv_bfloat16, float>(a, sms, st);
  return res_bf16 ? launch_types<float, __nv_bfloat16>(a, sms, st)
                  : launch_types<float, float>(a, sms, st);
}

}  // namespace moe
