// Norms around a block: the block's output is normed, gated and scaled, joins
// the residual, and the sum is normed for the next block.
//
//   u = N(y; post)      r = x + scale * gate * u      h = N(r; pre)
//
// One pass: a row lives in the registers of a block's threads, as fp32, from its
// loads to its stores, so that memory bounds the kernels. Means and variances are
// taken in two steps over the registers (the squares of what is left after the
// mean), where sums of squares less the mean's would cancel. h comes from r before
// r is rounded for x_out. A row belongs to as many warps as give each thread 16
// elements; rows of one warp need no barriers.
//
// Two kernels. Rows of whole 16-byte chunks go straight into registers
// (norm_whole_kernel). Others, and rows of more than kMostKeep threads, are copied
// to shared memory in 16-byte pieces from the last boundary before them, whatever
// their alignment, and taken from there in groups of four (norm_any_kernel).
//
// Measured: 8192 rows of 4096, bf16 with an fp32 residual, normed on both sides and
// gated by channel, 62.8 us: 6.4 TB/s, 94 % of a copy's rate (94 us with the weights
// read again for every row); 4097 rows of 5120 in fp32 55 us, 6.0 TB/s; 64 rows of
// 2048 2.2 us, a chain of two loads and the sum. Rows of 1001: 34 us, 3.9 TB/s, where
// instructions are the bound (elements taken one by one, each load and store of its
// own: 58 us). Rows of one warp, bf16 and fp32, a norm alone: 262144 of 128 channels
// 54 and 55 us (2.5 and 4.9 TB/s: 16 of 32 lanes have a chunk in bf16), 131072 of 512
// 51 and 91 us (5.3 and 5.9 TB/s; in fp32 244 bytes spill for five blocks an SM). 8192
// rows of 6144 that join a residual 71 and 122 us (5.7 and 6.6 TB/s).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>

#include "launch.cuh"
#include "ptx.cuh"
#include "serve.h"

namespace moe {
namespace {

constexpr int kMostThreads = 1024;
constexpr int kRowsPerBlock = 4;     // rows of one warp each
constexpr int kMostKeep = 512;       // threads of a row whose weights are kept
constexpr int kMostStages = 4;
// Bytes on the way per SM that keep memory busy, and shared memory for them, which
// leaves the L1 cache room for weights (rows of 3001, normed twice and gated: 76 us,
// and 86 with 128 of 200 KB, 96 with 48 of 80; rows of 12288 46, 50 and 45).
constexpr int kAhead = 96 * 1024, kSmemPerSm = 128 * 1024, kSmemMost = 226 * 1024;

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}

// Four values at p, or one by one where a group may lie anywhere.
__device__ __forceinline__ void get(const float* p, float (&v)[4]) {
  const float4 f = *reinterpret_cast<const float4*>(p);
  v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
}
__device__ __forceinline__ void get(const __nv_bfloat16* p, float (&v)[4]) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  v[0] = __uint_as_float(w.x << 16), v[1] = __uint_as_float(w.x & 0xffff0000u);
  v[2] = __uint_as_float(w.y << 16), v[3] = __uint_as_float(w.y & 0xffff0000u);
}
__device__ __forceinline__ float one(const float* p) { return *p; }
__device__ __forceinline__ float one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void put(float* p, const float (&v)[4]) {
  __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
}
__device__ __forceinline__ void put(__nv_bfloat16* p, const float (&v)[4]) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
  __stcs(reinterpret_cast<uint2*>(p), make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                                 *reinterpret_cast<const uint32_t*>(&b)));
}
__device__ __forceinline__ void put_one(float* p, float v) { *p = v; }
__device__ __forceinline__ void put_one(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

// The sum over the threads of a row, the same bits in each of them. Sums that
// follow one another take turns at two slots of shared memory: every thread
// has read a slot before the sum after the next one, behind a barrier, writes it.
template <bool kWarpRow>
__device__ __forceinline__ float row_sum(float v, float (*slots)[32], int& turn) {
#pragma unroll
  for (int d = 16; d > 0; d /= 2) v += __shfl_xor_sync(~0u, v, d);
  if constexpr (!kWarpRow) {
    float* slot = slots[turn];
    turn ^= 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0) slot[warp] = v;
    __syncthreads();
    v = lane < warps ? slot[lane] : 0.0f;
#pragma unroll
    for (int d = 16; d > 0; d /= 2) v += __shfl_xor_sync(~0u, v, d);
  }
  return v;
}

// Bytes that a row of n elements takes in shared memory.
__host__ __device__ constexpr int row_bytes(int n, int size) { return (n * size + 15 + 15) / 16 * 16; }

// TA: block output, gate and h, TR: residual. kWhole: all rows begin at groups of
// four and have whole ones. kAlike: they begin at the same place of a group in
// every tensor; else elements are taken one by one. kGroups: groups per thread.
// Blocks stay and take one row after the other; a row's place in shared memory goes
// to a later row as soon as it is in registers.
template <typename TA, typename TR, int kGroups, bool kWarpRow, bool kWhole, bool kAlike>
__global__ void __launch_bounds__(kWarpRow ? 32 * kRowsPerBlock : kMostThreads, kWarpRow ? 8 : 1)
    norm_any_kernel(NormArgs a, int stages, int stage_bytes) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float s_sum[2][32];
  int turn = 0;
  const int warp = threadIdx.x >> 5, lane = kWarpRow ? threadIdx.x & 31 : threadIdx.x;
  const int lanes = kWarpRow ? 32 : blockDim.x;
  const long step = kWarpRow ? static_cast<long>(gridDim.x) * kRowsPerBlock : gridDim.x;
  const long t0 = kWarpRow ? static_cast<long>(blockIdx.x) * kRowsPerBlock + warp : blockIdx.x;
  uint8_t* ring = smem + (kWarpRow ? warp * stages * stage_bytes : 0);
  const TA* y = static_cast<const TA*>(a.y);
  const TR* x = static_cast<const TR*>(a.x);
  const TA* gate = static_cast<const TA*>(a.gate);
  // gates: one per channel for all rows, one per element, or one per row
  const bool fixed = gate && a.gate_channel && a.gate_token == 0;
  const bool full = gate && a.gate_channel && a.gate_token != 0;
  const int H = a.H;
  const float inv = 1.0f / static_cast<float>(H);
  const int y_at = row_bytes(H, sizeof(TR)), g_at = y_at + (y ? row_bytes(H, sizeof(TA)) : 0);
  pdl_enter();

  auto copy_row = [&](uint8_t* dst, const auto* row) {
    const uint8_t* p = reinterpret_cast<const uint8_t*>(row);
    const int off = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15u);
    const int bytes = off + H * static_cast<int>(sizeof(*row));
    const uint32_t to = ptx::smem_u32(dst);
    for (int i = lane * 16; i < bytes; i += lanes * 16) copy16(to + i, p - off + i, min(16, bytes - i));
  };
  auto copy = [&](long t, int stage) {
    if (t < a.T) {
      uint8_t* dst = ring + stage * stage_bytes;
      copy_row(dst, x + t * a.x_stride);
      if (y) copy_row(dst + y_at, y + t * a.y_stride);
      if (full) copy_row(dst + g_at, gate + t * a.gate_token);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // What was copied of a row, from its first element.
  auto staged = [&](uint8_t* src, const auto* row) {
    return reinterpret_cast<decltype(row)>(src + (reinterpret_cast<uintptr_t>(row) & 15u));
  };
  for (int i = 0; i < stages; ++i) copy(t0 + i * step, i);

  auto inside = [&](int e) { return static_cast<unsigned>(e) < static_cast<unsigned>(H); };
  // Four elements from e of a vector of H channels, whose first one is aligned.
  auto channels = [&](const auto* vec, int e, float(&v)[4]) {
    if (kWhole) {
      get(vec + e, v);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = inside(e + i) ? one(vec + e + i) : 0.0f;
    }
  };
  // A group's weights, and the factors that its part of the block's output has in
  // all rows (the scale, and gates by channel).
  auto weights = [&](const float* w, int e, float(&v)[4]) {
    v[0] = v[1] = v[2] = v[3] = 1.0f;
    if (!w || e >= H) return;
    channels(w, e, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += a.offset;
  };
  auto factors = [&](int e, float(&v)[4]) {
    v[0] = v[1] = v[2] = v[3] = a.scale;
    if (!fixed || e >= H) return;
    channels(gate, e, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = a.scale * (a.sigmoid ? sigmoid(v[i]) : v[i]);
  };

  int stage = 0;
  for (long t = t0; t < a.T; t += step, stage = stage + 1 == stages ? 0 : stage + 1) {
    if (stages == 1) asm volatile("cp.async.wait_group 0;" ::: "memory");
    else if (stages == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else if (stages == 3) asm volatile("cp.async.wait_group 2;" ::: "memory");
    else asm volatile("cp.async.wait_group 3;" ::: "memory");
    if (kWarpRow) __syncwarp();
    else __syncthreads();
    // The row is in registers: its place goes to a later one.
    auto release = [&] {
      if (kWarpRow) __syncwarp();
      else __syncthreads();
      copy(t + stages * step, stage);
    };
    uint8_t* here = ring + stage * stage_bytes;
    const TR* xs = staged(here, x + t * a.x_stride);
    const TA* ys = staged(here + y_at, y + t * a.y_stride);
    const TA* gs = staged(here + g_at, gate + t * a.gate_token);
    // groups lie at multiples of four of the outputs' rows, which are contiguous
    const int shift = kWhole ? 0 : static_cast<int>(t * H & 3);
    auto first = [&](int c) { return (c * lanes + lane) * 4 - shift; };
    // Four elements from e of a row; what is outside the row reads as zero.
    auto take = [&](const auto* row, int e, float(&v)[4]) {
      if (kWhole || (kAlike && e >= 0 && e + 4 <= H)) {
        get(row + e, v);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = inside(e + i) ? one(row + e + i) : 0.0f;
      }
    };
    auto give = [&](auto* row, int e, const float(&v)[4]) {
      if (kWhole || (e >= 0 && e + 4 <= H)) {
        put(row + e, v);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (inside(e + i)) put_one(row + e + i, v[i]);
      }
    };
    // The row v normed in place.
    auto norm = [&](float(&v)[kGroups][4], const float* w, const float* b) {
      float mean = 0.0f;
      if (a.layer) {
        float sum = 0.0f;
#pragma unroll
        for (int c = 0; c < kGroups; ++c) sum += (v[c][0] + v[c][1]) + (v[c][2] + v[c][3]);
        mean = row_sum<kWarpRow>(sum, s_sum, turn) * inv;
#pragma unroll
        for (int c = 0; c < kGroups; ++c)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            v[c][i] = inside(kWhole ? first(c) : first(c) + i) ? v[c][i] - mean : 0.0f;
      }
      float sums[2] = {0.0f, 0.0f};
#pragma unroll
      for (int c = 0; c < kGroups; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) sums[i & 1] += v[c][i] * v[c][i];
      const float f =
          1.0f / sqrtf(row_sum<kWarpRow>(sums[0] + sums[1], s_sum, turn) * inv + a.eps);
#pragma unroll
      for (int c = 0; c < kGroups; ++c) {
        float k[4];
        weights(w, first(c), k);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[c][i] = v[c][i] * f * k[i];
        if (b && first(c) < H) {
          channels(b, first(c), k);
#pragma unroll
          for (int i = 0; i < 4; ++i) v[c][i] += k[i];
        }
      }
    };

    float r[kGroups][4], u[kGroups][4];
    auto gates = [&] {  // by element
#pragma unroll
      for (int c = 0; c < kGroups; ++c) {
        if (first(c) >= H) continue;
        float g[4];
        take(gs, first(c), g);
#pragma unroll
        for (int i = 0; i < 4; ++i) u[c][i] *= a.sigmoid ? sigmoid(g[i]) : g[i];
      }
    };
#pragma unroll
    for (int c = 0; c < kGroups; ++c) {
      r[c][0] = r[c][1] = r[c][2] = r[c][3] = 0.0f;
      u[c][0] = u[c][1] = u[c][2] = u[c][3] = 0.0f;
      if (first(c) >= H) continue;
      take(xs, first(c), r[c]);
      if (y) take(ys, first(c), u[c]);
    }
    if (full && !a.post) gates();
    if (!(full && a.post)) release();
    if (y) {
      if (a.post) {
        norm(u, a.post_w, a.post_b);
        if (full) {
          gates();
          release();
        }
      }
      if (gate && !fixed && !full) {
        const float g = one(gate + t * a.gate_token), every = a.sigmoid ? sigmoid(g) : g;
#pragma unroll
        for (int c = 0; c < kGroups; ++c)
#pragma unroll
          for (int i = 0; i < 4; ++i) u[c][i] *= every;
      }
#pragma unroll
      for (int c = 0; c < kGroups; ++c) {
        float k[4];
        factors(first(c), k);
        // (what is outside the row stays 0: u there has been 0 all along)
#pragma unroll
        for (int i = 0; i < 4; ++i) r[c][i] += k[i] * u[c][i];
        if (a.x_out && first(c) < H) give(static_cast<TR*>(a.x_out) + t * H, first(c), r[c]);
      }
    }
    if (a.h) {
      norm(r, a.pre_w, a.pre_b);
#pragma unroll
      for (int c = 0; c < kGroups; ++c)
        if (first(c) < H) give(static_cast<TA*>(a.h) + t * H, first(c), r[c]);
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// Rows that begin at chunks (16 bytes of the wider type) and have whole ones: straight
// from memory into registers, the next row's chunks under way while a row is summed up.
// A thread has the same channels of every row and keeps their weights and, where all
// rows share them, their gates. kChunks: chunks per thread.
template <typename T, int V>
struct Raw {
  uint32_t w[V * static_cast<int>(sizeof(T)) / 4];
};
template <typename T, int V>
__device__ __forceinline__ void fetch(Raw<T, V>& r, const T* p) {
  if constexpr (sizeof(r) == 8)
    asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];"
                 : "=r"(r.w[0]), "=r"(r.w[1])
                 : "l"(p)
                 : "memory");
  else
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3])
                 : "l"(p)
                 : "memory");
}
template <int V>
__device__ __forceinline__ void unpack(const Raw<float, V>& r, float (&x)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) x[i] = __uint_as_float(r.w[i]);
}
template <int V>
__device__ __forceinline__ void unpack(const Raw<__nv_bfloat16, V>& r, float (&x)[V]) {
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    x[2 * i] = __uint_as_float(r.w[i] << 16);
    x[2 * i + 1] = __uint_as_float(r.w[i] & 0xffff0000u);
  }
}
template <int V>
__device__ __forceinline__ void put_chunk(float* p, const float (&v)[V]) {
  __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
}
template <int V>
__device__ __forceinline__ void put_chunk(__nv_bfloat16* p, const float (&v)[V]) {
  uint32_t w[V / 2];
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  if constexpr (V == 8)
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
  else
    __stcs(reinterpret_cast<uint2*>(p), make_uint2(w[0], w[1]));
}
template <typename TA, typename TR>
__host__ __device__ constexpr int chunk_of() {
  return 16 / static_cast<int>(sizeof(TA) > sizeof(TR) ? sizeof(TA) : sizeof(TR));
}

//
// kTwo: two blocks an SM of up to kTwoThreads threads, where there are rows for more
// than that, for bf16 activations normed once: one row under way is too few bytes then
// (8192 rows of 5120 with a bf16 residual 51.4 us instead of 63.4, gated by element 62.8
// instead of 74.5, of 2880 34.0 instead of 37.5, with an fp32 residual 81 instead of 85;
// of 4096 45.8 and 45.0). fp32 rows of 5120 lose, 57.0 instead of 55.5, and rows normed on both
// sides, whose weights then spill (of 2048 29.9 instead of 23.2, of 5120 70.4 and 68.9).
// Wider rows need more threads, which have 72 registers with 448 (96 with 320, and 32 to
// 56 bytes spilled): 208 to 372 bytes spill, rows of 6144 100 instead of 74, of 7168 110
// instead of 80.
constexpr int kTwoThreads = 320;
template <typename TA, typename TR, int kChunks, bool kWarpRow, bool kPost, bool kTwo = false>
__global__ void __launch_bounds__(kWarpRow ? 32 * kRowsPerBlock : kTwo ? kTwoThreads : kMostKeep,
                                  kWarpRow ? (kPost ? 4 : 5) : kTwo ? 2 : 1)
    norm_whole_kernel(NormArgs a) {
  constexpr int V = chunk_of<TA, TR>();
  __shared__ float s_sum[2][32];
  int turn = 0;
  const int warp = threadIdx.x >> 5, lane = kWarpRow ? threadIdx.x & 31 : threadIdx.x;
  const int lanes = kWarpRow ? 32 : blockDim.x;
  const int step = kWarpRow ? gridDim.x * kRowsPerBlock : gridDim.x;
  int t = kWarpRow ? blockIdx.x * kRowsPerBlock + warp : blockIdx.x;
  const int H = a.H;
  const float inv = 1.0f / static_cast<float>(H);
  pdl_enter();
  // this thread's first chunk of its first row, and of the rows that follow
  const TR* x = static_cast<const TR*>(a.x) + t * a.x_stride + lane * V;
  const TA* y = static_cast<const TA*>(a.y) + (a.y ? t * a.y_stride + lane * V : 0);
  const bool by_channel = a.gate && a.gate_channel, full = by_channel && a.gate_token != 0;
  const TA* gate = static_cast<const TA*>(a.gate) +
                   (a.gate ? t * a.gate_token + (by_channel ? lane * V : 0) : 0);
  TR* x_out = static_cast<TR*>(a.x_out) + (a.x_out ? static_cast<long>(t) * H + lane * V : 0);
  TA* h = static_cast<TA*>(a.h) + (a.h ? static_cast<long>(t) * H + lane * V : 0);
  const int span = lanes * V, rest = H - lane * V;  // chunk c is there while c * span < rest
  auto there = [&](int c) { return c * span < rest; };

  Raw<TR, V> raw_x[kChunks];
  Raw<TA, V> raw_y[kChunks], raw_g[kChunks];
  float w_pre[kChunks][V], w_post[kPost ? kChunks : 1][V];
  auto next_row = [&] {
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
      if (there(c)) {
        fetch(raw_x[c], x + c * span);
        if (a.y) fetch(raw_y[c], y + c * span);
      }
    x += step * a.x_stride;
    y += step * a.y_stride;
  };
  auto next_gates = [&] {
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
      if (there(c)) fetch(raw_g[c], gate + c * span);
    gate += step * a.gate_token;
  };
  auto weights = [&](const float* w, float(&v)[V], int c) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = w && there(c) ? w[c * span + lane * V + i] + a.offset : 1.0f;
  };
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(raw_x[0]) / 4); ++i) raw_x[c].w[i] = 0;
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(raw_y[0]) / 4); ++i) raw_y[c].w[i] = raw_g[c].w[i] = 0;
  }
  if (t < a.T) {
    next_row();
    if (by_channel) next_gates();
  }
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    weights(a.pre_w, w_pre[c], c);
    if constexpr (kPost) weights(a.post_w, w_post[c], c);
  }
  for (; t < a.T; t += step) {
    float r[kChunks][V], u[kChunks][V];
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      unpack(raw_x[c], r[c]);
      unpack(raw_y[c], u[c]);
    }
    float every = a.scale;
    if (a.gate && !by_channel) {
      const float g = one(gate);
      every *= a.sigmoid ? sigmoid(g) : g;
      gate += step * a.gate_token;
    }
    if (t < a.T - step) next_row();

    auto norm = [&](float(&v)[kChunks][V], const float(&w)[kChunks][V], const float* b) {
      if (a.layer) {
        float sum = 0.0f;
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
#pragma unroll
          for (int i = 0; i < V; ++i) sum += v[c][i];
        const float mean = row_sum<kWarpRow>(sum, s_sum, turn) * inv;
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
          if (there(c)) {
#pragma unroll
            for (int i = 0; i < V; ++i) v[c][i] -= mean;
          }
      }
      float sums[2] = {0.0f, 0.0f};
#pragma unroll
      for (int c = 0; c < kChunks; ++c)
#pragma unroll
        for (int i = 0; i < V; ++i) sums[i & 1] += v[c][i] * v[c][i];
      const float f =
          1.0f / sqrtf(row_sum<kWarpRow>(sums[0] + sums[1], s_sum, turn) * inv + a.eps);
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[c][i] = v[c][i] * f * w[c][i];
      }
      if (b) {
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
          if (there(c)) {
#pragma unroll
            for (int i = 0; i < V; i += 4) {
              const float4 f4 = *reinterpret_cast<const float4*>(b + c * span + lane * V + i);
              v[c][i] += f4.x, v[c][i + 1] += f4.y, v[c][i + 2] += f4.z, v[c][i + 3] += f4.w;
            }
          }
      }
    };
    if (a.y) {
      if constexpr (kPost) norm(u, w_post, a.post_b);
      if (by_channel) {
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          float g[V];
          unpack(raw_g[c], g);
#pragma unroll
          for (int i = 0; i < V; ++i) u[c][i] *= a.sigmoid ? sigmoid(g[i]) : g[i];
        }
        if (full && t < a.T - step) next_gates();
      }
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
#pragma unroll
        for (int i = 0; i < V; ++i) r[c][i] += every * u[c][i];
        if (a.x_out && there(c)) put_chunk<V>(x_out + c * span, r[c]);
      }
      x_out += static_cast<long>(step) * H;
    }
    if (!a.h) continue;
    norm(r, w_pre, a.pre_b);
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
      if (there(c)) put_chunk<V>(h + c * span, r[c]);
    h += static_cast<long>(step) * H;
  }
}

template <typename TA, typename TR, int kChunks, bool kWarpRow, bool kPost, bool kTwo = false>
cudaError_t launch_whole(const NormArgs& a, int sms, cudaStream_t st) {
  constexpr int kWarp = 32 * chunk_of<TA, TR>() * kChunks;
  const int threads = kWarpRow ? 32 * kRowsPerBlock : (a.H + kWarp - 1) / kWarp * 32;
  const int rows = kWarpRow ? kRowsPerBlock : 1;
  auto* kern = &norm_whole_kernel<TA, TR, kChunks, kWarpRow, kPost, kTwo>;
  // as many blocks as an SM holds, by size (0: not asked yet)
  static std::atomic<int> held[kMostKeep / 32 + 1] = {};
  int blocks = held[threads / 32].load(std::memory_order_relaxed);
  if (blocks == 0) {
    const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&blocks, kern, threads, 0);
    if (e != cudaSuccess) return e;
    if (blocks < 1) blocks = 1;
    held[threads / 32].store(blocks, std::memory_order_relaxed);
  }
  const long need = (static_cast<long>(a.T) + rows - 1) / rows, fit = static_cast<long>(sms) * blocks;
  return launch_pdl(kern, dim3(static_cast<unsigned>(need < fit ? need : fit)), dim3(threads), 0, st, a);
}

// Elements that the threads of a row have to cover.
int row_span(const NormArgs& a, bool whole) { return a.H + (whole ? 0 : 3); }

template <typename TA, typename TR, int kGroups, bool kWarpRow, bool kWhole, bool kAlike>
cudaError_t launch_any(const NormArgs& a, int sms, cudaStream_t st) {
  constexpr int kWarp = 32 * 4 * kGroups;  // elements of a warp
  const int threads =
      kWarpRow ? 32 * kRowsPerBlock : (row_span(a, kWhole) + kWarp - 1) / kWarp * 32;
  const int rows = kWarpRow ? kRowsPerBlock : 1;
  const int stage = row_bytes(a.H, sizeof(TR)) + (a.y ? row_bytes(a.H, sizeof(TA)) : 0) +
                    (a.gate && a.gate_channel && a.gate_token ? row_bytes(a.H, sizeof(TA)) : 0);
  // blocks per SM by threads and memory, then as many stages as keep memory busy
  int blocks = kMostThreads / threads;
  if (blocks > kSmemPerSm / (rows * stage)) blocks = kSmemPerSm / (rows * stage);
  if (blocks < 1) blocks = 1;
  int stages = 1;
  while (stages < kMostStages && blocks * stages * rows * stage < kAhead &&
         blocks * (stages + 1) * rows * stage <= kSmemPerSm)
    ++stages;
  const long need = (static_cast<long>(a.T) + rows - 1) / rows;
  const long fit = static_cast<long>(sms) * blocks;
  if (need <= fit) stages = 1;  // a row each
  auto* kern = &norm_any_kernel<TA, TR, kGroups, kWarpRow, kWhole, kAlike>;
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = opt_in_smem(reinterpret_cast<const void*>(kern), kSmemMost, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(static_cast<unsigned>(need < fit ? need : fit)), dim3(threads),
                    static_cast<size_t>(stages) * rows * stage, st, a, stages, stage);
}

template <typename TA, typename TR>
cudaError_t launch_types(const NormArgs& a, int sms, cudaStream_t st) {
  // the place of a row's first element within a group of four, as the outputs'
  auto alike = [&](const void* p, long stride, size_t size) {
    return reinterpret_cast<uintptr_t>(p) % (4 * size) == 0 && (stride - a.H) % 4 == 0;
  };
  const bool same = alike(a.x, a.x_stride, sizeof(TR)) && (!a.y || alike(a.y, a.y_stride, sizeof(TA))) &&
                    (!a.gate || !a.gate_channel ||
                     alike(a.gate, a.gate_token ? a.gate_token : a.H, sizeof(TA)));
  const bool whole = same && a.H % 4 == 0, post = a.y && a.post;
  const int span = row_span(a, whole);
  constexpr int V = chunk_of<TA, TR>(), kRow = 16 / V;  // chunks per thread
  auto chunks = [&](const void* p, long stride, size_t size) {
    return reinterpret_cast<uintptr_t>(p) % (V * size) == 0 && stride % V == 0;
  };
  if (a.H % V == 0 && chunks(a.x, a.x_stride, sizeof(TR)) &&
      (!a.y || chunks(a.y, a.y_stride, sizeof(TA))) &&
      (!a.gate || !a.gate_channel || chunks(a.gate, a.gate_token, sizeof(TA)))) {
    if (a.H <= 32 * V)  // heads
      return post ? launch_whole<TA, TR, 1, true, true>(a, sms, st)
                  : launch_whole<TA, TR, 1, true, false>(a, sms, st);
    if (a.H <= 32 * 16)
      return post ? launch_whole<TA, TR, kRow, true, true>(a, sms, st)
                  : launch_whole<TA, TR, kRow, true, false>(a, sms, st);
    if constexpr (sizeof(TA) == 2)
      if (a.H <= kTwoThreads * 16 && !post && a.T > 2 * sms)
        return launch_whole<TA, TR, kRow, false, false, true>(a, sms, st);
    if (a.H <= kMostKeep * 16)
      return post ? launch_whole<TA, TR, kRow, false, true>(a, sms, st)
                  : launch_whole<TA, TR, kRow, false, false>(a, sms, st);
  }
  if (whole) return launch_any<TA, TR, 4, false, true, true>(a, sms, st);
  if (span <= 32 * 4 && same) return launch_any<TA, TR, 1, true, false, true>(a, sms, st);
  if (span <= 32 * 16)
    return same ? launch_any<TA, TR, 4, true, false, true>(a, sms, st)
                : launch_any<TA, TR, 4, true, false, false>(a, sms, st);
  // (five groups: 16384 channels and the places before the first one)
  if (!same) return launch_any<TA, TR, 5, false, false, false>(a, sms, st);
  return span <= kMostThreads * 16 ? launch_any<TA, TR, 4, false, false, true>(a, sms, st)
                                   : launch_any<TA, TR, 5, false, false, true>(a, sms, st);
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
