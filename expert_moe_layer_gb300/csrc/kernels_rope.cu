// Rotary positions, the append to the 4-bit paged cache, and reading it back.
//
// All of it is elementwise over rows, so memory bounds it at prompt sizes and
// launch latency at decode sizes. A thread takes 32 channels of a head (two
// groups of 16): the two halves of 16 pairs for the half layout, 32 neighbours
// for the interleaved one. Either way these are the pairs 16u .. 16u + 15, so
// their cosines and sines are loaded once and used for several heads, a key's
// rotation and its quantisation happen in registers, and a row rotated in
// place is read and written by one thread only.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "attn.h"
#include "kv4.cuh"
#include "launch.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f(float v) {
  return v;
}
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 v) {
  return __bfloat162float(v);
}
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f(float v) {
  return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f(float v) {
  return __float2bfloat16_rn(v);
}

// 16 consecutive elements, 16-byte aligned.
__device__ __forceinline__ void load16(const float* p, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 v = reinterpret_cast<const float4*>(p)[i];
    x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
  }
}
__device__ __forceinline__ void load16(const __nv_bfloat16* p, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 v = reinterpret_cast<const uint4*>(p)[i];
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
      x[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
  }
}
__device__ __forceinline__ void store16(float* p, const float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    reinterpret_cast<float4*>(p)[i] =
        make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
}
__device__ __forceinline__ void store16(__nv_bfloat16* p, const float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(x[8 * i + 2 * j], x[8 * i + 2 * j + 1]);
      w[j] = *reinterpret_cast<const uint32_t*>(&b);
    }
    reinterpret_cast<uint4*>(p)[i] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// The two products and their sum are rounded one by one (no fused
// multiply-add), so that a key's bits, and with them its 4-bit code, do not
// depend on how a compiler contracts the expression.
__device__ __forceinline__ void turn(float a, float b, float c, float s, float& u, float& v) {
  u = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  v = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
}

// Where a token's group of 16 channels is stored.
template <typename T>
__device__ __forceinline__ void store_group(const RopeArgs& a, bool value, long slot, int head,
                                            int group, float (&x)[16]) {
  const KvBlock blk = kv_block(a.page_size, a.D);
  const long page = slot / a.page_size;
  const int row = static_cast<int>(slot - page * a.page_size);
  uint8_t* base = a.cache + (page * a.kv_heads + head) * static_cast<long>(blk.bytes);
  uint32_t codes[2];
  const uint32_t s8 = kv_store_group(x, value ? a.v_inv : a.k_inv, codes);
  *reinterpret_cast<uint2*>(base + (value ? blk.v_code : 0u) + row * (a.D / 2) + group * 8) =
      make_uint2(codes[0], codes[1]);
  base[(value ? blk.v_scale : blk.k_scale) + row * (a.D / kKvGroup) + group] =
      static_cast<uint8_t>(s8);
}

// A chunk is up to `hb` heads of q, then of k, then of v, of one token.
struct Chunk {
  int t, kind, h0, h1;  // kind: 0 q, 1 k, 2 v
};
__device__ __forceinline__ Chunk chunk_of(const RopeArgs& a, unsigned rest, int hb, int cq, int ck) {
  const unsigned per = cq + 2 * ck;
  Chunk c;
  c.t = static_cast<int>(rest / per);
  int i = static_cast<int>(rest - c.t * per);
  c.kind = i < cq ? 0 : i < cq + ck ? 1 : 2;
  i -= c.kind == 0 ? 0 : c.kind == 1 ? cq : cq + ck;
  c.h0 = i * hb;
  c.h1 = min(c.h0 + hb, c.kind ? a.kv_heads : a.q_heads);
  return c;
}

// The table row of a token, or nullptr (nothing rotates, or `ok` turns false).
__device__ __forceinline__ const float* table_row(const RopeArgs& a, int t, bool& ok) {
  if (a.R == 0) return nullptr;
  const int pos = a.positions[t];
  ok = pos >= 0 && pos < a.table_rows;
  if (!ok && a.status) atomicOr(a.status, MOE_DEV_BAD_POSITION);
  return a.table + static_cast<long>(ok ? pos : 0) * a.R;
}
__device__ __forceinline__ long slot_of(const RopeArgs& a, int t) {
  const long slot = a.slots[t];
  if (slot >= 0 && slot < a.n_slots) return slot;
  if (slot != -1 && a.status) atomicOr(a.status, MOE_DEV_BAD_SLOT);
  return -1;
}

// D and R multiples of 32, 16-byte aligned rows.
template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) rope_kernel(RopeArgs a, int hb, int cq, int ck,
                                                        unsigned total) {
  pdl_enter();
  const unsigned idx = blockIdx.x * kThreads + threadIdx.x;
  if (idx >= total) return;
  const unsigned units = a.D / 32;
  const int u = static_cast<int>(idx % units);
  const Chunk c = chunk_of(a, idx / units, hb, cq, ck);
  long slot = 0;
  if (c.kind && (slot = slot_of(a, c.t)) < 0) return;
  bool ok = true;
  const int pairs = a.R / 2;
  const bool turns = c.kind != 2 && 16 * u < pairs;
  float cs[16], sn[16];
  if (c.kind != 2) {
    const float* row = table_row(a, c.t, ok);
    if (!ok) return;
    if (turns) {
      load16(row + 16 * u, cs);
      load16(row + pairs + 16 * u, sn);
      if (a.inverse)
#pragma unroll
        for (int i = 0; i < 16; ++i) sn[i] = -sn[i];
    }
  } else if (a.R > 0) {  // a token with a bad position is not stored at all
    table_row(a, c.t, ok);
    if (!ok) return;
  }
  // first channels of the two groups
  int c0 = 32 * u, c1 = 32 * u + 16;
  if (!kInterleaved && turns) c0 = 16 * u, c1 = pairs + 16 * u;
  const Rows rows = c.kind == 0 ? a.q : c.kind == 1 ? a.k : a.v;
  const T* src = static_cast<const T*>(rows.p) + c.t * rows.token;
#pragma unroll 2
  for (int h = c.h0; h < c.h1; ++h) {
    float x[16], y[16];
    load16(src + h * rows.head + c0, x);
    load16(src + h * rows.head + c1, y);
    if (turns) {
      if (kInterleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          turn(x[2 * i], x[2 * i + 1], cs[i], sn[i], x[2 * i], x[2 * i + 1]);
          turn(y[2 * i], y[2 * i + 1], cs[8 + i], sn[8 + i], y[2 * i], y[2 * i + 1]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) turn(x[i], y[i], cs[i], sn[i], x[i], y[i]);
      }
    }
    if (c.kind == 0) {
      T* dst = static_cast<T*>(a.q_out) + (static_cast<long>(c.t) * a.q_heads + h) * a.D;
      store16(dst + c0, x);
      store16(dst + c1, y);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = to_f(from_f<T>(x[i])), y[i] = to_f(from_f<T>(y[i]));
      store_group<T>(a, c.kind == 2, slot, h, c0 / kKvGroup, x);
      store_group<T>(a, c.kind == 2, slot, h, c1 / kKvGroup, y);
    }
  }
}

// Any D, R and strides, one element at a time. A query's pairs are shared out
// over the head's threads (each pair read and written by one thread); keys and
// values go group by group, a key's other channels read where they are.
template <typename T>
__global__ void __launch_bounds__(kThreads) rope_any_kernel(RopeArgs a, int hb, int cq, int ck,
                                                            unsigned total) {
  pdl_enter();
  const unsigned idx = blockIdx.x * kThreads + threadIdx.x;
  if (idx >= total) return;
  const int units = (a.D + 15) / 16;
  const int u = static_cast<int>(idx % units);
  const Chunk c = chunk_of(a, idx / units, hb, cq, ck);
  long slot = 0;
  if (c.kind && (slot = slot_of(a, c.t)) < 0) return;
  bool ok = true;
  const float* row = table_row(a, c.t, ok);
  if (!ok) return;
  const int pairs = a.R / 2;
  const float sign = a.inverse ? -1.0f : 1.0f;
  const Rows rows = c.kind == 0 ? a.q : c.kind == 1 ? a.k : a.v;
  for (int h = c.h0; h < c.h1; ++h) {
    const T* src = static_cast<const T*>(rows.p) + c.t * rows.token + h * rows.head;
    if (c.kind == 0) {
      T* dst = static_cast<T*>(a.q_out) + (static_cast<long>(c.t) * a.q_heads + h) * a.D;
      for (int i = u; i < pairs; i += units) {
        const int ia = a.interleaved ? 2 * i : i, ib = a.interleaved ? 2 * i + 1 : i + pairs;
        float p, q;
        turn(to_f(src[ia]), to_f(src[ib]), row[i], sign * row[pairs + i], p, q);
        dst[ia] = from_f<T>(p);
        dst[ib] = from_f<T>(q);
      }
      for (int i = a.R + u; i < a.D; i += units) dst[i] = src[i];
      continue;
    }
    float x[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int ch = 16 * u + j;
      float v = to_f(src[ch]);
      if (c.kind == 1 && ch < a.R) {
        const int i = a.interleaved ? ch / 2 : ch < pairs ? ch : ch - pairs;
        const bool first = a.interleaved ? (ch & 1) == 0 : ch < pairs;
        const int other = a.interleaved ? ch ^ 1 : first ? ch + pairs : ch - pairs;
        const float w = to_f(src[other]);
        float p, q;
        turn(first ? v : w, first ? w : v, row[i], sign * row[pairs + i], p, q);
        v = first ? p : q;
      }
      x[j] = to_f(from_f<T>(v));
    }
    store_group<T>(a, c.kind == 2, slot, h, u, x);
  }
}

// A frequency is a 64-bit fraction of a turn per position, so the angle's
// fraction of a turn is an integer product modulo 2^64: exact for every int32
// position, where an fp32 angle would lose all its bits at far positions and
// fp64 arithmetic is slow on this part. The fraction's leading 24 bits go
// through sincospif, the rest corrects its result to first order.
__global__ void __launch_bounds__(kThreads) rope_table_kernel(RopeTurns turns, int pairs,
                                                              float gain, int n,
                                                              const int32_t* positions,
                                                              float* table, int rows_per_block) {
  pdl_enter();
  const int lanes = kThreads / pairs;  // rows a block writes at a time (0: more pairs than threads)
  const int r0 = blockIdx.x * rows_per_block, r1 = min(n, r0 + rows_per_block);
  const int first = lanes ? threadIdx.x % pairs : threadIdx.x;
  if (lanes && static_cast<int>(threadIdx.x) >= lanes * pairs) return;
  for (int i = first; i < pairs; i += lanes ? pairs : kThreads) {
    const unsigned long long f = turns.f[i];
    for (int r = r0 + (lanes ? static_cast<int>(threadIdx.x) / pairs : 0); r < r1;
         r += lanes ? lanes : 1) {
      const long long pos = positions ? positions[r] : r;
      const long long t = static_cast<long long>(f * static_cast<unsigned long long>(pos));
      const float head = __ll2float_rn(t);
      const float rest = __ll2float_rn(t - __float2ll_rn(head)) * 0x1p-63f * 3.14159265f;
      float s, c;
      sincospif(head * 0x1p-63f, &s, &c);
      float* row = table + static_cast<long>(r) * (2 * pairs);
      row[i] = gain * fmaf(-s, rest, c);
      row[pairs + i] = gain * fmaf(c, rest, s);
    }
  }
}

// One thread per (slot, head, group of 16 channels): keys and values.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    kv_read_kernel(int N, const int64_t* slots, const uint8_t* cache, long n_slots, int kv_heads,
                   int D, int page_size, float k_scale, float v_scale, T* k_out, T* v_out,
                   unsigned* status) {
  pdl_enter();
  const unsigned groups = D / kKvGroup;
  const unsigned idx = blockIdx.x * kThreads + threadIdx.x;
  const unsigned g = idx % groups, rest = idx / groups;
  const unsigned h = rest % kv_heads, i = rest / kv_heads;
  if (i >= static_cast<unsigned>(N)) return;
  const long slot = slots[i];
  const bool ok = slot >= 0 && slot < n_slots;
  if (!ok && slot != -1 && status) atomicOr(status, MOE_DEV_BAD_SLOT);
  const KvBlock blk = kv_block(page_size, D);
  const long page = ok ? slot / page_size : 0;
  const int row = ok ? static_cast<int>(slot - page * page_size) : 0;
  const uint8_t* base = cache + (page * kv_heads + h) * static_cast<long>(blk.bytes);
  const long at = (static_cast<long>(i) * kv_heads + h) * D + g * kKvGroup;
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    float x[16] = {};
    if (ok) {
      const uint2 w = *reinterpret_cast<const uint2*>(base + (kv ? blk.v_code : 0u) +
                                                      row * (D / 2) + g * 8);
      const uint32_t s2 = base[(kv ? blk.v_scale : blk.k_scale) + row * groups + g];
      const uint32_t s = f16_low_twice(e4m3x2_to_f16(s2));
      uint32_t p[8];
      e2m1_to_f16(w.x, *reinterpret_cast<uint32_t(*)[4]>(p));
      e2m1_to_f16(w.y, *reinterpret_cast<uint32_t(*)[4]>(p + 4));
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t q = hmul2(p[j], s);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&q));
        x[2 * j] = f.x * (kv ? v_scale : k_scale);
        x[2 * j + 1] = f.y * (kv ? v_scale : k_scale);
      }
    }
    store16((kv ? v_out : k_out) + at, x);
  }
}

bool rows_aligned(const Rows& r, int eb) {
  return (reinterpret_cast<uintptr_t>(r.p) | static_cast<uintptr_t>(r.token * eb) |
          static_cast<uintptr_t>(r.head * eb)) % 16 == 0;
}

template <typename T>
cudaError_t launch_rope_t(const RopeArgs& a, cudaStream_t st) {
  const int eb = sizeof(T);
  const bool fast = a.D % 32 == 0 && a.R % 32 == 0 &&
                    (a.q_heads == 0 || (rows_aligned(a.q, eb) &&
                                        reinterpret_cast<uintptr_t>(a.q_out) % 16 == 0)) &&
                    (a.kv_heads == 0 || (rows_aligned(a.k, eb) && rows_aligned(a.v, eb))) &&
                    reinterpret_cast<uintptr_t>(a.table) % 16 == 0;
  const long units = fast ? a.D / 32 : (a.D + 15) / 16;
  // heads per thread: 4 once that still gives every SM its 2048 threads
  const long all = units * a.T * (a.q_heads + 2l * a.kv_heads);
  const int hb = all / 4 >= 152l * 2048 ? 4 : 1;
  const int cq = (a.q_heads + hb - 1) / hb, ck = (a.kv_heads + hb - 1) / hb;
  const long total = units * a.T * (cq + 2l * ck);
  if (total == 0) return cudaSuccess;
  if (total > 0xffffff00l) return cudaErrorInvalidValue;
  auto kern = !fast            ? &rope_any_kernel<T>
              : a.interleaved ? &rope_kernel<T, true>
                              : &rope_kernel<T, false>;
  return launch_pdl(kern, dim3(static_cast<unsigned>((total + kThreads - 1) / kThreads)),
                    dim3(kThreads), 0, st, a, hb, cq, ck, static_cast<unsigned>(total));
}

}  // namespace

cudaError_t launch_rope(bool bf16, const RopeArgs& a, cudaStream_t st) {
  return bf16 ? launch_rope_t<__nv_bfloat16>(a, st) : launch_rope_t<float>(a, st);
}

cudaError_t launch_rope_table(const RopeTurns& turns, int pairs, float gain, int n,
                              const int32_t* positions, float* table, cudaStream_t st) {
  // enough rows per block to use each thread's frequency several times, few
  // enough to give every SM work
  const int lanes = pairs <= kThreads ? kThreads / pairs : 1;
  int rows = n / (152 * 8);
  rows = (rows < lanes ? lanes : rows + lanes - 1) / lanes * lanes;
  return launch_pdl(&rope_table_kernel, dim3((n + rows - 1) / rows), dim3(kThreads), 0, st, turns,
                    pairs, gain, n, positions, table, rows);
}

cudaError_t launch_kv_read(bool bf16, int N, const int64_t* slots, const uint8_t* cache,
                           long n_slots, int kv_heads, int D, int page_size, float k_scale,
                           float v_scale, void* k_out, void* v_out, unsigned* status,
                           cudaStream_t st) {
  const long total = static_cast<long>(N) * kv_heads * (D / kKvGroup);
  const dim3 grid(static_cast<unsigned>((total + kThreads - 1) / kThreads));
  if (bf16)
    return launch_pdl(&kv_read_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, st, N, slots,
                      cache, n_slots, kv_heads, D, page_size, k_scale, v_scale,
                      static_cast<__nv_bfloat16*>(k_out), static_cast<__nv_bfloat16*>(v_out),
                      status);
  return launch_pdl(&kv_read_kernel<float>, grid, dim3(kThreads), 0, st, N, slots, cache, n_slots,
                    kv_heads, D, page_size, k_scale, v_scale, static_cast<float*>(k_out),
                    static_cast<float*>(v_out), status);
}

}  // namespace moe
