// Rotary positions, the append to the 4-bit paged cache, and reading it back.
//
// All of it is elementwise over rows, so memory bounds it at prompt sizes and
// launch latency at decode sizes. A thread takes two chunks of 16 bytes of a
// head, half the rotated channels apart: the two sides of the half layout's
// pairs, or neighbouring pairs of the interleaved one. Neighbouring lanes hold
// neighbouring chunks, so that every access covers whole sectors (with 32 bytes
// per lane and chunk, 4097 x 16 heads of 256 in fp32 took 34.4 us instead of
// 27.4). The rows are loaded before the position and the table row, which have
// to be fetched one after the other (23.0 us then: 6.0 TB/s, 89 % of a copy's
// rate; bf16, 8192 x 40 heads of 128 half rotated: 29.8 us, 5.7 TB/s). The
// cosines and sines serve several heads; a row rotated in place is read and
// written by one thread only.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "attn.h"
#include "kv4.cuh"
#include "launch.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kSms = 152;  // of this part: sizes of work are measured by it
// CTAs per SM of the kernels of one and of four heads per thread. Three of the
// latter spill 10 registers and are still faster (29.8 us, the case below) than
// two without (34.0) or four (34.3); the former need the registers of five.
constexpr int ctas_per_sm(int heads) { return heads == 1 ? 5 : 3; }

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

// One 16-byte chunk: 8 bf16 or 4 fp32 elements.
__device__ __forceinline__ void unpack_chunk(uint4 v, float (&x)[4]) {
  x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y);
  x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
}
__device__ __forceinline__ void unpack_chunk(uint4 v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[2 * j] = __uint_as_float(w[j] << 16);
    x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
  }
}
__device__ __forceinline__ void store_chunk(float* p, const float (&x)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void store_chunk(__nv_bfloat16* p, const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
    w[j] = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// N consecutive floats, aligned to their size or to 16 bytes.
template <int N>
__device__ __forceinline__ void load_floats(const float* p, float* x) {
  if constexpr (N == 2) {
    const float2 v = *reinterpret_cast<const float2*>(p);
    x[0] = v.x, x[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const float4 v = reinterpret_cast<const float4*>(p)[i];
      x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
    }
  }
}

// The two products and their sum are rounded one by one (no fused
// multiply-add), so that a key's bits, and with them its 4-bit code, do not
// depend on how a compiler contracts the expression.
__device__ __forceinline__ void turn(float a, float b, float c, float s, float& u, float& v) {
  u = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  v = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
}

// The (page, kv head) block and row of a slot.
struct Place {
  uint8_t* block;  // of kv head 0
  int row;
};
__device__ __forceinline__ Place place_of(const RopeArgs& a, long slot) {
  const long page = slot >> a.page_shift;
  return {a.cache + page * a.kv_heads * static_cast<long>(kv_block(1 << a.page_shift, a.D).bytes),
          static_cast<int>(slot) & ((1 << a.page_shift) - 1)};
}
// Stores V channels from `ch`; the 16 / V neighbouring lanes of the group's
// channels do the same together.
template <int V>
__device__ __forceinline__ void store_codes(const RopeArgs& a, bool value, Place at, int head,
                                            int ch, const float (&x)[V], unsigned lanes) {
  const KvBlock blk = kv_block(1 << a.page_shift, a.D);
  uint8_t* base = at.block + head * static_cast<long>(blk.bytes);
  float y[V], top = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float t = __fmul_rn(x[i], value ? a.v_inv : a.k_inv);
    y[i] = t == t ? fminf(fmaxf(t, -kKvMost), kKvMost) : 0.0f;
    top = fmaxf(top, fabsf(y[i]));
  }
#pragma unroll
  for (int d = 1; d < kKvGroup / V; d *= 2) top = fmaxf(top, __shfl_xor_sync(lanes, top, d));
  uint32_t codes[(V + 7) / 8];
  const uint32_t s8 = kv_codes<V>(y, top, codes);
  uint8_t* dst = base + (value ? blk.v_code : 0u) + at.row * (a.D / 2) + ch / 2;
  if constexpr (V == 16)
    *reinterpret_cast<uint2*>(dst) = make_uint2(codes[0], codes[1]);
  else if constexpr (V == 8)
    *reinterpret_cast<uint32_t*>(dst) = codes[0];
  else
    *reinterpret_cast<uint16_t*>(dst) = static_cast<uint16_t>(codes[0]);
  if (ch % kKvGroup == 0)
    base[(value ? blk.v_scale : blk.k_scale) + at.row * (a.D / kKvGroup) + ch / kKvGroup] =
        static_cast<uint8_t>(s8);
}

// Up to `hb` heads of k, of v or of q of one token. The kinds follow one
// another over the whole grid, so that no warp has to do two of them.
struct Chunk {
  int t, kind, h0, h1;  // kind: 0 q, 1 k, 2 v
};
__device__ __forceinline__ Chunk chunk_of(const RopeArgs& a, unsigned i, int hb, int cq, int ck) {
  const unsigned nk = static_cast<unsigned>(a.T) * ck;
  Chunk c;
  c.kind = i < nk ? 1 : i < 2 * nk ? 2 : 0;
  i -= c.kind == 1 ? 0 : c.kind == 2 ? nk : 2 * nk;
  const unsigned per = c.kind ? ck : cq;
  c.t = static_cast<int>(i / per);
  c.h0 = static_cast<int>(i - c.t * per) * hb;
  c.h1 = min(c.h0 + hb, c.kind ? a.kv_heads : a.q_heads);
  return c;
}

// The table row of a token, or nullptr (nothing rotates, or `ok` turns false). An
// append's queries look at their token's slot here, fetched beside the position:
// nowhere is no matter to them, outside the cache skips them. (One after the
// other costs 8192 tokens of 40 and 8 heads 2 us, side by side 0.5 us.)
__device__ __forceinline__ const float* table_row(const RopeArgs& a, int t, int kind, bool& ok) {
  const int pos = a.R ? a.positions[t] : 0;
  if (kind == 0 && a.slots) {
    const long slot = a.slots[t];
    ok = slot >= -1 && slot < a.n_slots;
    if (!ok && a.status) atomicOr(a.status, MOE_DEV_BAD_SLOT);
  }
  if (a.R == 0) return nullptr;
  const bool known = pos >= 0 && pos < a.table_rows;
  if (!known && a.status) atomicOr(a.status, MOE_DEV_BAD_POSITION);
  ok &= known;
  return a.table + static_cast<long>(known ? pos : 0) * a.R;
}
// The slot of a token's keys and values, or -1.
__device__ __forceinline__ long slot_of(const RopeArgs& a, int t) {
  const long slot = a.slots[t];
  if (slot >= 0 && slot < a.n_slots) return slot;
  if (slot != -1 && a.status) atomicOr(a.status, MOE_DEV_BAD_SLOT);
  return -1;
}

// D and R multiples of 32, 16-byte aligned rows.
template <typename T, bool kInterleaved, int kHeads>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(kHeads))
    rope_kernel(RopeArgs a, int cq, int ck, unsigned total) {
  constexpr int V = 16 / sizeof(T);     // elements of a chunk
  constexpr int kSharers = kKvGroup / V;  // lanes that share a scale
  pdl_enter();
  const unsigned idx = blockIdx.x * kThreads + threadIdx.x;
  if (idx >= total) return;
  const unsigned units = a.D / (2 * V);
  const int u = static_cast<int>(idx % units);
  const Chunk c = chunk_of(a, idx / units, kHeads, cq, ck);
  const int pairs = a.R / 2, turned = pairs / V;  // units that rotate
  const bool turns = c.kind != 2 && u < turned;
  // first channels of the two chunks
  int c0 = V * u, c1 = a.D / 2 + V * u;
  if (c.kind != 2) {
    c0 = turns ? V * u : a.R + V * (u - turned);
    c1 = c0 + (turns ? pairs : (a.D - a.R) / 2);
  }
  // the rows first: they depend on nothing that has to be fetched before
  const Rows rows = c.kind == 0 ? a.q : c.kind == 1 ? a.k : a.v;
  const T* src = static_cast<const T*>(rows.p) + c.t * rows.token + c.h0 * rows.head;
  uint4 raw[kHeads][2];
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    if (c.h0 + i < c.h1) {
      raw[i][0] = *reinterpret_cast<const uint4*>(src + i * rows.head + c0);
      raw[i][1] = *reinterpret_cast<const uint4*>(src + i * rows.head + c1);
    }
  }
  long slot = 0;
  if (c.kind && (slot = slot_of(a, c.t)) < 0) return;
  bool ok = true;
  const float* row = table_row(a, c.t, c.kind, ok);
  if (!ok) return;
  float cs[V], sn[V];
  if (turns) {
    if (kInterleaved) {
      load_floats<V / 2>(row + c0 / 2, cs);
      load_floats<V / 2>(row + c1 / 2, cs + V / 2);
      load_floats<V / 2>(row + pairs + c0 / 2, sn);
      load_floats<V / 2>(row + pairs + c1 / 2, sn + V / 2);
    } else {
      load_floats<V>(row + c0, cs);
      load_floats<V>(row + pairs + c0, sn);
    }
    if (a.inverse)
#pragma unroll
      for (int i = 0; i < V; ++i) sn[i] = -sn[i];
  }
  Place at = {nullptr, 0};
  if (c.kind) at = place_of(a, slot);
  const int lane = threadIdx.x & 31;
  const unsigned lanes = ((1u << kSharers) - 1u) << (lane & ~(kSharers - 1));
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    const int h = c.h0 + i;
    if (h >= c.h1) break;
    float x[V], y[V];
    unpack_chunk(raw[i][0], x);
    unpack_chunk(raw[i][1], y);
    if (turns) {
      if (kInterleaved) {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
          turn(x[2 * i], x[2 * i + 1], cs[i], sn[i], x[2 * i], x[2 * i + 1]);
          turn(y[2 * i], y[2 * i + 1], cs[V / 2 + i], sn[V / 2 + i], y[2 * i], y[2 * i + 1]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) turn(x[i], y[i], cs[i], sn[i], x[i], y[i]);
      }
    }
    if (c.kind == 0) {
      T* dst = static_cast<T*>(a.q_out) + (static_cast<long>(c.t) * a.q_heads + h) * a.D;
      store_chunk(dst + c0, x);
      store_chunk(dst + c1, y);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = to_f(from_f<T>(x[i])), y[i] = to_f(from_f<T>(y[i]));
      store_codes<V>(a, c.kind == 2, at, h, c0, x, lanes);
      store_codes<V>(a, c.kind == 2, at, h, c1, y, lanes);
    }
  }
}

// Any even R, 16-byte aligned rows: a thread makes one 16-byte chunk of the
// output. The other elements of a half-layout chunk's pairs start anywhere and
// are read one by one (they are other lanes' chunks, so L1 has them). A row
// rotated in place is read by all of its lanes before any of them writes, which
// one warp has to do: the launch sees to it.
template <typename T, bool kInterleaved, int kHeads>
__global__ void __launch_bounds__(kThreads) rope_wide_kernel(RopeArgs a, int cq, int ck,
                                                             unsigned total) {
  constexpr int V = 16 / sizeof(T);
  constexpr int kSharers = kKvGroup / V;
  pdl_enter();
  const unsigned idx = blockIdx.x * kThreads + threadIdx.x;
  if (idx >= total) return;
  const unsigned units = a.D / V;
  const int c0 = static_cast<int>(idx % units) * V;
  const Chunk c = chunk_of(a, idx / units, kHeads, cq, ck);
  const int pairs = c.kind == 2 ? 0 : a.R / 2;
  const Rows rows = c.kind == 0 ? a.q : c.kind == 1 ? a.k : a.v;
  const T* src = static_cast<const T*>(rows.p) + c.t * rows.token + c.h0 * rows.head;
  uint4 raw[kHeads];
  T other[kInterleaved ? 1 : kHeads][V];
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    if (c.h0 + i < c.h1) {
      const T* p = src + i * rows.head;
      raw[i] = *reinterpret_cast<const uint4*>(p + c0);
      if constexpr (!kInterleaved) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const int ch = c0 + j;
          if (ch < 2 * pairs) other[i][j] = p[ch < pairs ? ch + pairs : ch - pairs];
        }
      }
    }
  }
  long slot = 0;
  if (c.kind && (slot = slot_of(a, c.t)) < 0) return;
  bool ok = true;
  const float* row = table_row(a, c.t, c.kind, ok);
  if (!ok) return;
  float cs[V], sn[V];  // of each channel: own * cos + other * (+- sin)
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int ch = c0 + j;
    if (ch < 2 * pairs) {
      const int pair = kInterleaved ? ch / 2 : ch < pairs ? ch : ch - pairs;
      const bool first = kInterleaved ? j % 2 == 0 : ch < pairs;
      cs[j] = row[pair];
      const float v = row[pairs + pair];
      sn[j] = first != (a.inverse != 0) ? -v : v;
    }
  }
  Place at = {nullptr, 0};
  if (c.kind) at = place_of(a, slot);
  const int lane = threadIdx.x & 31;
  const unsigned lanes = ((1u << kSharers) - 1u) << (lane & ~(kSharers - 1));
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    const int h = c.h0 + i;
    if (h >= c.h1) break;
    float x[V], y[V];
    unpack_chunk(raw[i], x);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      y[j] = x[j];
      if (c0 + j < 2 * pairs) {
        float o;
        if constexpr (kInterleaved) o = x[j ^ 1];
        else o = to_f(other[i][j]);
        y[j] = __fadd_rn(__fmul_rn(x[j], cs[j]), __fmul_rn(o, sn[j]));
      }
    }
    if (c.kind == 0) {
      store_chunk(static_cast<T*>(a.q_out) + (static_cast<long>(c.t) * a.q_heads + h) * a.D + c0, y);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) y[j] = to_f(from_f<T>(y[j]));
      store_codes<V>(a, c.kind == 2, at, h, c0, y, lanes);
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
  const float* row = table_row(a, c.t, c.kind, ok);
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
    store_codes<16>(a, c.kind == 2, place_of(a, slot), h, 16 * u, x, 0);
  }
}

// sin and cos of x/2^32 of a quarter turn, x in [-2^31, 2^31): Taylor's series
// in the fraction u, |u| <= 1/2, whose first missing terms are below 2^-29 (sin,
// (pi/4)^11/11!) and 2^-33 (cos). sin's first coefficient has two parts, so that
// neither its rounding nor the angle's enters.
__device__ __forceinline__ void quarter_sincos(int x, float& s, float& c) {
  constexpr double k1 = 1.5707963267948966, k2 = k1 * k1, k4 = k2 * k2, k8 = k4 * k4;
  constexpr float high = static_cast<float>(k1), low = static_cast<float>(k1 - high);
  const float u = static_cast<float>(x) * 0x1p-32f, z = u * u;
  float p = fmaf(z, static_cast<float>(k8 * k1 / 362880), static_cast<float>(-k4 * k2 * k1 / 5040));
  p = fmaf(z, p, static_cast<float>(k4 * k1 / 120));
  p = fmaf(z, p, static_cast<float>(-k2 * k1 / 6));
  p = fmaf(z, p, low);
  s = fmaf(u, high, u * p);
  float q = fmaf(z, static_cast<float>(-k8 * k2 / 3628800), static_cast<float>(k8 / 40320));
  q = fmaf(z, q, static_cast<float>(-k4 * k2 / 720));
  q = fmaf(z, q, static_cast<float>(k4 / 24));
  q = fmaf(z, q, static_cast<float>(-k2 / 2));
  c = fmaf(z, q, 1.0f);
}

// A frequency is a 64-bit fraction of a turn per position, so the angle's
// fraction of a turn is an integer product modulo 2^64, in which the frequency
// as it is held loses nothing at any int32 position (an fp32 angle would lose all
// its bits at far ones, and fp64 arithmetic is slow on this part). The frequency
// itself comes from fp64 and has 53 bits: the angle is off by 2^-32 at a million
// positions and by up to 2^-21 at 2^31. Of the fraction's leading 32 bits (what
// is cut off is below 2^-29 in the angle), two choose the quarter turn and the
// others the angle in it, within half a quarter either way. 131072 x 64 pairs:
// 17.5 us, 3.8 TB/s written, bound by issue slots (sincospif and a first-order
// correction took 23.4 us, 64-bit conversions instead of integer parts 45). A
// block takes rows enough to use each thread's frequency several times.
__global__ void __launch_bounds__(kThreads) rope_table_kernel(RopeTurns turns, int pairs,
                                                              float gain, int n,
                                                              const int32_t* positions,
                                                              float* table, int rows_per_block) {
  pdl_enter();
  const int lanes = kThreads / pairs;  // rows a block writes at a time
  if (static_cast<int>(threadIdx.x) >= lanes * pairs) return;
  const int i = threadIdx.x % pairs;
  const unsigned long long f = turns.f[i];
  const int r1 = min(n, (static_cast<int>(blockIdx.x) + 1) * rows_per_block);
#pragma unroll 4
  for (int r = blockIdx.x * rows_per_block + threadIdx.x / pairs; r < r1; r += lanes) {
    const long long pos = positions ? positions[r] : r;
    const unsigned long long t = f * static_cast<unsigned long long>(pos);
    const unsigned turn = static_cast<unsigned>(t >> 32);  // of 2^32
    const unsigned quarter = (turn + (1u << 29)) >> 30;
    float qs, qc;
    quarter_sincos(static_cast<int>(turn << 2), qs, qc);
    const float s0 = quarter & 1 ? qc : qs, c0 = quarter & 1 ? qs : qc;
    const float s = __int_as_float(__float_as_int(s0) ^ ((quarter & 2) << 30));
    const float c = __int_as_float(__float_as_int(c0) ^ (((quarter + 1) & 2) << 30));
    float* row = table + static_cast<long>(r) * (2 * pairs);
    row[i] = gain * c;
    row[pairs + i] = gain * s;
  }
}

// One thread per (slot, head, 16 bytes of output): keys and values, whose codes
// are both asked for before the first is converted. 8192 slots of 8 heads of 128
// in bf16 take about 11 us, 3.9 TB/s; four heads per thread gain 2 us there and
// lose as much with longer pages or fewer slots.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    kv_read_kernel(int N, const int64_t* slots, const uint8_t* cache, long n_slots, int kv_heads,
                   int D, int page_shift, float k_scale, float v_scale, T* k_out, T* v_out,
                   unsigned* status) {
  constexpr int V = 16 / sizeof(T);
  pdl_enter();
  const unsigned chunks = D / V;
  const unsigned idx = blockIdx.x * kThreads + threadIdx.x;
  const unsigned rest = idx / chunks, ch = (idx - rest * chunks) * V;
  const unsigned i = rest / kv_heads, h = rest - i * kv_heads;
  if (i >= static_cast<unsigned>(N)) return;
  const long slot = slots[i];
  const bool ok = slot >= 0 && slot < n_slots;
  if (!ok && slot != -1 && status) atomicOr(status, MOE_DEV_BAD_SLOT);
  const KvBlock blk = kv_block(1 << page_shift, D);
  const long page = ok ? slot >> page_shift : 0;
  const int row = ok ? static_cast<int>(slot) & ((1 << page_shift) - 1) : 0;
  const uint8_t* base = cache + (page * kv_heads + h) * static_cast<long>(blk.bytes);
  const long at = (static_cast<long>(i) * kv_heads + h) * D + ch;
  uint32_t w[2], s2[2];
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    const uint8_t* src = base + (kv ? blk.v_code : 0u) + row * (D / 2) + ch / 2;
    if constexpr (V == 8)
      w[kv] = *reinterpret_cast<const uint32_t*>(src);
    else
      w[kv] = *reinterpret_cast<const uint16_t*>(src);
    s2[kv] = base[(kv ? blk.v_scale : blk.k_scale) + row * (D / kKvGroup) + ch / kKvGroup];
  }
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    const uint32_t s = f16_low_twice(e4m3x2_to_f16(s2[kv]));
    uint32_t p[4];
    e2m1_to_f16(w[kv], p);
    float x[V];
#pragma unroll
    for (int j = 0; j < V / 2; ++j) {
      const uint32_t q = hmul2(p[j], s);
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&q));
      x[2 * j] = ok ? f.x * (kv ? v_scale : k_scale) : 0.0f;
      x[2 * j + 1] = ok ? f.y * (kv ? v_scale : k_scale) : 0.0f;
    }
    store_chunk((kv ? v_out : k_out) + at, x);
  }
}

bool rows_aligned(const Rows& r, int eb) {
  return (reinterpret_cast<uintptr_t>(r.p) | static_cast<uintptr_t>(r.token * eb) |
          static_cast<uintptr_t>(r.head * eb)) % 16 == 0;
}

template <typename T>
cudaError_t launch_rope_t(const RopeArgs& a, cudaStream_t st) {
  const int eb = sizeof(T);
  const bool rows16 = a.D % kKvGroup == 0 &&
                      (a.q_heads == 0 || (rows_aligned(a.q, eb) &&
                                          reinterpret_cast<uintptr_t>(a.q_out) % 16 == 0)) &&
                      (a.kv_heads == 0 || (rows_aligned(a.k, eb) && rows_aligned(a.v, eb)));
  const bool fast = rows16 && a.D % 32 == 0 && a.R % 32 == 0 &&
                    reinterpret_cast<uintptr_t>(a.table) % 16 == 0;
  // (8192 tokens, 40 heads of 128 in bf16: 29.8 us fast; wide 58.8 us for 66 of the
  // channels in halves and 39.3 us for 98 interleaved; one element at a time
  // 124 and 131 us)
  const int lanes = a.D / (16 / eb);
  const bool wide = rows16 && !fast && (a.q.p != a.q_out || 32 % lanes == 0);
  const long units = fast ? lanes / 2 : wide ? lanes : (a.D + 15) / 16;
  // Heads per thread, one or four: a table row serves all of them. Queries alone
  // (32 heads of 128 in bf16): 256 tokens 2.2 us with one and 2.6 with four, 512
  // tokens 2.8 and 2.7, 4096 tokens 18.3 and 14.4. Keys and values are quantised
  // one head after the other (8 of each beside them): 64 tokens 4.9 and 7.1 us,
  // 1024 tokens 10.0 and 11.1, 2048 tokens 17.7 and 15.5.
  const long all = units * a.T * (a.q_heads + 2l * a.kv_heads);
  const int hb = all / 4 >= static_cast<long>(kSms) * (a.kv_heads ? 1024 : 192) ? 4 : 1;
  const int cq = (a.q_heads + hb - 1) / hb, ck = (a.kv_heads + hb - 1) / hb;
  const long total = units * a.T * (cq + 2l * ck);
  if (total == 0) return cudaSuccess;
  if (total > 0xffffff00l) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>((total + kThreads - 1) / kThreads)), block(kThreads);
  const unsigned n = static_cast<unsigned>(total);
  if (wide) {
    auto* kern = a.interleaved
                     ? (hb == 1 ? &rope_wide_kernel<T, true, 1> : &rope_wide_kernel<T, true, 4>)
                     : (hb == 1 ? &rope_wide_kernel<T, false, 1> : &rope_wide_kernel<T, false, 4>);
    return launch_pdl(kern, grid, block, 0, st, a, cq, ck, n);
  }
  if (!fast) return launch_pdl(&rope_any_kernel<T>, grid, block, 0, st, a, hb, cq, ck, n);
  auto* kern = a.interleaved ? (hb == 1 ? &rope_kernel<T, true, 1> : &rope_kernel<T, true, 4>)
                             : (hb == 1 ? &rope_kernel<T, false, 1> : &rope_kernel<T, false, 4>);
  return launch_pdl(kern, grid, block, 0, st, a, cq, ck, n);
}

}  // namespace

cudaError_t launch_rope(bool bf16, const RopeArgs& a, cudaStream_t st) {
  return bf16 ? launch_rope_t<__nv_bfloat16>(a, st) : launch_rope_t<float>(a, st);
}

cudaError_t launch_rope_table(const RopeTurns& turns, int pairs, float gain, int n,
                              const int32_t* positions, float* table, cudaStream_t st) {
  // enough rows per block to use each thread's frequency several times, few
  // enough to give every SM work
  const int lanes = kThreads / pairs;
  int rows = n / (kSms * 16);
  rows = (rows < lanes ? lanes : rows + lanes - 1) / lanes * lanes;
  return launch_pdl(&rope_table_kernel, dim3((n + rows - 1) / rows), dim3(kThreads), 0, st, turns,
                    pairs, gain, n, positions, table, rows);
}

cudaError_t launch_kv_read(bool bf16, int N, const int64_t* slots, const uint8_t* cache,
                           long n_slots, int kv_heads, int D, int page_shift, float k_scale,
                           float v_scale, void* k_out, void* v_out, unsigned* status,
                           cudaStream_t st) {
  const long total = static_cast<long>(N) * kv_heads * (D / (bf16 ? 8 : 4));
  if (total > 0xffffff00l) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>((total + kThreads - 1) / kThreads));
  if (bf16)
    return launch_pdl(&kv_read_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, st, N, slots,
                      cache, n_slots, kv_heads, D, page_shift, k_scale, v_scale,
                      static_cast<__nv_bfloat16*>(k_out), static_cast<__nv_bfloat16*>(v_out),
                      status);
  return launch_pdl(&kv_read_kernel<float>, grid, dim3(kThreads), 0, st, N, slots, cache, n_slots,
                    kv_heads, D, page_shift, k_scale, v_scale, static_cast<float*>(k_out),
                    static_cast<float*>(v_out), status);
}

}  // namespace moe
