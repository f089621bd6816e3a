// The 4-bit cache format (include/moe.h) and its conversions.
//
// e2m1 codes and e4m3 scales are the 4- and 8-bit floats that sm_103a converts
// in hardware. Their product has at most 2 + 4 significant bits and lies in
// 2^-10 .. 2688, so it is exact in f16: a stored element enters a matrix
// instruction without any rounding.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstddef>
#include <cstdint>

namespace moe {

constexpr int kKvGroup = 16;  // channels per scale

// Byte offsets inside one (page, kv head) block.
struct KvBlock {
  uint32_t k_scale, v_code, v_scale, bytes;
};
__host__ __device__ constexpr KvBlock kv_block(int page_size, int D) {
  const uint32_t codes = static_cast<uint32_t>(page_size) * D / 2;
  const uint32_t scales = static_cast<uint32_t>(page_size) * D / kKvGroup;
  return {codes, codes + scales, 2 * codes + scales, 2 * (codes + scales)};
}

// Two floats -> two e2m1 codes, nearest even, saturating; `lo` in the low half.
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 b;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\t"
      "cvt.u32.u8 %0, b;\n\t}"
      : "=r"(r)
      : "f"(hi), "f"(lo));
  return r;
}

// One float -> e4m3, nearest even, saturating at 448.
__device__ __forceinline__ uint32_t e4m3(float x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(x));
  return r & 0xffu;
}

// Eight codes (one word) -> eight f16 values, two by two in channel order.
__device__ __forceinline__ void e2m1_to_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// Two e4m3 scales -> f16x2 (first scale in the low half).
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t two) {
  uint32_t r;
  const uint16_t h = static_cast<uint16_t>(two);
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(h));
  return r;
}
__device__ __forceinline__ uint32_t f16_low_twice(uint32_t h) { return __byte_perm(h, 0, 0x1010); }
__device__ __forceinline__ uint32_t f16_high_twice(uint32_t h) { return __byte_perm(h, 0, 0x3232); }

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Values are cut off here before they are stored: beyond 6 * 448, the largest
// value that a code and a scale can hold, and infinities become finite.
constexpr float kKvMost = 4096.0f;

// V of the 16 scaled values of a group (NaN already replaced, cut off at
// kKvMost) whose largest magnitude is `top` -> codes, eight to a word, and the
// scale byte. The quotients have to be rounded correctly: for 16-bit inputs many
// lie exactly between two codes. They are made from the correctly rounded
// reciprocal, the product with it and one correction by the exact remainder
// (Markstein, 1990), three operations where a division takes some fifteen;
// the scale is between 2^-9 and 448, so nothing leaves the normal range that
// would not round to the code 0.
template <int V>
__device__ __forceinline__ uint32_t kv_codes(const float (&y)[V], float top,
                                             uint32_t (&codes)[(V + 7) / 8]) {
  const uint32_t s8 = e4m3(__fmul_rn(top, 1.0f / 6.0f));
  const float s = __half2float(__ushort_as_half(static_cast<uint16_t>(e4m3x2_to_f16(s8) & 0xffffu)));
  const float r = s > 0.0f ? __frcp_rn(s) : 0.0f;
#pragma unroll
  for (int i = 0; i < (V + 7) / 8; ++i) codes[i] = 0;
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    float q[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float p = __fmul_rn(y[2 * i + j], r);
      q[j] = __fmaf_rn(__fmaf_rn(-p, s, y[2 * i + j]), r, p);
    }
    codes[i >> 2] |= e2m1x2(q[0], q[1]) << (8 * (i & 3));
  }
  return s8;
}

}  // namespace moe
