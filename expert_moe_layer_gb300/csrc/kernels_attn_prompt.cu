// Attention over the 4-bit paged cache: the prompt kernel (bf16).
//
// Many query tokens share a request's keys, so matrix work bounds this kernel:
// 4 D operations per (row, key) on the tcgen05 tensor cores, and one
// exponential. A unit is 256 rows of one (request, kv head); a row is one
// (query token, head of the group) pair, so that a group's heads share every
// dequantised key. Per 128 keys:
//   - four warps turn codes and scales into f16 (exactly) in shared memory, K
//     as rows of channels, V transposed to rows of tokens, both in the 128-byte
//     swizzle that the matrix unit reads, two stages deep;
//   - one thread issues S = Q K^T and O += P V for the two halves of 128 rows
//     in turn, S and O in tensor memory, P read from tensor memory in the place
//     of the S it came from;
//   - four warps per half take S (a thread holds a whole row: no shuffles),
//     mask, exponentiate and write P, one half while the other's products run.
// The running maximum may lag behind (kLag): a tile is exponentiated on the
// old one in a single pass over S, and done again, with O rescaled, in the
// rare case that a row's maximum has outgrown it. Units are drawn from a
// counter, a request's longest rows first.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>

#include "attn_dev.cuh"
#include "internal.h"
#include "launch.cuh"
#include "ptx.cuh"

namespace moe {

MOE_WAIT_LIMIT_SETTER(set_wait_limit_attn)

namespace {

constexpr int kHalf = 128;                    // rows of a half, lanes of tensor memory
constexpr int kKeys = 128;                    // keys per tile
constexpr int kSoftWarps = 8, kFillWarps = 4;
constexpr int kMmaWarp = kSoftWarps + kFillWarps;
constexpr int kWarpsAll = kMmaWarp + 1;       // warps with a role
constexpr int kThreads = 512;                 // whole groups of four warps (three idle ones)
// Registers per thread: launched with 128 each (65,536 in all); the matrix
// warp's group gives most of its share to the two softmax groups:
// 128 * (2 * 152 + 128 + 80) = 65,536.
constexpr int kSoftRegs = 152, kMmaRegs = 80;
constexpr int kBadRing = 4;  // tiles whose bad-page bits are kept: a fill warp is at most
                             // two tiles ahead of the slower half
constexpr float kMostP = 16384.0f;  // 2^(kLift + kLag)
constexpr uint32_t kColsS = 0, kColsO = 256;  // columns of S (128 each half) and of O

template <int D>
struct Smem {
  static constexpr int kQ = kHalf * D * 2;   // one half's queries
  static constexpr int kK = kKeys * D * 2;   // one stage of keys, or of values
  static constexpr int kBytes = 2 * kQ + 4 * kK + 1024;
};

struct Bars {
  uint64_t unit_full[2], unit_empty[2], q_ready[2], k_full[2], k_empty[2], v_full[2], v_empty[2],
      s_full[2], p_ready[2], o_done[2], drain;
};

// 32 consecutive columns of this warp's 32 lanes.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,"
      "%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,"
      "%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
      "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// D[tmem] (+)= A[tmem] * B[smem]^T (f16).
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Two fp32 values in a 64-bit register, and the instructions on both at once.
__device__ __forceinline__ uint64_t pair_b32(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ uint64_t pair_f32(float lo, float hi) {
  return pair_b32(__float_as_uint(lo), __float_as_uint(hi));
}
__device__ __forceinline__ void unpair_f32(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                       uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// Byte offset of 16-byte chunk `chunk` of row `row` in a 128-byte-swizzled
// operand whose panels (64 f16 wide) hold `rows` rows.
__device__ __forceinline__ uint32_t swizzled(int row, int chunk, int rows) {
  return (chunk >> 3) * rows * 128 + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
}

// What every role derives from a unit number.
struct Unit {
  int b, kvh, row0, rows, halves;  // rows: of the request
  int lo, hi, tiles;               // keys [lo, hi) are seen by some row; tiles from lo / kKeys
  SeqInfo sq;
};
__device__ __forceinline__ Unit unit_of(const AttnArgs& a, long u, const SeqInfo* info,
                                        const long* starts) {
  int lo = 0, hi = a.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (starts[mid] <= u) lo = mid;
    else hi = mid;
  }
  Unit r;
  r.b = lo;
  r.sq = info[lo];
  const int group = a.heads / a.kv_heads;
  r.rows = r.sq.q_len * group;
  const long local = u - starts[lo];
  const int row_tiles = (r.rows + kPromptTile - 1) / kPromptTile;
  r.kvh = static_cast<int>(local % a.kv_heads);
  r.row0 = (row_tiles - 1 - static_cast<int>(local / a.kv_heads)) * kPromptTile;
  const int last = min(r.rows, r.row0 + kPromptTile) - 1;
  r.halves = last >= r.row0 + kHalf ? 2 : 1;
  const int before = r.sq.len - r.sq.q_len;
  const int p0 = before + r.row0 / group, p1 = before + last / group;
  r.lo = a.window > 0 ? max(0, p0 - a.window + 1) : 0;
  r.hi = p1 + 1;
  r.tiles = r.hi <= 0 ? 0 : (r.hi + kKeys - 1) / kKeys - r.lo / kKeys;
  return r;
}

template <int D>
struct RawTile {
  Words<D / 8> k;   // one key row
  uint32_t ks[D / 64];
  uint2 v[8];       // 16 channels of eight value rows
  uint32_t vs[2];   // and their scales
  uint32_t bad;     // key rows of this warp on a bad page
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_prompt_kernel(AttnArgs a, unsigned* status, const SeqInfo* info, const long* starts,
                       int* ticket) {
  using S = Smem<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Bars bars;
  __shared__ int s_units[2];
  __shared__ __align__(16) uint32_t s_bad[kBadRing][4];
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  const uint32_t base = (ptx::smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sm_q = base, sm_k = base + 2 * S::kQ, sm_v = sm_k + 2 * S::kK;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto bar = [&](const uint64_t& b) { return ptx::smem_u32(&b); };

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(bar(bars.unit_full[i]), 1);
      ptx::mbar_init(bar(bars.unit_empty[i]), kWarpsAll);
      ptx::mbar_init(bar(bars.q_ready[i]), 4);
      ptx::mbar_init(bar(bars.k_full[i]), kFillWarps);
      ptx::mbar_init(bar(bars.k_empty[i]), 1);
      ptx::mbar_init(bar(bars.v_full[i]), kFillWarps);
      ptx::mbar_init(bar(bars.v_empty[i]), 1);
      ptx::mbar_init(bar(bars.s_full[i]), 1);
      ptx::mbar_init(bar(bars.p_ready[i]), 4);
      ptx::mbar_init(bar(bars.o_done[i]), 1);
    }
    ptx::mbar_init(bar(bars.drain), 1);
    ptx::fence_barrier_init();
    s_abort = 0;
  }
  if (warp == kMmaWarp) {
    ptx::tmem_alloc(ptx::smem_u32(&s_tmem), 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = s_tmem;
  pdl_enter();
  const long total = starts[a.B];
  const int group = a.heads / a.kv_heads;
  auto wait = [&](const uint64_t& b, uint32_t parity) {
    return ptx::mbar_wait(bar(b), parity, &s_abort, status);
  };
  // The same for a whole warp: all lanes go on or none (a timeout may reach
  // some lanes only, and tensor memory is read by whole warps).
  auto wait_warp = [&](const uint64_t& b, uint32_t parity) {
    return __all_sync(~0u, wait(b, parity)) != 0;
  };
  // The next unit of the ring for a warp of any role (-1: none, or a timeout).
  uint32_t turn = 0;
  auto next_unit = [&]() -> long {
    const uint32_t slot = turn & 1, parity = (turn >> 1) & 1;
    ++turn;
    if (!wait_warp(bars.unit_full[slot], parity)) return -1;
    const int u = *reinterpret_cast<volatile int*>(&s_units[slot]);
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(bar(bars.unit_empty[slot]));
    return u;
  };

  if (warp < kSoftWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    // ---------------------------------------------------------------- softmax
    const int x = warp >> 2;
    const int row_l = (warp & 3) * 32 + lane;  // row of the half, lane of tensor memory
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;
    const uint32_t ts = tmem + lanes + kColsS + x * kHalf, to = tmem + lanes + kColsO + x * D;
    uint32_t s_phase = 0, o_phase = 0, tile_no = 0;
    for (;;) {
      const long u = next_unit();
      if (u < 0) break;
      const Unit t = unit_of(a, u, info, starts);
      const int r = t.row0 + x * kHalf + row_l;
      const bool live = r < t.rows;
      const int tok = r / group, head = t.kvh * group + (r - tok * group);
      if (x < t.halves && t.tiles > 0) {
        // this row's queries, scaled to f16
        const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.q.p) +
                                   (t.sq.q0 + (live ? tok : 0)) * a.q.token +
                                   (live ? head : 0) * a.q.head;
        uint4 w[D / 8];
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          w[i] = live ? reinterpret_cast<const uint4*>(src)[i] : make_uint4(0, 0, 0, 0);
          const uint32_t v[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            top = fmaxf(top, fmaxf(fabsf(__uint_as_float(v[j] << 16)),
                                   fabsf(__uint_as_float(v[j] & 0xffff0000u))));
        }
        float up, down;
        row_power(top, up, down);
        const float gain = down * a.scale_log2;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          const uint32_t v[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
          uint32_t h[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            h[j] = pack_f16(__uint_as_float(v[j] << 16) * up,
                            __uint_as_float(v[j] & 0xffff0000u) * up);
          sts128(sm_q + x * S::kQ + swizzled(row_l, i, kHalf), h[0], h[1], h[2], h[3]);
        }
        ptx::fence_proxy_async();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(bars.q_ready[x]));

        const int p = t.sq.len - t.sq.q_len + tok;
        const int last = live ? p : 0x7fffffff;
        const int first = live && a.window > 0 ? p - a.window + 1 : 0;
        // keys that every row of the half sees
        const int r_lo = t.row0 + x * kHalf, r_hi = min(t.rows, r_lo + kHalf) - 1;
        const int all_last = t.sq.len - t.sq.q_len + r_lo / group;
        const int all_first =
            a.window > 0 ? t.sq.len - t.sq.q_len + r_hi / group - a.window + 1 : 0;
        float m = -INFINITY, mbase = -kLift, l = 0.0f;
        bool ok = true;
        for (int j = 0; j < t.tiles; ++j, ++tile_no) {
          if (!(ok = wait_warp(bars.s_full[x], s_phase))) break;
          s_phase ^= 1;
          ptx::tc_fence_after();
          const int tok0 = (t.lo / kKeys + j) * kKeys;
          const uint4 bad = lds128(ptx::smem_u32(s_bad[tile_no % kBadRing]));
          const bool whole = tok0 >= all_first && tok0 + kKeys - 1 <= all_last &&
                             (bad.x | bad.y | bad.z | bad.w) == 0;
          uint32_t pk[kKeys / 2];
          float sum;
          bool over;  // a P has outgrown the lag allowed to the maximum
          auto visible = [&](int c, uint32_t(&v)[32]) {
            const uint32_t bits = c == 0 ? bad.x : c == 1 ? bad.y : c == 2 ? bad.z : bad.w;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const int key = tok0 + 32 * c + i;
              if (key < first || key > last || ((bits >> i) & 1u)) v[i] = 0xff800000u;
            }
          };
          auto pass = [&](bool masked) {
            const uint64_t gain2 = pair_f32(gain, gain), off2 = pair_f32(-mbase, -mbase);
            uint64_t sums[2] = {0, 0};
            uint32_t top = 0;
#pragma unroll
            for (int c = 0; c < kKeys / 32; ++c) {
              uint32_t v[32];
              tmem_ld32(ts + 32 * c, v);
              if (masked) visible(c, v);
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                float x0, x1;
                unpair_f32(fma_f32x2(pair_b32(v[2 * i], v[2 * i + 1]), gain2, off2), x0, x1);
                const float p0 = ex2(x0), p1 = ex2(x1);
                sums[i & 1] = add_f32x2(sums[i & 1], pair_f32(p0, p1));
                pk[16 * c + i] = pack_f16(p0, p1);
                top = max_f16x2(top, pk[16 * c + i]);
              }
            }
            float s0, s1;
            unpair_f32(add_f32x2(sums[0], sums[1]), s0, s1);
            sum = s0 + s1;
            const float2 t2 = unpack_f16(top);
            over = fmaxf(t2.x, t2.y) > kMostP;
          };
          if (whole) pass(false);
          else pass(true);
          if (__any_sync(~0u, over || m == -INFINITY)) {
            float mx = -INFINITY;
#pragma unroll 1
            for (int c = 0; c < kKeys / 32; ++c) {
              uint32_t v[32];
              tmem_ld32(ts + 32 * c, v);
              if (!whole) visible(c, v);
#pragma unroll
              for (int i = 0; i < 32; ++i) mx = fmaxf(mx, __uint_as_float(v[i]));
            }
            const float nm = fmaxf(m, mx * gain);
            const float nb = nm == -INFINITY ? -kLift : nm - kLift;
            const float f = m == -INFINITY ? 0.0f : ex2(mbase - nb);
            l *= f;
            m = nm;
            mbase = nb;
            if (j > 0) {  // the products of the tiles before have all landed (s_full)
#pragma unroll
              for (int c = 0; c < D / 32; ++c) {
                uint32_t v[32];
                tmem_ld32(to + 32 * c, v);
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f);
                tmem_st32(to + 32 * c, v);
              }
            }
            if (whole) pass(false);
            else pass(true);
          }
          l += sum;
#pragma unroll
          for (int c = 0; c < kKeys / 64; ++c) tmem_st32(ts + 32 * c, pk + 32 * c);
          tmem_wait_st();
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(bar(bars.p_ready[x]));
        }
        if (!ok || !wait_warp(bars.o_done[x], o_phase)) break;
        o_phase ^= 1;
        ptx::tc_fence_after();
        const float f = out_factor(l, a.v_scale);
        const long at_row = static_cast<long>(t.sq.q0 + tok) * a.heads + head;
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) + at_row * D;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t v[32];
          tmem_ld32(to + 32 * c, v);
          if (live) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t h[4];
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const __nv_bfloat162 b2 =
                    __floats2bfloat162_rn(__uint_as_float(v[8 * i + 2 * q]) * f,
                                          __uint_as_float(v[8 * i + 2 * q + 1]) * f);
                h[q] = *reinterpret_cast<const uint32_t*>(&b2);
              }
              *reinterpret_cast<uint4*>(dst + 32 * c + 8 * i) = make_uint4(h[0], h[1], h[2], h[3]);
            }
          }
        }
        if (live && a.lse) a.lse[at_row] = log_sum(mbase, l);
        ptx::tc_fence_before();
      } else if (x < t.halves) {
        // no row of the unit sees a key
        if (live) {
          const long at_row = static_cast<long>(t.sq.q0 + tok) * a.heads + head;
          uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + at_row * D);
#pragma unroll
          for (int i = 0; i < D / 8; ++i) dst[i] = make_uint4(0, 0, 0, 0);
          if (a.lse) a.lse[at_row] = -INFINITY;
        }
      } else {
        tile_no += t.tiles;
      }
    }
  } else if (warp < kMmaWarp) {
    // ------------------------------------------------- codes to f16 operands
    const int ft = threadIdx.x - kSoftWarps * 32;   // 0..127: key row of the tile
    const int fw = warp - kSoftWarps;
    // values: eight tokens from vt, 16 channels from vc (D = 64: half the threads)
    const int vt = ((lane & 7) + 8 * (fw & 1)) * 8, vg = (lane >> 3) + 4 * (fw >> 1);
    const bool has_v = vg < D / kKvGroup;
    const KvBlock blk = kv_block(a.page_size, D);
    const int page_mask = a.page_size - 1, page_shift = 31 - __clz(a.page_size);
    uint32_t kc = 0, produced = 0;
    for (;;) {
      if (fw == 0 && lane == 0) {  // draw a unit for everybody
        const uint32_t slot = produced & 1;
        if (wait(bars.unit_empty[slot], ((produced >> 1) & 1) ^ 1)) {
          const long u = atomicAdd(ticket, 1);
          *reinterpret_cast<volatile int*>(&s_units[slot]) = u < total ? static_cast<int>(u) : -1;
        } else {
          *reinterpret_cast<volatile int*>(&s_units[slot]) = -1;
        }
        ptx::mbar_arrive(bar(bars.unit_full[slot]));
        ++produced;
      }
      __syncwarp();
      const long u = next_unit();
      if (u < 0) break;
      const Unit t = unit_of(a, u, info, starts);
      const int32_t* pages = a.page_table + static_cast<long>(t.b) * a.max_pages;
      RawTile<D> raw;
      auto fetch = [&](int j) {
        const int tok0 = (t.lo / kKeys + j) * kKeys;
        // the block of keys key .. key + more, of which some row sees one
        auto block_of = [&](int key, int more, bool& ok) -> const uint8_t* {
          const int id = key < t.hi && key + more >= t.lo ? pages[key >> page_shift] : 0;
          ok = id >= 0 && id < a.num_pages;
          return a.cache + (static_cast<long>(ok ? id : 0) * a.kv_heads + t.kvh) * blk.bytes;
        };
        bool ok;
        const uint8_t* p = block_of(tok0 + ft, 0, ok);
        const int kr = (tok0 + ft) & page_mask;
        raw.k = load_words<D / 8>(p + kr * (D / 2));
#pragma unroll
        for (int i = 0; i < D / 64; ++i)
          raw.ks[i] = *reinterpret_cast<const uint32_t*>(p + blk.k_scale + kr * (D / 16) + 4 * i);
        raw.bad = __ballot_sync(~0u, !ok);
        if (has_v) {
          p = block_of(tok0 + vt, 7, ok);
          const int vr = (tok0 + vt) & page_mask;
          raw.vs[0] = raw.vs[1] = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            raw.v[i] = *reinterpret_cast<const uint2*>(p + blk.v_code + (vr + i) * (D / 2) + vg * 8);
            // a key that no row sees may be uninitialised memory: a zero scale
            // keeps 0 * NaN out of the sum
            const int key = tok0 + vt + i;
            const uint32_t s = p[blk.v_scale + (vr + i) * (D / 16) + vg];
            raw.vs[i >> 2] |= (ok && key >= t.lo && key < t.hi ? s : 0u) << (8 * (i & 3));
          }
        }
      };
      if (t.tiles > 0) fetch(0);
      bool ok = true;
      for (int j = 0; j < t.tiles; ++j, ++kc) {
        const uint32_t st = kc & 1, parity = ((kc >> 1) & 1) ^ 1;
        if (!(ok = wait_warp(bars.k_empty[st], parity))) break;
        if (raw.bad && lane == 0) atomicOr(status, MOE_DEV_BAD_PAGE);
        if (lane == 0) *reinterpret_cast<volatile uint32_t*>(&s_bad[kc % kBadRing][fw]) = raw.bad;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          uint32_t h[4];
          e2m1_to_f16(raw.k.w[c], h);
          const uint32_t two = e4m3x2_to_f16(raw.ks[c / 8] >> (16 * ((c / 4) & 1)));
          const uint32_t s = (c / 2) & 1 ? f16_high_twice(two) : f16_low_twice(two);
          sts128(sm_k + st * S::kK + swizzled(ft, c, kKeys), hmul2(h[0], s), hmul2(h[1], s),
                 hmul2(h[2], s), hmul2(h[3], s));
        }
        ptx::fence_proxy_async();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(bars.k_full[st]));
        if (!(ok = wait_warp(bars.v_empty[st], parity))) break;
        if (has_v) {
          uint32_t s[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) s[i] = e4m3x2_to_f16(raw.vs[i >> 1] >> (16 * (i & 1)));
#pragma unroll
          for (int w = 0; w < 2; ++w) {  // eight channels
            uint32_t h[8][4];
#pragma unroll
            for (int i = 0; i < 8; ++i) e2m1_to_f16(w ? raw.v[i].y : raw.v[i].x, h[i]);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int ch = vg * 16 + w * 8 + 2 * q;
#pragma unroll
              for (int o = 0; o < 2; ++o) {
                uint32_t d[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  d[i] = hmul2(__byte_perm(h[2 * i][q], h[2 * i + 1][q], o ? 0x7632 : 0x5410), s[i]);
                sts128(sm_v + st * S::kK + swizzled(ch + o, vt / 8, D), d[0], d[1], d[2], d[3]);
              }
            }
          }
        }
        ptx::fence_proxy_async();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(bars.v_full[st]));
        if (j + 1 < t.tiles) fetch(j + 1);
      }
      if (!ok) break;
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kMmaRegs));
  }
  if (warp == kMmaWarp) {
    // ------------------------------------------------------ the matrix thread
    uint32_t kc = 0, q_phase[2] = {0, 0}, p_phase[2] = {0, 0};
    const uint32_t id_s = ptx::idesc_make(0, kHalf, kKeys), id_o = ptx::idesc_make(0, kHalf, D);
    for (;;) {
      const long u = next_unit();
      if (u < 0) break;
      const Unit t = unit_of(a, u, info, starts);
      bool ok = true;
      if (lane == 0 && t.tiles > 0) {
        auto scores = [&](int x, uint32_t st) {
#pragma unroll
          for (int pnl = 0; pnl < D / 64; ++pnl) {
            const uint64_t da = ptx::sdesc_sw128(sm_q + x * S::kQ + pnl * kHalf * 128);
            const uint64_t db = ptx::sdesc_sw128(sm_k + st * S::kK + pnl * kKeys * 128);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              ptx::tc_mma<false>(tmem + kColsS + x * kHalf, da + 2 * kk, db + 2 * kk, id_s,
                                 pnl + kk > 0);
          }
          ptx::tc_commit(bar(bars.s_full[x]));
        };
        auto sums = [&](int x, uint32_t st, bool more) {
#pragma unroll
          for (int pnl = 0; pnl < kKeys / 64; ++pnl) {
            const uint64_t db = ptx::sdesc_sw128(sm_v + st * S::kK + pnl * D * 128);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_ts(tmem + kColsO + x * D, tmem + kColsS + x * kHalf + pnl * 32 + kk * 8,
                     db + 2 * kk, id_o, more || pnl + kk > 0);
          }
        };
        for (int x = 0; ok && x < t.halves; ++x) {
          ok = wait(bars.q_ready[x], q_phase[x]);
          q_phase[x] ^= 1;
        }
        ok = ok && wait(bars.k_full[kc & 1], (kc >> 1) & 1);
        if (ok) {
          ptx::tc_fence_after();
          for (int x = 0; x < t.halves; ++x) scores(x, kc & 1);
          ptx::tc_commit(bar(bars.k_empty[kc & 1]));
        }
        for (int j = 0; ok && j < t.tiles; ++j, ++kc) {
          const bool again = j + 1 < t.tiles;
          const uint32_t st = kc & 1, nst = (kc + 1) & 1;
          ok = wait(bars.v_full[st], (kc >> 1) & 1);
          for (int x = 0; ok && x < t.halves; ++x) {
            if (!(ok = wait(bars.p_ready[x], p_phase[x]))) break;
            p_phase[x] ^= 1;
            ptx::tc_fence_after();
            sums(x, st, j > 0);
            if (x == t.halves - 1) ptx::tc_commit(bar(bars.v_empty[st]));
            if (again) {
              // S takes the place of the P that the products before it read:
              // matrix instructions of one thread run in the order of issue
              if (x == 0 && !(ok = wait(bars.k_full[nst], ((kc + 1) >> 1) & 1))) break;
              scores(x, nst);
              if (x == t.halves - 1) ptx::tc_commit(bar(bars.k_empty[nst]));
            } else {
              ptx::tc_commit(bar(bars.o_done[x]));
            }
          }
        }
      }
      if (!__shfl_sync(~0u, static_cast<int>(ok), 0)) break;
    }
    // whatever was issued has to land before the tensor memory is given back
    if (lane == 0) {
      ptx::tc_commit(bar(bars.drain));
      ptx::mbar_wait_drain(bar(bars.drain), 0);
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == kMmaWarp) ptx::tmem_dealloc(tmem, 512);
}

template <int D>
cudaError_t launch_dim(const AttnArgs& a, void* ws, const AttnLayout& L, cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = opt_in_smem(reinterpret_cast<const void*>(&attn_prompt_kernel<D>),
                              Smem<D>::kBytes, done);
  if (e != cudaSuccess) return e;
  char* w = static_cast<char*>(ws);
  return launch_pdl(&attn_prompt_kernel<D>, dim3(a.sms), dim3(kThreads), Smem<D>::kBytes, st, a,
                    reinterpret_cast<unsigned*>(w + L.status),
                    reinterpret_cast<const SeqInfo*>(w + L.info),
                    reinterpret_cast<const long*>(w + L.starts),
                    reinterpret_cast<int*>(w + L.counters));
}

}  // namespace

cudaError_t launch_prompt(const AttnArgs& a, void* ws, const AttnLayout& L, cudaStream_t st) {
  return a.D == 64 ? launch_dim<64>(a, ws, L, st) : launch_dim<128>(a, ws, L, st);
}

}  // namespace moe
