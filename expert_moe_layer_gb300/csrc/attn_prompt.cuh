// Attention over the 4-bit paged cache: the prompt kernel (bf16).
//
// Many query tokens share a request's keys, so matrix work bounds this kernel:
// 4 D operations per (row, key) on the tcgen05 tensor cores, and one
// exponential. A row is one (query token, head of the group) pair, so that a
// group's heads share every dequantised key; a row tile is one or two halves of
// 128 rows. Per tile of 128 keys (64 with 256 channels):
//   - four warps turn codes and scales into f16 (exactly) in shared memory, K
//     as rows of channels, V transposed to rows of tokens, both in the 128-byte
//     swizzle that the matrix unit reads, two stages deep;
//   - one elected lane of a converged warp issues S = Q K^T and O += P V for the
//     halves in turn, S and O in tensor memory, P read from tensor memory in the
//     place of the S it came from;
//   - four warps per half take S (a thread holds a row: no shuffles), mask,
//     exponentiate and write P, one half while the other's products run.
// The running maximum may lag behind (kLag), so that a pass over S needs no
// maximum beforehand; in the rare case that a row has outgrown it, the maximum
// moves up by whole powers of two, and O, the sums and the tile's earlier P are
// scaled down exactly.
//
// The tiles of all (row tile, kv head) segments form one list, cut into equal
// ranges, one per CTA, as in the split kernel: causal lengths differ, and a
// short chunk after a long context has few row tiles. Pieces of a segment leave
// fp32 sums, and the last CTA joins them in CTA order.
//
// Measured: four chunks of 2048 queries that end at 2 to 16 thousand tokens, 32
// query and 8 kv heads of 128, 743 us: 1.1 PFLOP/s, 57 % of the measured matrix
// rate. A tile takes about 4700 cycles of an SM, its matrix instructions 2500;
// the fill warps work 4300 of them and a half's chain of S, softmax and P V
// takes 4000, so both would have to become shorter at once.
//
// Over prefixes (kPrefix) the requests of a group are the rows, every row sees
// every key, and a fifth kind of warp copies: whole parts, the codes and scales of a
// tile's keys or of its values, by bulk copies into a ring of three. The fill warps
// then only convert: keys with their chunks in an order of the lane's own, values
// through transposing matrix stores, no bank conflicts in either; both take 1900
// cycles of a tile. A tile of 256 rows takes 3900 cycles (4300 with the fill warps' own
// copies): softmax 2300 and 1600 of waiting for S. The matrix unit and the fill warps
// share the SM's shared memory, 2300 cycles of a tile at 128 bytes each, so that
// products in smaller steps lose: the next tile's first 64 scores ahead of P V took
// 4500 cycles, P V in two halves 4100. Of row tiles with no more than 128 rows both
// halves take the same rows and every other key tile: 2900 cycles, where one half
// alone takes 3900, and then the fill warps are the bound.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <type_traits>

#include "attn_dev.cuh"
#include "attn_groups.cuh"
#include "internal.h"
#include "launch.cuh"
#include "ptx.cuh"

namespace moe {
namespace {
namespace prompt {

constexpr int kHalf = 128;  // rows of a half, lanes of tensor memory
constexpr int kSoftWarps = 8, kFillWarps = 4;
constexpr int kStageBytes = 32 * 32;  // a softmax warp's staging rows on the way out
constexpr int kMmaWarp = kSoftWarps + kFillWarps;
constexpr int kThreads = 512;  // whole groups of four warps (three idle ones)
// Registers per thread: launched with 128 each (65,536 in all), shared out anew
// by the groups of four warps: 128 * (2 * 184 + 80 + 64) = 65,536.
constexpr int kSoftRegs = 184, kFillRegs = 80, kMmaRegs = 64;
// Over prefixes: parts (a tile's keys, or its values) in shared memory or on the
// way, and tiles whose bad-page bits are kept (one and a half of those are ahead of
// the fill warps).
constexpr int kParts = 3, kPrefixBadRing = 8;
constexpr int kBadRing = 4;  // tiles whose bad-page bits are kept: a fill warp is at most
                             // two tiles ahead of the slower half
// List entries of a segment beside its tiles: its set-up and store. (The chunks
// above take 760, 743 and 771 us with 2, 4 and 8.)
constexpr int kSetup = 4;
// Smallest range of a CTA: 64 queries after 32768 tokens take 79 us with 16
// tiles and 77 with 8, 8 prompts of 512 tokens 58 and 58 (32 tiles: 111 and 82).
constexpr int kMinTiles = 16;
// A cut this near to a segment's begin or end moves there: a piece's way
// through the workspace and the join take longer than so few tiles. Chunks of
// 1000 queries that end at 1000 to 3000 tokens: 102 us, and 117 with 8, 122 with
// 12. A piece has a tile beside its kSetup entries.
constexpr int kSnap = 4;
static_assert(kSnap >= kSetup && kSnap < kMinTiles, "pieces have tiles, cuts do not cross");
constexpr int kPlanThreads = 1024;
constexpr float kMostP = 16384.0f;              // 2^(kLift + kLag)
constexpr uint32_t kColsS = 0, kColsO = 256;  // columns of S and of O

template <int D>
struct Shape {
  static constexpr int kTile = prompt_tile(D);      // rows of a row tile
  static constexpr int kHalves = kTile / kHalf;
  static constexpr int kKeys = D == 256 ? 64 : 128;  // keys per tile
  static constexpr int kQ = kHalf * D * 2;          // bytes of one half's queries
  static constexpr int kK = kKeys * D * 2;          // of one stage of keys, or of values
  // Codes and scales on their way, per fill warp: 32 rows of up to 128 of a
  // key's channels, and 64 tokens by 64 value channels.
  static constexpr int kChans = D < 128 ? D : 128;
  static constexpr int kRawKs = 32 * kChans / 2, kRawV = kRawKs + 32 * kChans / 16;
  static constexpr int kRawVs = kRawV + 64 * 32, kRaw = kRawVs + 64 * 4;
  static constexpr int kBytes =
      kHalves * kQ + 4 * kK + kFillWarps * kRaw + kSoftWarps * kStageBytes + 1024;
  // Over prefixes: codes and scales of a tile's keys, or of its values.
  static constexpr int kCodes = kKeys * D / 2, kScales = kKeys * D / 16, kPartBytes = kCodes + kScales;
  static constexpr int kPrefixBytes = kHalves * kQ + 4 * kK + kParts * kPartBytes + 1024;
};

struct Bars {
  uint64_t q_ready[2], k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_ready[2],
      o_done[2], written[2], joined[2], drain;
  uint64_t raw_full[kParts], raw_empty[kParts];  // over prefixes
};

// 32 consecutive columns of this warp's 32 lanes. The values are there after
// tmem_landed.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,"
      "%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_landed(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
      : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
        "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]),
        "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]),
        "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]),
        "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
      :
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,"
      "%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
        "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
        "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
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

// The lowest n bits, of none to all.
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u;
}

// True in one lane of a warp that runs converged.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
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

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
// 4 or 8 bytes global -> shared.
template <int N>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(N) : "memory");
}

// Four 8x8 matrices of f16, transposed: lane l holds row l / 4, columns 2 (l % 4)
// and + 1 of each, and names the place of stored row l % 8 of matrix l / 8.
__device__ __forceinline__ void stmatrix_trans(uint32_t addr, const uint32_t (&m)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr),
               "r"(m[0]), "r"(m[1]), "r"(m[2]), "r"(m[3])
               : "memory");
}

// Byte offset of 16-byte chunk `chunk` of row `row` in a 128-byte-swizzled
// operand whose panels (64 f16 wide) hold `rows` rows.
__device__ __forceinline__ uint32_t swizzled(int row, int chunk, int rows) {
  return (chunk >> 3) * rows * 128 + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
}

// A row tile of the list: its request and its first row there.
struct RowTile {
  int b, row0;
};

// Clears the status and the counters and builds the list: firsts[b] is the
// first row tile of request b, starts[r] the first entry of row tile r, whose
// segments, one per kv head, have kSetup entries and their key tiles each.
template <int D>
__global__ void __launch_bounds__(kPlanThreads)
    prompt_plan_kernel(AttnArgs a, int max_row_tiles, unsigned* status, int* counters,
                       int n_counters, SeqInfo* info, int* firsts, RowTile* row_tiles,
                       long* starts) {
  using H = Shape<D>;
  __shared__ long warp_sum[kPlanThreads / 32];
  pdl_enter();
  if (threadIdx.x == 0) *status = 0;
  for (int i = threadIdx.x; i < n_counters; i += kPlanThreads) counters[i] = 0;
  __syncthreads();
  const int group = a.heads / a.kv_heads;
  unsigned flags = 0;
  long total = 0;
  for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
    const int b = b0 + threadIdx.x;
    long n = 0;
    if (b < a.B) {
      const SeqInfo s = seq_info(a, b, flags);
      info[b] = s;
      n = (static_cast<long>(s.q_len) * group + H::kTile - 1) / H::kTile;
    }
    const long before = block_scan<kPlanThreads>(n, warp_sum, total);
    // offsets that overlap could ask for more row tiles than T rows have
    if (b < a.B) firsts[b] = static_cast<int>(min(before, static_cast<long>(max_row_tiles)));
  }
  if (total > max_row_tiles) flags |= MOE_DEV_BAD_SEGMENT;
  const int n_tiles = static_cast<int>(min(total, static_cast<long>(max_row_tiles)));
  if (threadIdx.x == 0) firsts[a.B] = n_tiles;
  __syncthreads();
  long entries = 0;
  for (int r0 = 0; r0 < n_tiles; r0 += kPlanThreads) {
    const int r = r0 + threadIdx.x;
    long n = 0;
    if (r < n_tiles) {
      int lo = 0, hi = a.B;  // the last request whose first row tile is at most r
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (firsts[mid] <= r) lo = mid;
        else hi = mid;
      }
      const SeqInfo s = info[lo];
      const int row0 = (r - firsts[lo]) * H::kTile;
      row_tiles[r] = {lo, row0};
      const int last = min(s.q_len * group, row0 + H::kTile) - 1;
      const int before = s.len - s.q_len;
      const int first_key = a.window > 0 ? max(0, before + row0 / group - a.window + 1) : 0;
      const int end_key = before + last / group + 1;
      const int tiles =
          end_key <= 0 ? 0 : (end_key + H::kKeys - 1) / H::kKeys - first_key / H::kKeys;
      n = static_cast<long>(a.kv_heads) * (kSetup + tiles);
    }
    const long before = block_scan<kPlanThreads>(n, warp_sum, entries);
    if (r < n_tiles) starts[r] = before;
  }
  if (threadIdx.x == 0) starts[n_tiles] = entries;
  if (flags) atomicOr(status, flags);
}

// A CTA's part of a segment.
struct Piece {
  int b, kvh, row0, rows, halves;  // rows: of the request
  int lo, hi;                      // keys [lo, hi) are seen by some row
  int first, tiles;                // its key tiles
  bool alone;                      // it is the whole segment
  bool keys;                       // over prefixes: both halves have its rows, and every
                                   // other tile each
  int cta0, cta1;                  // CTAs of the segment's pieces
  SeqInfo sq;
};

// Walks a CTA's range of the list, whose cuts move to a segment's ends where
// those are near (kSnap < kMinTiles, so that no two cuts move to the same end).
// Every warp keeps one.
template <int D>
struct Cursor {
  using H = Shape<D>;
  long at, end, per, total;
  int r;
  __device__ __forceinline__ void begin(const long* starts, int n_tiles, int lane) {
    total = starts[n_tiles];
    per = (total + gridDim.x - 1) / gridDim.x;
    if (per < kMinTiles) per = kMinTiles;
    at = blockIdx.x * per;
    end = min(total, at + per);
    int lo = 0, hi = n_tiles;  // the last row tile that starts at or before `at`
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32, probe = lo + lane * step;
      const unsigned below = __ballot_sync(~0u, probe < hi && starts[probe] <= at);
      const int k = below ? 31 - __clz(below) : 0;
      lo += k * step;
      hi = min(hi, lo + step);
    }
    r = lo;
  }
  __device__ __forceinline__ bool next(const AttnArgs& a, const SeqInfo* info,
                                       const RowTile* row_tiles, const long* starts, Piece& p) {
    for (;;) {
      if (at >= end) return false;
      while (starts[r + 1] <= at) ++r;
      const RowTile rt = row_tiles[r];
      p.b = rt.b;
      p.row0 = rt.row0;
      p.sq = info[rt.b];
      const int group = a.heads / a.kv_heads;
      p.rows = p.sq.q_len * group;
      const int last = min(p.rows, p.row0 + H::kTile) - 1;
      p.halves = last >= p.row0 + kHalf ? 2 : 1;
      const int before = p.sq.len - p.sq.q_len;
      p.lo = a.window > 0 ? max(0, before + p.row0 / group - a.window + 1) : 0;
      p.hi = before + last / group + 1;
      const int tiles = p.hi <= 0 ? 0 : (p.hi + H::kKeys - 1) / H::kKeys - p.lo / H::kKeys;
      const int len = kSetup + tiles;
      p.kvh = static_cast<int>((at - starts[r]) / len);
      const long seg = starts[r] + static_cast<long>(p.kvh) * len;
      int p0 = static_cast<int>(at - seg);
      if (p0 <= kSnap) {
        p0 = 0;
      } else if (len - p0 <= kSnap) {  // the CTA before takes all of it
        at = seg + len;
        continue;
      }
      int p1 = static_cast<int>(min(static_cast<long>(len), end - seg));
      if (p1 < len && p1 <= kSnap) return false;  // the next CTA takes all of it
      if (len - p1 <= kSnap) p1 = len;
      const int t0 = max(0, p0 - kSetup);
      p.first = p.lo / H::kKeys + t0;
      p.tiles = p1 - kSetup - t0;
      p.alone = p0 == 0 && p1 == len;
      p.cta0 = static_cast<int>((seg + kSnap) / per);
      p.cta1 = max(p.cta0, static_cast<int>((seg + len - kSnap - 1) / per));
      at = seg + p1;
      return true;
    }
  }
};

// The same over prefixes: a group's segments have as many entries, but those of a
// last row tile with one half's rows. There both halves take the same rows and every
// other key tile, which then takes 1.4 us of an SM, and 1.9 with two halves' rows: three
// entries, and four. (128 rows over 131072 tokens 103 us, and 121 with one half alone;
// 384 rows 212 and 232. 256 rows over 32768 tokens pay for it with 1 of 56.)
constexpr int kUnit = 4, kHalfUnit = 3;
constexpr int kPrefixSetup = kSetup * kUnit;
// A cut in a segment's set-up entries, which stand for no tiles, moves to its begin;
// near the end only one tile is not cut off, since joining pieces is cheap here and a
// CTA with four tiles more holds up the others (56 us instead of 48, 256 rows over
// 32768 tokens).
constexpr int kPrefixSnap = kUnit;
// Smallest range of a CTA: pieces of two tiles.
constexpr int kMinPrefix = 2 * kUnit;
static_assert(kMinPrefix >= kPrefixSnap + kUnit, "cuts do not cross, pieces have tiles");
template <int D>
struct PrefixCursor {
  using H = Shape<D>;
  const SeqInfo* groups;
  const long* bases;
  long at, end, per;
  int g;
  __device__ __forceinline__ void begin(const PrefixSums& p, const SeqInfo* groups_in,
                                        const long* bases_in) {
    groups = groups_in;
    bases = bases_in;
    const long total = bases[p.gr.n];
    per = prefix_per(p.shape, total);
    at = blockIdx.x * per;
    end = min(total, at + per);
    g = last_at_most(bases, p.gr.n, at);
  }
  __device__ __forceinline__ bool next(const AttnArgs& a, Piece& p) {
    for (;;) {
      if (at >= end) return false;
      while (bases[g + 1] <= at) ++g;
      p.sq = groups[g];
      p.rows = p.sq.q_len * (a.heads / a.kv_heads);
      const int key_tiles = (p.sq.len + H::kKeys - 1) / H::kKeys;
      int len = kPrefixSetup + key_tiles * kUnit;
      const int i = static_cast<int>(quotient(at - bases[g], len));
      const int row_tile = i / a.kv_heads;  // (also in a last one of shorter segments)
      p.row0 = row_tile * H::kTile;
      p.halves = H::kHalves == 2 && p.rows - p.row0 > kHalf ? 2 : 1;
      p.kvh = i - row_tile * a.kv_heads;
      long seg = bases[g] + static_cast<long>(i) * len;
      const bool shorter = H::kHalves == 2 && p.halves == 1;
      if (shorter) {
        seg -= static_cast<long>(p.kvh) * len;
        len = kPrefixSetup + key_tiles * kHalfUnit;
        p.kvh = static_cast<int>(quotient(at - seg, len));
        seg += static_cast<long>(p.kvh) * len;
      }
      p.lo = 0;
      p.hi = p.sq.len;
      int p0 = static_cast<int>(at - seg);
      if (p0 <= kPrefixSetup) {
        p0 = 0;
      } else if (len - p0 <= kPrefixSnap) {  // the CTA before takes all of it
        at = seg + len;
        continue;
      }
      int p1 = static_cast<int>(min(static_cast<long>(len), end - seg));
      if (p1 < len && p1 <= kPrefixSetup) return false;  // the next CTA takes all of it
      if (len - p1 <= kPrefixSnap) p1 = len;
      // the tiles whose first entry lies between the cuts
      auto tiles_to = [&](int entry) {
        const unsigned e = max(0, entry - kPrefixSetup);
        return static_cast<int>(shorter ? (e + kHalfUnit - 1) / kHalfUnit : (e + kUnit - 1) / kUnit);
      };
      p.first = tiles_to(p0);
      p.tiles = tiles_to(p1) - p.first;
      p.alone = p0 == 0 && p1 == len;
      p.keys = H::kHalves == 2 && p.halves == 1 && p.tiles > 1 && !p.alone;
      p.cta0 = static_cast<int>(quotient(seg + kPrefixSetup, per));
      at = seg + p1;
      return true;
    }
  }
};

// kPart kPrefix: a request is a group of requests, its first_key names the row of
// the page table, every row sees all keys, and sums are left in fp32.
template <int D, int kPart = kWhole>
__global__ void __launch_bounds__(kThreads, 1)
    attn_prompt_kernel(AttnArgs a, unsigned* status, int* counters, const SeqInfo* info,
                       const int* firsts, const RowTile* row_tiles, const long* starts,
                       float2* stats, float4* partial, PartArgs<kPart> part) {
  using H = Shape<D>;
  constexpr int kKeys = H::kKeys;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Bars bars;
  constexpr int kBadTiles = kPart == kPrefix ? kPrefixBadRing : kBadRing;
  __shared__ __align__(16) uint32_t s_bad[kBadTiles][4];
  __shared__ uint32_t s_tmem;
  __shared__ int s_last[2];
  __shared__ volatile int s_abort;
  const uint32_t base = (ptx::smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sm_q = base, sm_k = base + H::kHalves * H::kQ, sm_v = sm_k + 2 * H::kK,
                 sm_raw = sm_v + 2 * H::kK, sm_stage = sm_raw + kFillWarps * H::kRaw;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto bar = [&](const uint64_t& b) { return ptx::smem_u32(&b); };

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(bar(bars.q_ready[i]), 4);
      ptx::mbar_init(bar(bars.k_full[i]), kFillWarps);
      ptx::mbar_init(bar(bars.k_empty[i]), 1);
      ptx::mbar_init(bar(bars.v_full[i]), kFillWarps);
      ptx::mbar_init(bar(bars.v_empty[i]), 1);
      ptx::mbar_init(bar(bars.s_full[i]), 1);
      ptx::mbar_init(bar(bars.p_ready[i]), 4);
      ptx::mbar_init(bar(bars.o_done[i]), 1);
      ptx::mbar_init(bar(bars.written[i]), 4);
      ptx::mbar_init(bar(bars.joined[i]), 1);
    }
    for (int i = 0; i < kParts; ++i) {
      ptx::mbar_init(bar(bars.raw_full[i]), 1);
      ptx::mbar_init(bar(bars.raw_empty[i]), kFillWarps);
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
  const uint32_t tmem = __shfl_sync(~0u, s_tmem, 0);  // (known to be uniform)
  // Over prefixes every CTA sums up the list itself. What the kernel before this
  // one, the call's plan, writes concerns the own kernel: an idle warp waits for it
  // (behind its group's register release, which all four warps take part in).
  const SeqInfo* groups = nullptr;
  const long* bases = nullptr;
  bool planned = true;
  if constexpr (kPart == kPrefix) {
    __shared__ GroupSmem s_groups;
    __shared__ long s_sum[kThreads / 32];
    groups = part.p.groups;
    bases = part.p.bases;
    planned = part.p.gr.n > kSmallGroups;
    if (!planned) {
      unsigned reported = 0;  // by the plan
      plan_groups<kThreads>(a, part.p.gr, part.p.shape, s_groups.lists(), &s_groups, s_sum, reported,
                            [](int, const SeqInfo&, int) {});
      groups = s_groups.groups;
      bases = s_groups.bases;
    }
  }
  if (planned) pdl_enter();
  const int group = a.heads / a.kv_heads;
  const uint64_t limit = ptx::wait_limit();
  auto wait = [&](const uint64_t& b, uint32_t parity) {
    return ptx::mbar_wait_asleep(bar(b), parity, limit, &s_abort, status);
  };
  // The same for a whole warp: all lanes go on or none (a timeout may reach
  // some lanes only, and tensor memory is read by whole warps).
  auto wait_warp = [&](const uint64_t& b, uint32_t parity) {
    return __all_sync(~0u, wait(b, parity)) != 0;
  };
  std::conditional_t<kPart == kPrefix, PrefixCursor<D>, Cursor<D>> cur;
  Piece t;
  auto begin = [&] {
    if constexpr (kPart == kPrefix)
      cur.begin(part.p, groups, bases);
    else
      cur.begin(starts, firsts[a.B], lane);
  };
  auto next = [&] {
    if constexpr (kPart == kPrefix)
      return cur.next(a, t);
    else
      return cur.next(a, info, row_tiles, starts, t);
  };

  constexpr bool kByKeys = kPart == kPrefix && H::kHalves == 2;
  auto by_keys = [&] { return kByKeys && t.keys; };

  if (warp < kSoftWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    // ---------------------------------------------------------------- softmax
    const int x = warp >> 2, wl = warp & 3;
    const int row_l = wl * 32 + lane;  // row of the half, lane of tensor memory
    const uint32_t ts = tmem + (wl << 21) + kColsS + x * kKeys;
    const uint32_t to = tmem + (wl << 21) + kColsO + x * D;
    const uint32_t sm_rows = sm_q + x * H::kQ;
    const uint32_t stage = sm_stage + warp * kStageBytes;
    uint32_t s_phase = 0, o_phase = 0, join_phase = 0, tile_no = 0;
    // This thread's row of the current piece.
    int r, tok, head;
    bool live;
    float gain = 0.0f;
    auto place = [&] {
      r = t.row0 + (by_keys() ? 0 : x * kHalf) + row_l;
      live = r < t.rows;
      tok = r / group;
      head = t.kvh * group + (r - tok * group);
    };
    // The next piece with keys for this half; what has none is zeroed.
    auto advance = [&] {
      while (next()) {
        if (x >= t.halves && !by_keys()) {
          tile_no += t.tiles;
          if constexpr (kByKeys) {
            if (!t.alone) {  // a single tile: nothing is left for this half
              const long row = (2l * blockIdx.x + (blockIdx.x == t.cta0)) * H::kTile + kHalf + row_l;
              stats[row] = make_float2(-INFINITY, 0.0f);
              for (int i = 0; i < D / 4; ++i)
                partial[sums_at(row, i, D / 4)] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
          }
          continue;
        }
        place();
        if (t.tiles > 0) return true;
        if (live) {
          const long at_row = static_cast<long>(t.sq.q0 + tok) * a.heads + head;
          uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + at_row * D);
          for (int i = 0; i < D / 8; ++i) dst[i] = make_uint4(0, 0, 0, 0);
          if (a.lse) a.lse[at_row] = -INFINITY;
        }
      }
      return false;
    };
    // The warp's rows of queries, whole rows by neighbouring lanes, scaled to
    // f16; each lane keeps its own row's gain.
    auto load_queries = [&] {
      // rows asked for together: over a prefix a CTA has one piece, as a rule, and
      // its queries are what the first product waits for
      constexpr int kRowLanes = D / 8, kRowsStep = 32 / kRowLanes;
      constexpr int kBatch = kPart == kPrefix ? 8 : 4;
      const long src = (t.sq.q0 + (live ? tok : 0)) * a.q.token + (live ? head : 0) * a.q.head;
#pragma unroll 1
      for (int first = 0; first < kRowLanes; first += kBatch) {
        uint4 w[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int rl = (first + i) * kRowsStep + lane / kRowLanes;
          const long at = __shfl_sync(~0u, src, rl);
          const bool there = __shfl_sync(~0u, static_cast<int>(live), rl);
          w[i] = there ? *reinterpret_cast<const uint4*>(
                             static_cast<const __nv_bfloat16*>(a.q.p) + at + lane % kRowLanes * 8)
                       : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int rl = (first + i) * kRowsStep + lane / kRowLanes;
          const uint32_t v[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
          float top = 0.0f;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            top = fmaxf(top, fmaxf(fabsf(__uint_as_float(v[j] << 16)),
                                   fabsf(__uint_as_float(v[j] & 0xffff0000u))));
#pragma unroll
          for (int d = kRowLanes / 2; d > 0; d /= 2)
            top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
          float up, down;
          row_power(top, up, down);
          uint32_t h[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            h[j] = pack_f16(__uint_as_float(v[j] << 16) * up,
                            __uint_as_float(v[j] & 0xffff0000u) * up);
          sts128(sm_rows + swizzled(wl * 32 + rl, lane % kRowLanes, kHalf), h[0], h[1], h[2], h[3]);
          const float mine = __shfl_sync(~0u, down, (lane % kRowsStep) * kRowLanes);
          if (lane / kRowsStep == first + i) gain = score_gain(mine, a.scale_log2);
        }
      }
      ptx::fence_proxy_async();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar(bars.q_ready[x]));
    };
    // 32 columns of the warp's rows as bf16 to their places in `out`, through
    // the warp's staging rows of 32 bytes: whole sectors by lane pairs.
    auto store_columns = [&](int c, const float* v, float f, long at_row, bool there) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t h[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const __nv_bfloat162 b2 =
              __floats2bfloat162_rn(v[16 * q + 2 * i] * f, v[16 * q + 2 * i + 1] * f);
          h[i] = *reinterpret_cast<const uint32_t*>(&b2);
        }
        const int flip = (lane >> 2) & 1;  // spreads eight rows over the banks
        __syncwarp();
        sts128(stage + lane * 32 + 16 * flip, h[0], h[1], h[2], h[3]);
        sts128(stage + lane * 32 + 16 * (flip ^ 1), h[4], h[5], h[6], h[7]);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int rl = 16 * i + (lane >> 1);
          const long row = __shfl_sync(~0u, at_row, rl);
          const bool store = __shfl_sync(~0u, static_cast<int>(there), rl);
          const uint4 w = lds128(stage + rl * 32 + 16 * ((lane & 1) ^ ((rl >> 2) & 1)));
          if (store)
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + row * D + 32 * c +
                                      16 * q + 8 * (lane & 1)) = w;
        }
      }
    };

    begin();
    bool more = x < H::kHalves && advance();
    if (more) load_queries();
    while (more) {
      const int p = kPart == kPrefix ? t.sq.len - 1 : t.sq.len - t.sq.q_len + tok;
      const int last = live ? p : 0x7ffffff0;  // (one more is added below)
      const int first = live && a.window > 0 ? p - a.window + 1 : 0;
      // keys that every row of the half sees
      const int r_lo = t.row0 + x * kHalf, r_hi = min(t.rows, r_lo + kHalf) - 1;
      const int all_last = kPart == kPrefix ? t.sq.len - 1 : t.sq.len - t.sq.q_len + r_lo / group;
      const int all_first = a.window > 0 ? t.sq.len - t.sq.q_len + r_hi / group - a.window + 1 : 0;
      const bool keys = by_keys();
      const bool frees = (keys || x == t.halves - 1) && threadIdx.x % 128 == 0;
      float m = -INFINITY, mbase = -kLift;  // m: a whole number
      uint64_t l2[2] = {0, 0};              // partial sums of P
      const uint64_t gain2 = pair_f32(gain, gain);
      bool ok = true;
      const uint32_t tile0 = tile_no;
      const int step = keys ? 2 : 1;
#pragma unroll 1
      for (int j = keys ? x : 0; j < t.tiles; j += step) {
        tile_no = tile0 + j;
        if (!(ok = wait_warp(bars.s_full[x], s_phase))) break;
        s_phase ^= 1;
        ptx::tc_fence_after();
        // This half's scores are the tile's last ones: the keys are free, and the
        // values of the tile before, whose products were issued earlier. (A
        // commit for each would hold up the matrix thread; where the halves take
        // tiles in turn there is one for each, since a half's next scores come late.)
        if (frees) {
          ptx::mbar_arrive(bar(bars.k_empty[tile_no & 1]));
          if (j > 0 && !keys) ptx::mbar_arrive(bar(bars.v_empty[(tile_no - 1) & 1]));
        }
        const int tok0 = (t.first + j) * kKeys;
        const uint32_t bad_at = ptx::smem_u32(s_bad[tile_no % kBadTiles]);
        const bool inside = tok0 >= all_first && tok0 + kKeys - 1 <= all_last;
#pragma unroll 1
        for (int c = 0; c < kKeys / 64; ++c) {
          uint32_t s[64];
          tmem_ld32(ts + 64 * c, *reinterpret_cast<uint32_t(*)[32]>(s));
          tmem_ld32(ts + 64 * c + 32, *reinterpret_cast<uint32_t(*)[32]>(s + 32));
          const uint2 bad = lds64(bad_at + 8 * c);
          tmem_landed(*reinterpret_cast<uint32_t(*)[32]>(s));
          tmem_landed(*reinterpret_cast<uint32_t(*)[32]>(s + 32));
          if (!inside || (bad.x | bad.y) != 0) {
            // keys from `first` to `last`, but those on bad pages, as bits
            const int key0 = tok0 + 64 * c;
            const uint32_t seen[2] = {low_bits(last + 1 - key0) & ~low_bits(first - key0) & ~bad.x,
                                      low_bits(last - 31 - key0) & ~low_bits(first - 32 - key0) &
                                          ~bad.y};
#pragma unroll
            for (int i = 0; i < 64; ++i)
              if (!(seen[i / 32] & (1u << (i % 32)))) s[i] = 0xff800000u;
          }
          uint32_t pk[32];
          uint64_t add[2];
#pragma unroll 1
          for (bool again = false;; again = true) {
            const uint64_t off2 = pair_f32(-mbase, -mbase);
            uint32_t tops[4] = {0, 0, 0, 0};
            add[0] = add[1] = 0;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              float x0, x1;
              unpair_f32(fma_f32x2(pair_b32(s[2 * i], s[2 * i + 1]), gain2, off2), x0, x1);
              const float p0 = ex2(x0), p1 = ex2(x1);
              add[i & 1] = add_f32x2(add[i & 1], pair_f32(p0, p1));
              pk[i] = pack_f16(p0, p1);
              tops[i & 3] = max_f16x2(tops[i & 3], pk[i]);
            }
            const float2 top = unpack_f16(
                max_f16x2(max_f16x2(tops[0], tops[1]), max_f16x2(tops[2], tops[3])));
            if (again || !__any_sync(~0u, fmaxf(top.x, top.y) > kMostP || m == -INFINITY)) break;
            // A row has outgrown its maximum (or has none yet): move it up by
            // whole powers of two and scale down what has been summed.
            float mx = __uint_as_float(s[0]);
#pragma unroll
            for (int i = 1; i < 64; ++i) mx = fmaxf(mx, __uint_as_float(s[i]));
            const float nm = fmaxf(m, ceilf(mx * gain));
            const float nb = nm == -INFINITY ? -kLift : nm - kLift;
            const float f = m == -INFINITY ? 0.0f : ex2(mbase - nb);
            m = nm;
            mbase = nb;
            l2[0] = fma_f32x2(l2[0], pair_f32(f, f), 0);
            l2[1] = fma_f32x2(l2[1], pair_f32(f, f), 0);
            if (c > 0) {  // P of this tile's first columns
              uint32_t w[32];
              tmem_wait_st();
              tmem_ld32(ts, w);
              tmem_landed(w);
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const float2 g2 = unpack_f16(w[i]);
                w[i] = pack_f16(g2.x * f, g2.y * f);
              }
              tmem_st32(ts, w);
            }
            if (j >= step) {  // the products of the tiles before have landed (s_full)
#pragma unroll 1
              for (int q = 0; q < D / 32; ++q) {
                uint32_t w[32];
                tmem_ld32(to + 32 * q, w);
                tmem_landed(w);
#pragma unroll
                for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * f);
                tmem_st32(to + 32 * q, w);
              }
            }
          }
          l2[0] = add_f32x2(l2[0], add[0]);
          l2[1] = add_f32x2(l2[1], add[1]);
          tmem_st32(ts + 32 * c, pk);
        }
        tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(bars.p_ready[x]));
      }
      if (!ok) break;
      // The next piece's queries go in first (every score of this one is done),
      // so that its first product does not wait for this one's rows.
      const long at_row = static_cast<long>(t.sq.q0 + tok) * a.heads + head;
      const bool there = live, alone = t.alone;
      const int cta0 = t.cta0, cta1 = t.cta1;
      tile_no = tile0 + t.tiles;
      const uint32_t last_tile = tile_no - 1;
      more = advance();
      if (more) load_queries();
      if (!wait_warp(bars.o_done[x], o_phase)) break;
      o_phase ^= 1;
      if (frees && !keys) ptx::mbar_arrive(bar(bars.v_empty[last_tile & 1]));
      ptx::tc_fence_after();
      float l;
      {
        float l0, l1;
        unpair_f32(add_f32x2(l2[0], l2[1]), l0, l1);
        l = l0 + l1;
      }
      if constexpr (kPart == kPrefix) {
        // sums and statistics by row: whole segments to the rows' places, pieces
        // to the CTA's slot (1 where the segment begins in it)
        const long row = alone ? at_row
                               : (2l * blockIdx.x + (blockIdx.x == cta0)) * H::kTile + x * kHalf + row_l;
        const bool store = there || !alone;
        float4* dst = (alone ? part.p.row_sums : partial) + sums_at(row, 0, D / 4);
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t v[32];
          tmem_ld32(to + 32 * c, v);
          tmem_landed(v);
          // column 8 (4 c + m) + 2 q + b is channel D / 4 q + 8 c + 2 m + b
          if (store)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int q = i / 2, at = 16 * (i % 2) + 2 * q;
              dst[(D / 16 * q + 2 * c + i % 2) * 8] =
                  make_float4(__uint_as_float(v[at]), __uint_as_float(v[at + 1]),
                              __uint_as_float(v[at + 8]), __uint_as_float(v[at + 9]));
            }
        }
        if (store)
          (alone ? part.p.row_stats : stats)[row] = make_float2(m == -INFINITY ? -INFINITY : mbase, l);
        ptx::tc_fence_before();
        continue;
      } else if (alone) {
        const float f = out_factor(l, a.v_scale);
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t v[32];
          tmem_ld32(to + 32 * c, v);
          tmem_landed(v);
          store_columns(c, reinterpret_cast<const float*>(v), f, at_row, there);
        }
        if (there && a.lse) a.lse[at_row] = log_sum(mbase, l);
        ptx::tc_fence_before();
        continue;
      }
      // A piece: sums [D / 4][row] and statistics [row] to the workspace, lanes
      // at neighbouring rows. The CTA a segment begins in keeps its piece in
      // slot 1, later ones in slot 0.
      auto slot_of = [&](int cta) { return (2l * cta + (cta == cta0)) * H::kHalves + x; };
      {
        const long slot = slot_of(blockIdx.x);
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t v[32];
          tmem_ld32(to + 32 * c, v);
          tmem_landed(v);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            partial[(slot * (D / 4) + 8 * c + i) * kHalf + row_l] =
                make_float4(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1]),
                            __uint_as_float(v[4 * i + 2]), __uint_as_float(v[4 * i + 3]));
        }
        stats[slot * kHalf + row_l] = make_float2(m == -INFINITY ? -INFINITY : mbase, l);
      }
      ptx::tc_fence_before();
      __threadfence();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar(bars.written[x]));
      if (wl == 0) {
        if (!wait_warp(bars.written[x], join_phase)) break;
        if (lane == 0) {
          __threadfence();
          *reinterpret_cast<volatile int*>(&s_last[x]) =
              ptx::add_acq_rel(counters + 2 * cta0 + x, 1) == cta1 - cta0;
          ptx::mbar_arrive(bar(bars.joined[x]));
        }
      }
      if (!wait_warp(bars.joined[x], join_phase)) break;
      join_phase ^= 1;
      if (!*reinterpret_cast<volatile int*>(&s_last[x])) continue;
      __threadfence();
      float top = -INFINITY, den = 0.0f;
#pragma unroll 4
      for (int k = cta0; k <= cta1; ++k)
        top = fmaxf(top, __ldcg(&stats[slot_of(k) * kHalf + row_l]).x);
      auto weight = [&](float b2) { return b2 == -INFINITY ? 0.0f : ex2(b2 - top); };
#pragma unroll 4
      for (int k = cta0; k <= cta1; ++k) {
        const float2 st = __ldcg(&stats[slot_of(k) * kHalf + row_l]);
        den += weight(st.x) * st.y;
      }
      const float f = out_factor(den, a.v_scale);
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        float sum[32] = {};
#pragma unroll 1
        for (int k = cta0; k <= cta1; k += 2) {  // two pieces' loads at a time
          float4 v[2][8];
          float w[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const long slot = slot_of(min(k + e, cta1));
            w[e] = __ldcg(&stats[slot * kHalf + row_l]).x;
#pragma unroll
            for (int i = 0; i < 8; ++i)
              v[e][i] = __ldcg(&partial[(slot * (D / 4) + 8 * c + i) * kHalf + row_l]);
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float g2 = k + e <= cta1 ? weight(w[e]) : 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              sum[4 * i] += g2 * v[e][i].x, sum[4 * i + 1] += g2 * v[e][i].y;
              sum[4 * i + 2] += g2 * v[e][i].z, sum[4 * i + 3] += g2 * v[e][i].w;
            }
          }
        }
        store_columns(c, sum, f, at_row, there);
      }
      if (there && a.lse) a.lse[at_row] = log_sum(top, den);
    }
  } else if (warp < kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFillRegs));
    // ------------------------------------------------- codes to f16 operands
    // A warp converts slices of its own, so that the codes it has under way in
    // shared memory concern nobody else. The loops stay rolled: the three
    // roles' code has to fit the instruction cache together (fully unrolled, the
    // kernel spent most of its time fetching instructions).
    const int ft = threadIdx.x - kSoftWarps * 32, fw = warp - kSoftWarps;
    // keys: lane's row kr, all of its channels or half of 256
    constexpr int kChans = H::kChans;
    const int kr = ft % kKeys, kpart = ft / kKeys;
    if constexpr (kPart == kPrefix) {
      // Whole parts come from the copying warp, so that all four warps wait for the
      // same ones; copies issued by these warps took half of their time.
      // Keys: a lane has a row, its 16-byte chunks in an order of its own, so that
      // eight lanes read, and write, different banks. Values: a lane has a quarter
      // of a token's channels; words of eight channels of eight tokens are turned
      // into rows of tokens by matrix stores. Channel D / 4 q + 8 k + 2 m + b (q:
      // lane, k: word, m: matrix) becomes row 8 (4 k + m) + 2 q + b of the operand,
      // so that a matrix's rows follow one another; the sums' columns go back to
      // their channels as they are stored.
      constexpr int kChunks = kChans / 32, kWords = D / 32;
      const int spin = D == 128 ? lane >> 1 : D == 64 ? lane >> 2 : lane;
      uint32_t kc = 0, slot = 0, phase = 0;
      auto part_at = [&] { return sm_raw + slot * H::kPartBytes; };
      auto part_done = [&] {
        if (lane == 0) ptx::mbar_arrive(bar(bars.raw_empty[slot]));
        if (++slot == kParts) slot = 0, phase ^= 1;
      };
      bool ok = true;
      begin();
      while (ok && next()) {
#pragma unroll 1
        for (int j = 0; j < t.tiles; ++j, ++kc) {
          const uint32_t st = kc & 1, parity = ((kc >> 1) & 1) ^ 1;
          if (!(ok = wait_warp(bars.raw_full[slot], phase) && wait_warp(bars.k_empty[st], parity)))
            break;
          const uint32_t codes = part_at() + kr * (D / 2) + kpart * (kChans / 2);
          const uint32_t scales = part_at() + H::kCodes + kr * (D / 16) + kpart * (kChans / 16);
#pragma unroll 2
          for (int n = 0; n < kChunks; ++n) {
            const int i = (n + spin) % kChunks;
            const uint4 w = lds128(codes + 16 * i);
            const uint32_t two = e4m3x2_to_f16(lds16(scales + 2 * i));
            const uint32_t s2[2] = {f16_low_twice(two), f16_high_twice(two)};
            const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t h[4];
              e2m1_to_f16(words[c], h);
              const uint32_t sc = s2[c / 2];
              sts128(sm_k + st * H::kK + swizzled(kr, kpart * (kChans / 8) + 4 * i + c, kKeys),
                     hmul2(h[0], sc), hmul2(h[1], sc), hmul2(h[2], sc), hmul2(h[3], sc));
            }
          }
          ptx::fence_proxy_async();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(bar(bars.k_full[st]));
          part_done();
          if (!(ok = wait_warp(bars.raw_full[slot], phase) && wait_warp(bars.v_empty[st], parity)))
            break;
#pragma unroll 1
          for (int n = 0; n < kKeys / 8 / kFillWarps; ++n) {
            const int eight = fw * (kKeys / 8 / kFillWarps) + n;  // of the tile's tokens
            const int tok = 8 * eight + lane / 4, q = lane & 3;
            const uint32_t row = part_at() + tok * (D / 2) + q * (D / 8);
            uint32_t words[kWords];
            if constexpr (kWords == 2) {
              const uint2 w = lds64(row);
              words[0] = w.x, words[1] = w.y;
            } else {
#pragma unroll
              for (int k = 0; k < kWords; k += 4) {
                const uint4 w = lds128(row + 4 * k);
                words[k] = w.x, words[k + 1] = w.y, words[k + 2] = w.z, words[k + 3] = w.w;
              }
            }
            // a key that no row sees may be uninitialised memory: a zero scale keeps
            // 0 * NaN out of the sum
            const uint32_t bad = lds32(ptx::smem_u32(&s_bad[kc % kBadTiles][tok / 32]));
            const bool seen = (t.first + j) * kKeys + tok < t.hi && !((bad >> (tok % 32)) & 1u);
            const uint32_t at = part_at() + H::kCodes + tok * (D / 16) + q * (D / 64);
            uint32_t bytes = D == 64 ? lds8(at) : D == 128 ? lds16(at) : lds32(at);
            if (!seen) bytes = 0;
            uint32_t two = 0;
#pragma unroll
            for (int k = 0; k < kWords; ++k) {
              if (k % 4 == 0) two = e4m3x2_to_f16(bytes >> (4 * k));
              const uint32_t sc = k % 4 < 2 ? f16_low_twice(two) : f16_high_twice(two);
              uint32_t h[4];
              e2m1_to_f16(words[k], h);
#pragma unroll
              for (int m = 0; m < 4; ++m) h[m] = hmul2(h[m], sc);
              stmatrix_trans(sm_v + st * H::kK + swizzled(32 * k + lane, eight, D), h);
            }
          }
          ptx::fence_proxy_async();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(bar(bars.v_full[st]));
          part_done();
        }
      }
    } else {
    // values: 64 tokens from v0, 64 channels from 64 * vq; lane's eight tokens
    // begin at vt, its 16 channels at 16 * vg. Eight neighbouring lanes have
    // different tokens and the same channels: their 16-byte stores fall on the
    // eight chunks of one 128-byte row.
    const int v0 = kKeys == 128 ? 64 * (fw & 1) : 0, vq = kKeys == 128 ? fw >> 1 : fw;
    const int vt = v0 + (lane & 7) * 8, vg = 4 * vq + (lane >> 3);
    const bool has_v = vq < D / 64;
    const KvBlock blk = kv_block(a.page_size, D);
    const int page_mask = a.page_size - 1, page_shift = 31 - __clz(a.page_size);
    const uint32_t raw = sm_raw + fw * H::kRaw;
    uint32_t kc = 0;
    begin();
    while (next()) {
      const int32_t* pages =
          a.page_table + static_cast<long>(kPart == kPrefix ? t.sq.first_key : t.b) * a.max_pages;
      // The page of eight keys from `key` (0 where no row sees one of them).
      auto page_of = [&](int key) {
        return key < t.hi && key + 7 >= t.lo ? pages[key >> page_shift] : 0;
      };
      auto checked = [&](int id, bool& ok) {
        ok = id >= 0 && id < a.num_pages;
        return ok ? id : 0;
      };
      auto block_of = [&](int id) {
        return a.cache + (static_cast<long>(id) * a.kv_heads + t.kvh) * blk.bytes;
      };
      // While a tile's keys or values are converted, its values or the next
      // tile's keys are copied; page ids are read one tile ahead of that. Eight
      // neighbouring tokens lie on one page.
      bool k_ok = true, v_ok = true;
      int kid = page_of(t.first * kKeys + (kr & ~7)), vid = page_of(t.first * kKeys + vt);
      auto copy_k = [&](int j) {
        if (j < t.tiles) {
          const int key = (t.first + j) * kKeys + kr, key0 = key - lane;
          const int id = checked(kid, k_ok);
          constexpr int kChunks = kChans / 32, kRows = 32 / kChunks;  // 16-byte chunks of a row,
          const int r0 = lane / kChunks, c = lane % kChunks;          // rows copied at a time
          // chunks of a row are swizzled by the row: lanes read one chunk of 32
          // rows at a time
          const int place = kChunks == 4 ? c ^ ((r0 >> 1) & 3) : c ^ ((r0 >> 2) & 1);
#pragma unroll
          for (int i = 0; i < kChunks; ++i) {
            const int r = kRows * i + r0;
            const uint8_t* p = block_of(__shfl_sync(~0u, id, r & ~7));
            ptx::cp_async16(raw + (r * kChunks + place) * 16,
                            p + ((key0 + r) & page_mask) * (D / 2) + kpart * (kChans / 2) + 16 * c);
          }
          cp_async_small<kChans / 16>(raw + H::kRawKs + lane * (kChans / 16),
                                      block_of(id) + blk.k_scale + (key & page_mask) * (D / 16) +
                                          kpart * (kChans / 16));
          if (j + 1 < t.tiles) kid = page_of((key & ~7) + kKeys);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
      auto copy_v = [&](int j) {
        if (j < t.tiles && has_v) {
          const int key = (t.first + j) * kKeys + vt, key0 = (t.first + j) * kKeys + v0;
          const int id = checked(vid, v_ok);
          // token 8 * g + e of the slice goes to row 8 * e + g: the lanes' g-th
          // groups lie side by side
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int tok = 16 * i + (lane >> 1), g = tok >> 3, e = tok & 7;
            const uint8_t* p = block_of(__shfl_sync(~0u, id, g));
            ptx::cp_async16(raw + H::kRawV + (8 * e + g) * 32 + (lane & 1) * 16,
                            p + blk.v_code + ((key0 + tok) & page_mask) * (D / 2) + vq * 32 +
                                (lane & 1) * 16);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int tok = 32 * i + lane, g = tok >> 3, e = tok & 7;
            const uint8_t* p = block_of(__shfl_sync(~0u, id, g));
            cp_async_small<4>(raw + H::kRawVs + (8 * e + g) * 4,
                              p + blk.v_scale + ((key0 + tok) & page_mask) * (D / 16) + vq * 4);
          }
          if (j + 1 < t.tiles) vid = page_of(key + kKeys);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
      copy_k(0);
      copy_v(0);
      bool ok = true;
#pragma unroll 1
      for (int j = 0; j < t.tiles; ++j, ++kc) {
        const uint32_t st = kc & 1, parity = ((kc >> 1) & 1) ^ 1;
        if (!(ok = wait_warp(bars.k_empty[st], parity))) break;
        const uint32_t bad = __ballot_sync(~0u, !k_ok);
        if (lane == 0) {
          if (bad) atomicOr(status, MOE_DEV_BAD_PAGE);
          // (with 64 keys, warps 2 and 3 see the same rows again)
          *reinterpret_cast<volatile uint32_t*>(&s_bad[kc % kBadTiles][fw]) = bad;
        }
        asm volatile("cp.async.wait_group 1;" ::: "memory");  // the keys, not the values
        __syncwarp();
#pragma unroll 2
        for (int i = 0; i < kChans / 32; ++i) {
          constexpr int kChunks = kChans / 32;
          const int place = kChunks == 4 ? i ^ ((lane >> 1) & 3) : i ^ ((lane >> 2) & 1);
          const uint4 w = lds128(raw + (lane * kChunks + place) * 16);
          const uint32_t two =
              e4m3x2_to_f16(lds16(raw + H::kRawKs + lane * (kChans / 16) + 2 * i));
          const uint32_t s2[2] = {f16_low_twice(two), f16_high_twice(two)};
          const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t h[4];
            e2m1_to_f16(words[c], h);
            const uint32_t s = s2[c / 2];
            sts128(sm_k + st * H::kK + swizzled(kr, kpart * (kChans / 8) + 4 * i + c, kKeys),
                   hmul2(h[0], s), hmul2(h[1], s), hmul2(h[2], s), hmul2(h[3], s));
          }
        }
        ptx::fence_proxy_async();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(bars.k_full[st]));
        copy_k(j + 1);
        if (!(ok = wait_warp(bars.v_empty[st], parity))) break;
        asm volatile("cp.async.wait_group 1;" ::: "memory");  // the values, not the next keys
        __syncwarp();
        if (has_v) {
          const int key = (t.first + j) * kKeys + vt;
          uint32_t s[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t two = 0;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              // a key that no row sees may be uninitialised memory: a zero scale
              // keeps 0 * NaN out of the sum
              const int n = 2 * i + e;
              const uint32_t b =
                  lds8(raw + H::kRawVs + (8 * n + (lane & 7)) * 4 + (lane >> 3));
              two |= (v_ok && key + n >= t.lo && key + n < t.hi ? b : 0u) << (8 * e);
            }
            s[i] = e4m3x2_to_f16(two);
          }
#pragma unroll 1
          for (int w = 0; w < 2; ++w) {  // eight channels
            uint32_t h[8][4];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              e2m1_to_f16(lds32(raw + H::kRawV + (8 * i + (lane & 7)) * 32 + (lane >> 3) * 8 + 4 * w),
                          h[i]);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int ch = vg * 16 + w * 8 + 2 * q;
#pragma unroll
              for (int o = 0; o < 2; ++o) {
                uint32_t d[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  d[i] = hmul2(__byte_perm(h[2 * i][q], h[2 * i + 1][q], o ? 0x7632 : 0x5410), s[i]);
                sts128(sm_v + st * H::kK + swizzled(ch + o, vt / 8, D), d[0], d[1], d[2], d[3]);
              }
            }
          }
        }
        ptx::fence_proxy_async();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(bars.v_full[st]));
        copy_v(j + 1);
      }
      if (!ok) break;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kMmaRegs));
    if (!planned && warp == kMmaWarp + 1) pdl_enter();
  }
  if (kPart == kPrefix && warp == kMmaWarp + 2) {
    // ------------------------------------------------------ the copying warp
    // A tile lies on up to eight pages, one per lane: a bulk copy of the codes and
    // one of the scales of keys, then of values.
    const KvBlock blk = kv_block(a.page_size, D);
    const int seg = min(a.page_size, kKeys), segs = kKeys / seg;
    uint32_t issued = 0, kc = 0;
    bool ok = true;
    begin();
    while (ok && next()) {
      const int32_t* pages = a.page_table + static_cast<long>(t.sq.first_key) * a.max_pages;
      auto page_of = [&](int j) {
        const int key = (t.first + j) * kKeys + lane * seg;
        return lane < segs && j < t.tiles && key < t.hi ? pages[key / a.page_size] : 0;
      };
      int id = page_of(0);
#pragma unroll 1
      for (int j = 0; ok && j < t.tiles; ++j, ++kc) {
        const int key = (t.first + j) * kKeys + lane * seg;
        const bool wanted = lane < segs && key < t.hi;
        const bool good = wanted && id >= 0 && id < a.num_pages;
        const unsigned bad = __ballot_sync(~0u, wanted && !good);
        const int copies = __popc(__ballot_sync(~0u, good));
        const uint8_t* block =
            a.cache + (static_cast<long>(good ? id : 0) * a.kv_heads + t.kvh) * blk.bytes;
        const int row = key & (a.page_size - 1);
        id = page_of(j + 1);
        if (bad && lane == 0) atomicOr(status, MOE_DEV_BAD_PAGE);
        if (lane < 4) {  // 32 tokens each
          uint32_t bits = 0;
          for (int i = 0; i < segs; ++i)
            if ((bad >> i) & 1u)
              bits |= low_bits((i + 1) * seg - 32 * lane) & ~low_bits(i * seg - 32 * lane);
          *reinterpret_cast<volatile uint32_t*>(&s_bad[kc % kBadTiles][lane]) = bits;
        }
        __syncwarp();
#pragma unroll 1
        for (int v = 0; v < 2; ++v) {
          const uint32_t slot = issued % kParts;
          if (!(ok = wait_warp(bars.raw_empty[slot], ((issued / kParts) & 1) ^ 1))) break;
          ++issued;
          const uint32_t full = bar(bars.raw_full[slot]), dst = sm_raw + slot * H::kPartBytes;
          if (lane == 0) ptx::mbar_arrive_expect_tx(full, copies * seg * (D / 2 + D / 16));
          __syncwarp();
          if (good) {
            ptx::bulk_load(dst + lane * seg * (D / 2), block + (v ? blk.v_code : 0) + row * (D / 2),
                           seg * (D / 2), full);
            ptx::bulk_load(dst + H::kCodes + lane * seg * (D / 16),
                           block + (v ? blk.v_scale : blk.k_scale) + row * (D / 16),
                           seg * (D / 16), full);
          }
        }
      }
    }
    // what was asked for has to land before the CTA's shared memory is given up
    for (uint32_t i = issued > kParts ? issued - kParts : 0; i < issued; ++i)
      ptx::mbar_wait_drain(bar(bars.raw_full[i % kParts]), (i / kParts) & 1);
  }
  if (warp == kMmaWarp) {
    // -------------------------------------------------------- the matrix warp
    // The whole warp walks the loop and one elected lane issues: only in code
    // that all lanes run can the operands stay in uniform registers (otherwise
    // issuing takes 60 to 100 cycles per instruction, more than executing).
    uint32_t kc = 0, q_phase = 0, p_phase = 0;
    const uint32_t id_s = ptx::idesc_make(0, kHalf, kKeys), id_o = ptx::idesc_make(0, kHalf, D);
    auto scores = [&](int x, uint32_t st) {
      const uint64_t da = ptx::sdesc_sw128(sm_q + x * H::kQ);
      const uint64_t db = ptx::sdesc_sw128(sm_k + st * H::kK);
      const uint32_t d = tmem + kColsS + x * kKeys;
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)  // 16-byte units: panels, 32 bytes within one
          ptx::tc_mma<false>(d, da + (kk / 4) * (kHalf * 8) + (kk % 4) * 2,
                             db + (kk / 4) * (kKeys * 8) + (kk % 4) * 2, id_s, kk > 0);
        ptx::tc_commit(bar(bars.s_full[x]));
      }
      __syncwarp();
    };
    begin();
    while (next()) {
      const int halves = __shfl_sync(~0u, t.halves, 0), tiles = __shfl_sync(~0u, t.tiles, 0);
      if (tiles == 0) continue;
      const bool keys = kByKeys && __shfl_sync(~0u, static_cast<int>(by_keys()), 0);
      const int both = keys ? 2 : halves;
      bool ok = true;
#pragma unroll 1
      for (int x = 0; ok && x < both; ++x) ok = wait_warp(bars.q_ready[x], (q_phase >> x) & 1);
      q_phase ^= (1u << both) - 1u;
      if constexpr (kByKeys) {
        if (keys) {
          // scores of the first two tiles, then P V of a tile and the scores of the
          // next but one, by the halves in turn: two chains that overlap
          for (int j = 0; ok && j < 2; ++j) {
            const uint32_t n = kc + j;
            if (!(ok = wait_warp(bars.k_full[n & 1], (n >> 1) & 1))) break;
            ptx::tc_fence_after();
            scores(j, n & 1);
          }
#pragma unroll 1
          for (int j = 0; ok && j < tiles; ++j) {
            const uint32_t n = kc + j, st = n & 1, x = j & 1;
            if (!(ok = wait_warp(bars.v_full[st], (n >> 1) & 1) &&
                       wait_warp(bars.p_ready[x], (p_phase >> x) & 1)))
              break;
            p_phase ^= 1u << x;
            ptx::tc_fence_after();
            const uint64_t db = ptx::sdesc_sw128(sm_v + st * H::kK);
            const uint32_t d = tmem + kColsO + x * D, p = tmem + kColsS + x * kKeys;
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < kKeys / 16; ++kk)
                mma_ts(d, p + kk * 8, db + (kk / 4) * (D * 8) + (kk % 4) * 2, id_o, j / 2 + kk > 0);
              ptx::tc_commit(bar(bars.v_empty[st]));
              if (j + 2 >= tiles) ptx::tc_commit(bar(bars.o_done[x]));
            }
            __syncwarp();
            if (j + 2 < tiles) {
              if (!(ok = wait_warp(bars.k_full[st], ((n + 2) >> 1) & 1))) break;
              ptx::tc_fence_after();
              scores(x, st);
            }
          }
          if (!ok) break;
          kc += tiles;
          continue;
        }
      }
      ok = ok && wait_warp(bars.k_full[kc & 1], (kc >> 1) & 1);
      if (!ok) break;
      ptx::tc_fence_after();
#pragma unroll 1
      for (int x = 0; x < halves; ++x) scores(x, kc & 1);
#pragma unroll 1
      for (int j = 0; ok && j < tiles; ++j, ++kc) {
        const bool again = j + 1 < tiles;
        const uint32_t st = kc & 1, nst = (kc + 1) & 1;
        if (!(ok = wait_warp(bars.v_full[st], (kc >> 1) & 1))) break;
#pragma unroll 1
        for (int x = 0; x < halves; ++x) {
          if (!(ok = wait_warp(bars.p_ready[x], (p_phase >> x) & 1))) break;
          ptx::tc_fence_after();
          const uint64_t db = ptx::sdesc_sw128(sm_v + st * H::kK);
          const uint32_t d = tmem + kColsO + x * D, p = tmem + kColsS + x * kKeys;
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < kKeys / 16; ++kk)
              mma_ts(d, p + kk * 8, db + (kk / 4) * (D * 8) + (kk % 4) * 2, id_o, j + kk > 0);
            if (!again) ptx::tc_commit(bar(bars.o_done[x]));
          }
          __syncwarp();
          // S takes the place of the P that the products before it read: matrix
          // instructions of one thread run in the order of issue
          if (again) {
            if (x == 0 && !(ok = wait_warp(bars.k_full[nst], ((kc + 1) >> 1) & 1))) break;
            scores(x, nst);
          }
        }
        p_phase ^= (1u << halves) - 1u;
      }
      if (!ok) break;
    }
    // whatever was issued has to land before the tensor memory is given back
    if (elect_one()) ptx::tc_commit(bar(bars.drain));
    __syncwarp();
    ptx::mbar_wait_drain(bar(bars.drain), 0);
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == kMmaWarp) ptx::tmem_dealloc(tmem, 512);
}

}  // namespace prompt
}  // namespace
}  // namespace moe
