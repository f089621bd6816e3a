// Attention over the 4-bit paged cache: the split kernel.
//
// A work unit is a tile of 32 cached tokens of one (request, row tile, kv
// head) segment; a row is one (query token, query head of the group) pair and
// a row tile has 4, 8 or 16 of them. All segments' tiles form one list, which is
// cut into equal ranges, one per CTA, so that requests of any lengths fill the
// GPU evenly. A CTA whose range covers a segment writes its rows, others leave
// fp32 partial sums and statistics, which the last CTA of the segment joins in
// CTA order (the result does not depend on who is last).
//
// Few rows read many bytes, so the cache's bandwidth bounds this kernel and
// the arithmetic has to hide behind it. A warp reads its codes straight
// into the operands of the matrix instruction: the k index of
// S^T = K Q^T and the m index of O^T = V^T P^T may be permuted freely as long
// as both operands agree, so a lane takes D/4 neighbouring channels of two key
// rows and D/8 neighbouring channels of four value rows, whole words of codes
// under one or two scales. Codes times scales are exact in f16. The codes come
// through a ring of tiles in shared memory that belongs to the warp alone, so
// that enough bytes are on the way without registers and without barriers.
//
// Measured (bf16, 32 query and 8 kv heads of 128): 8 requests of 131071 tokens
// 226 us, 5.3 TB/s of codes (79 % of a copy's rate); 64 requests of 1 to 16384
// tokens 38 us; one request of 1000 tokens (16 and 2 heads) 8.5 us, a chain of
// dependent loads. Instruction issue is the bound: 331 warp instructions per 16
// tokens, 65 % of the issue slots while an SM is busy, the half-rate pipe that
// converts codes at 56 %. One vote and one set of copies per 32 tokens instead
// of 16: 237 us, from 259 with as many bytes on the way. Four CTAs per SM: five
// were no faster, and three stages of 32 tokens (three CTAs fit) took 304 us.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "attn_dev.cuh"
#include "attn_groups.cuh"
#include "launch.cuh"
#include "ptx.cuh"

namespace moe {
namespace {
namespace split {

constexpr int kSub = 16;    // cached tokens per matrix instruction, never across pages
constexpr int kTile = 32;   // cached tokens per tile: what a warp takes at a time
constexpr int kWarps = 4;   // per CTA; each takes every fourth tile of a segment
constexpr int kThreads = kWarps * 32;
// Smallest range of a CTA: a tile for each warp. One request of 1000 tokens takes
// 9.9 us with two tiles, 8.5 with four and 8.8 with eight, one of 4096 tokens
// 13.2, 10.7 and 10.3, one of 300 tokens 7.4, 7.2 and 7.9; long lists do not notice.
constexpr int kMinTiles = kWarps;
// A segment's set-up (its queries, the join of the warps, its rows' stores)
// takes a CTA as long as this many tiles; the list counts them. (64 requests
// of 1 to 16384 tokens: 47.4 us with 5, 43.7 with 7, 41.2 with 9.)
constexpr int kSetup = 9;
constexpr int kStages = 2;  // tiles a warp has in shared memory or on the way
constexpr int kMaxCtasPerSm = 4;
constexpr int kJoin = 16;  // pieces whose sums the joining CTA loads together (ten pieces
                           // of 16 rows: 57 us; one by one, after their statistics, 68)
constexpr int kPlanThreads = 1024;
// Up to so many requests are planned by every CTA itself, more by the kernel
// before: 17.3 against 20.4 us (21 requests), 40.9 and 42.7 (64), 35.7 and 37.2
// (256 of 200 tokens). Beyond, the lists would take the ring's shared memory.
constexpr int kInlineSeqs = 256;

// Checks every request and sums up the work list with a block of N threads:
// starts[b] is the first tile of request b in it. Each thread gets the MOE_DEV_*
// flags of the requests it checked.
template <int N>
__device__ __forceinline__ unsigned sum_work(const AttnArgs& a, int row_tile, SeqInfo* info,
                                             long* starts) {
  __shared__ long warp_sum[N / 32];
  const int g = a.heads / a.kv_heads;
  unsigned flags = 0;
  long base = 0;
  for (int b0 = 0; b0 < a.B; b0 += N) {
    const int b = b0 + threadIdx.x;
    long tiles = 0;
    if (b < a.B) {
      const SeqInfo s = seq_info(a, b, flags);
      info[b] = s;
      const long row_tiles = (static_cast<long>(s.q_len) * g + row_tile - 1) / row_tile;
      const int per = (s.len + kTile - 1) / kTile - s.first_key / kTile;
      tiles = row_tiles * a.kv_heads * (kSetup + (per < 0 ? 0 : per));
    }
    const long before = block_scan<N>(tiles, warp_sum, base);
    if (b < a.B) starts[b] = before;
  }
  if (threadIdx.x == 0) starts[a.B] = base;
  return flags;
}

// Clears the status and the counters, and with `info` sums up the work. (For
// few requests every CTA of the split kernel does that itself, sooner than a
// kernel before it could hand it over; its first loads then overlap this one.)
__global__ void __launch_bounds__(kPlanThreads)
    attn_plan_kernel(AttnArgs a, int row_tile, unsigned* status, int* counters, int n_counters,
                     SeqInfo* info, long* starts) {
  pdl_enter();
  if (threadIdx.x == 0) *status = 0;
  for (int i = threadIdx.x; i < n_counters; i += blockDim.x) counters[i] = 0;
  if (!info) return;
  __syncthreads();
  const unsigned flags = sum_work<kPlanThreads>(a, row_tile, info, starts);
  if (flags) atomicOr(status, flags);
}

// Tiles per CTA: CTA c takes [c * per, (c + 1) * per) of the list, but a cut
// that falls into a segment's first kSetup entries, which stand for no tiles,
// moves to its beginning.
__device__ __forceinline__ long range_len(long total, int ctas) {
  const long per = (total + ctas - 1) / ctas;
  return per < kMinTiles ? kMinTiles : per;
}

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Transposes an 8x8 matrix of f16 held by the warp (two neighbours per lane).
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// N scale bytes of neighbouring groups.
template <int N>
__device__ __forceinline__ uint32_t load_scales(const uint8_t* p) {
  if constexpr (N == 4) return *reinterpret_cast<const uint32_t*>(p);
  if constexpr (N == 2) return *reinterpret_cast<const uint16_t*>(p);
  return *p;
}

template <int D>
struct KeyRegs {
  Words<D / 32> k[2];  // key rows g, g + 8 of a sub-tile: D/4 channels
  uint32_t s[2];
};
template <int D>
struct ValueRegs {
  Words<D / 64> v[4];  // value rows 2c, 2c+1, 2c+8, 2c+9: D/8 channels
  uint32_t s[4];
};

// A sub-tile in shared memory: the rows of key codes, value codes, key scales and
// value scales. Value rows are swizzled (bits 5 and 6 of the offset), so that
// the four even or odd rows that a quarter of the lanes reads lie in different
// banks.
template <int D>
struct TileBytes {
  static constexpr int kRow = D / 2, kScales = D / kKvGroup;
  static constexpr int kCodes = kSub * kRow, kAllScales = kSub * kScales;
  static constexpr int kV = kCodes, kKs = 2 * kCodes, kVs = kKs + kAllScales;
  static constexpr int kBytes = kVs + kAllScales, kTileBytes = kTile / kSub * kBytes;
  __device__ static constexpr uint32_t value(int row, int byte) {
    return static_cast<uint32_t>((row * kRow + byte) ^ (((row >> 1) & 3) << 5));
  }
};

// Copies a sub-tile (rows row0 .. row0 + 15 of a block) into its place.
template <int D>
__device__ __forceinline__ void copy_tile(uint32_t stage, const uint8_t* block, int page_size,
                                          int row0, int lane) {
  using B = TileBytes<D>;
  const KvBlock blk = kv_block(page_size, D);
  const uint8_t* k = block + row0 * B::kRow;
  const uint8_t* v = k + blk.v_code;
#pragma unroll
  for (int i = lane; i < B::kCodes / 16; i += 32) ptx::cp_async16(stage + 16 * i, k + 16 * i);
#pragma unroll
  for (int i = lane; i < B::kCodes / 16; i += 32)
    ptx::cp_async16(stage + B::kV + B::value(16 * i / B::kRow, 16 * i % B::kRow), v + 16 * i);
  constexpr int kChunks = B::kAllScales / 16;
  if (lane < 2 * kChunks) {
    const uint32_t off = lane < kChunks ? blk.k_scale : blk.v_scale;
    ptx::cp_async16(stage + B::kKs + 16 * lane,
                    block + off + row0 * B::kScales + 16 * (lane < kChunks ? lane : lane - kChunks));
  }
}

// The codes and scales of a staged sub-tile for lane (g, c) = (lane / 4, lane % 4).
template <int D>
__device__ __forceinline__ void load_keys(KeyRegs<D>& t, const uint8_t* stage, int g, int c) {
  using B = TileBytes<D>;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = g + 8 * i;
    t.k[i] = load_words<D / 32>(stage + r * B::kRow + c * (D / 8));
    t.s[i] = load_scales<D / 64>(stage + B::kKs + r * B::kScales + c * (D / 64));
  }
}
template <int D>
__device__ __forceinline__ void load_values(ValueRegs<D>& t, const uint8_t* stage, int g, int c) {
  using B = TileBytes<D>;
  constexpr int kVs = D >= 128 ? D / 128 : 1;  // scales a lane's value channels fall under
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 2 * c + (i & 1) + 8 * (i >> 1);
    t.v[i] = load_words<D / 64>(stage + B::kV + B::value(r, g * (D / 16)));
    t.s[i] = load_scales<kVs>(stage + B::kVs + r * B::kScales + g * D / 8 / kKvGroup);
  }
}

// Where the sums of one of a request's rows over the shared prefix lie: n pieces
// in slots of CTAs that follow one another (two slots each; the first one's piece
// is in its second), or one whole row (n 1, no slots between). With `twice` 1, a
// slot has two parts of a piece, one after the other, and n counts parts.
struct RowPieces {
  const float2* stat;
  const float4* sum;
  int n, part_rows, twice;
};
__device__ __forceinline__ RowPieces find_pieces(const PrefixSums& p, long per, const OwnPrefix& own,
                                                 int at, int kvh, int kv_heads, long at_row,
                                                 int chunks) {
  if (own.len == 0) return {nullptr, nullptr, 0, 0, 0};
  const int tile = at / p.shape.tile_rows, r = at - tile * p.shape.tile_rows;
  const bool half = own.rows - tile * p.shape.tile_rows <= p.shape.half_rows;  // the last one
  const int len = half ? own.half_len : own.len;
  const long seg = own.base + static_cast<long>(tile) * kv_heads * own.len + static_cast<long>(kvh) * len;
  const long cta0 = quotient(seg + p.lo, per), cta1 = quotient(seg + len - p.hi, per);
  if (cta1 <= cta0) return {p.row_stats + at_row, p.row_sums + sums_at(at_row, 0, chunks), 1, 0, 0};
  const long rows = 2 * cta0 * p.shape.tile_rows;
  return {p.stats + rows + r, p.sums + rows * chunks + sums_at(r, 0, chunks),
          static_cast<int>(cta1 - cta0 + 1) << half, half ? p.shape.half_rows : p.shape.tile_rows,
          half};
}

// Four channels (chunk c) of those sums, pieces in CTA order, added to the row's own.
__device__ __forceinline__ void add_pieces(const RowPieces& p, int chunks, int c, float4& sum,
                                           float& top, float& den) {
  constexpr int kBatch = 10;  // pieces asked for together
  const int n = p.n, twice = p.twice;
  const long rows = p.part_rows, slot = rows * chunks;
  const float2* stat = p.stat;
  const float4* v0 = p.sum + 8 * c;
  for (int k0 = 0; k0 < n; k0 += kBatch) {
    float2 st[kBatch];
    float4 v[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int k = k0 + i;
      st[i] = make_float2(-INFINITY, 0.0f);
      v[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (k < n) {
        // slot 2 (k >> twice), and 1 instead of 0, part k & twice
        const int at = 2 * k - (k & twice) + (i <= 1 && k <= twice ? 1 + twice : 0);
        st[i] = __ldcg(stat + at * rows);
        v[i] = __ldcg(v0 + at * slot);
      }
    }
    float most = top;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) most = fmaxf(most, st[i].x);
    const float f = top == -INFINITY ? 0.0f : ex2(top - most);
    den *= f, sum.x *= f, sum.y *= f, sum.z *= f, sum.w *= f;
    top = most;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const float g = st[i].x == -INFINITY ? 0.0f : ex2(st[i].x - most);
      den += g * st[i].y;
      sum.x += g * v[i].x, sum.y += g * v[i].y, sum.z += g * v[i].z, sum.w += g * v[i].w;
    }
  }
}

template <int D, int kRows>
__host__ __device__ constexpr int split_smem() {
  constexpr int stages = kWarps * kStages * TileBytes<D>::kTileBytes, sums = kWarps * kRows * D * 4;
  constexpr int join = kAttnMaxSms * (kRows == 16 ? 2 : kMaxCtasPerSm) * kRows * 8;
  constexpr int most = stages > sums ? stages : sums;
  return (most > join ? most : join) + kWarps * kRows * 8;
}
template <int D, int kRows, int kTerms>
__host__ __device__ constexpr int ctas_per_sm() {
  if (D == 256) return 2;
  // as many as fit without spills: 16 rows of 128 channels take 68 us with two and
  // 74 with three, fp32 rows of 64 channels 49 with two and 45 with three. With 256
  // channels 16 bf16 rows spill up to 176 bytes and 8 fp32 rows 116 at the 255 registers
  // that a thread has at most, with any number of CTAs; over own keys, with the place of
  // the prefix's sums, 336 and 164.
  return kRows == 16 || (kTerms == 2 && D == 128) ? 2 : kTerms == 2 ? 3 : kMaxCtasPerSm;
}

// kRows is 4, 8 or 16. The matrix instruction pairs neighbouring k indices in
// a register, and codes come as pairs of neighbouring channels of one token, so
// for O^T the k index runs over (token, parity of the channel) and the m index
// over channel pairs: P of a token stands at one parity and zero at the other,
// one set of columns for even and one for odd channels. No value has to change
// places then. With 4 rows, both sets fit the instruction's 8 columns.
//
// kTerms = 1: q and P are one f16 each (q bf16: exact). kTerms = 2 (fp32
// layers): q and P are a sum of two f16 each, 22 bits, and the products of 32
// channels (scores) or of 16 tokens (sums), the low terms before the high ones,
// are added to the running value by fp32 additions, because the matrix unit's
// own accumulation truncates. (All D channels of both terms in one accumulator
// lost up to 18.4 * 2^-23 of a score at 256 channels, now 4.6; the additions cost
// 8 requests of 8 to 16 thousand tokens 39.6 us instead of 39.1, with 128 channels.)
//
// kPart kPrefix: a request is a group of requests here, its first_key names the
// row of the page table. kOwn: lists of the kernel two places before, so that it
// waits for the prefix kernel as late as a kInline one for the clearing kernel.
template <typename T, int D, int kRows, int kTerms, bool kInline, int kPart = kWhole>
__global__ void __launch_bounds__(kThreads, (ctas_per_sm<D, kRows, kTerms>()))
    attn_split_kernel(AttnArgs a, unsigned* status, int* counters, const SeqInfo* info_in,
                      const long* starts_in, float* stats, float* partial, int page_shift,
                      PartArgs<kPart> part) {
  constexpr bool kBoth = kRows == 4;             // columns 4-7 repeat rows 0-3
  constexpr int NT = kBoth ? 1 : kRows / 8;      // column tiles of the scores
  constexpr int NP = kBoth ? 1 : 2 * NT;         // column tiles of the sums
  constexpr int kVs = D >= 128 ? D / 128 : 1;
  // The warps' stages; after a segment's last tile [kWarps][kRows][D] sums in
  // their place. Behind them [kWarps][kRows][2] statistics.
  extern __shared__ __align__(16) float smem[];
  float* s_stat = smem + split_smem<D, kRows>() / 4 - kWarps * kRows * 2;
  __shared__ int s_last;
  const SeqInfo* info = info_in;
  const long* starts = starts_in;
  // The kernel before this one only clears status and counters, which are not
  // touched before the first segment's join: everything else that is read was
  // written before that kernel began, and the wait for it comes that late.
  bool entered = !kInline && kPart == kWhole;
  unsigned flags = 0;
  if constexpr (kInline) {
    __shared__ SeqInfo s_info[kInlineSeqs];
    __shared__ long s_starts[kInlineSeqs + 1];
    flags = sum_work<kThreads>(a, kRows, s_info, s_starts);
    if (blockIdx.x != 0) flags = 0;  // one CTA reports the requests
    __syncthreads();
    info = s_info;
    starts = s_starts;
  } else if (kPart == kWhole) {
    pdl_enter();
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int group = a.heads / a.kv_heads;
  const KvBlock blk = kv_block(a.page_size, D);
  long total, per;
  int piece = 0;  // kOwn: segments are whole pieces of so many tiles, without set-up entries
  if constexpr (kPart == kPrefix) {
    __shared__ GroupSmem s_groups;
    __shared__ long s_sum[kWarps];
    info = part.p.groups;
    starts = part.p.bases;
    if (part.p.gr.n <= kSmallGroups) {
      unsigned reported = 0;  // by the plan
      plan_groups<kThreads>(a, part.p.gr, part.p.shape, s_groups.lists(), &s_groups, s_sum, reported,
                            [](int, const SeqInfo&, int) {});
      info = s_groups.groups;
      starts = s_groups.bases;
    } else {
      pdl_enter();
      entered = true;
    }
    total = starts[part.p.gr.n];
    per = prefix_per(part.p.shape, total);
  } else if constexpr (kPart == kOwn) {
    total = starts[a.B];
    per = part.p.head->own_per;
    piece = part.p.head->own_piece;
  } else {
    total = starts[a.B];
    per = range_len(total, gridDim.x);
  }
  long at = blockIdx.x * per;
  const long end = min(total, at + per);
  // the request of the first tile: the last b with starts[b] <= at (requests
  // without query rows have no tiles and share their start with the next)
  int b = 0;
  if constexpr (kPart == kOwn) {
    b = part.p.begins[blockIdx.x];
  } else if constexpr (kPart == kPrefix) {
    b = last_at_most(starts, part.p.gr.n, at);
  } else {
    int lo = 0, hi = a.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (starts[mid] <= at) lo = mid;
      else hi = mid;
    }
    b = lo;
  }
  // the segment of the first tile; later segments follow by counting
  long seg_start = -1;
  int row_tile = 0, kvh = 0;
  while (at < end) {
    const SeqInfo sq = info[b];
    const int first_tile = kPart == kPrefix ? 0 : sq.first_key / kTile;
    const int rows = sq.q_len * group;
    int per_seg = max(0, (sq.len + kTile - 1) / kTile - first_tile);
    const int setup = kPart == kOwn && piece > 0 ? 0 : kSetup;
    if (setup == 0)
      per_seg = max(1, (per_seg + piece - 1) / piece) * piece;
    else
      per_seg += kSetup;
    if (seg_start < 0) {
      const long seg = (at - starts[b]) / per_seg;
      seg_start = starts[b] + seg * per_seg;
      row_tile = static_cast<int>(seg / a.kv_heads);
      kvh = static_cast<int>(seg - static_cast<long>(row_tile) * a.kv_heads);
    }
    const long seg_end = seg_start + per_seg;
    if (at - seg_start < setup) at = seg_start;
    if (end - seg_start < setup) break;  // a later CTA takes all of it
    // this CTA's part [p0, p1) of the segment's list, and of its tiles
    const int p0 = static_cast<int>(at - seg_start);
    const int p1 = static_cast<int>(min(seg_end, end) - seg_start);
    const int t0 = max(0, p0 - setup), t1 = p1 - setup;
    const int row0 = row_tile * kRows;
    auto token_of = [&](int r) { return sq.q_len == 1 ? 0 : r / group; };

    // this lane's score columns are rows nt*8 + 2c and + 1: their token limits
    int last[NT][2], first[NT][2];
    int tile_first, tile_last, all_first, all_last;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = row0 + nt * 8 + (kBoth ? (2 * c + j) & 3 : 2 * c + j);
        // padding rows (zero queries whose columns are never written) see all
        const int p = kPart == kPrefix ? sq.len - 1 : sq.len - sq.q_len + token_of(r);
        last[nt][j] = r < rows ? p : 0x7fffffff;
        first[nt][j] = r < rows && a.window > 0 ? max(0, p - a.window + 1) : 0;
      }
    {
      const int r_end = min(rows, row0 + kRows) - 1;
      int pos0 = sq.len - 1, pos1 = sq.len - 1;
      if constexpr (kPart != kPrefix) {
        pos0 = sq.len - sq.q_len + token_of(row0);
        pos1 = sq.len - sq.q_len + token_of(r_end);
      }
      tile_last = pos1;
      tile_first = a.window > 0 ? max(0, pos0 - a.window + 1) : 0;
      // tokens that every row of the tile sees
      all_last = pos0;
      all_first = a.window > 0 ? max(0, pos1 - a.window + 1) : 0;
    }

    // tiles of this row tile that hold a visible token
    const int tA = max(t0, tile_first / kTile - first_tile);
    const int tB = min(t1, tile_last < 0 ? 0 : tile_last / kTile + 1 - first_tile);
    const int32_t* pages =
        a.page_table + static_cast<long>(kPart == kPrefix ? sq.first_key : b) * a.max_pages;
    // The CTA's warps take the tiles of the range in turn. Each keeps a ring of
    // kStages tiles: the copies run kStages - 1 tiles ahead, the page ids one
    // more. The two sub-tiles may lie on two pages.
    constexpr int kSubs = kTile / kSub;
    uint8_t* ring = reinterpret_cast<uint8_t*>(smem) + warp * kStages * TileBytes<D>::kTileBytes;
    const uint32_t ring_addr = ptx::smem_u32(ring);
    auto pages_of = [&](int t) {  // (0 for a sub-tile that no row sees)
      int2 ids = make_int2(0, 0);
      if (t < tB) {
        const int tok = (t + first_tile) * kTile;
        if (tok + kSub > tile_first) ids.x = pages[tok >> page_shift];
        if (tok + kSub <= tile_last)
          ids.y = page_shift == 4 ? pages[(tok + kSub) >> 4] : pages[tok >> page_shift];
      }
      return ids;
    };
    uint32_t ok_bits = 0;  // by stage and sub-tile: the page id was good
    auto copy = [&](int t, int stage, int2 ids) {
      if (t < tB) {
        const int row = ((t + first_tile) * kTile) & ((1 << page_shift) - 1);
#pragma unroll
        for (int sub = 0; sub < kSubs; ++sub) {
          const int id = sub ? ids.y : ids.x;
          const bool ok = id >= 0 && id < a.num_pages;
          if (!ok) flags |= MOE_DEV_BAD_PAGE;
          const uint32_t bit = 1u << (stage * kSubs + sub);
          ok_bits = ok ? ok_bits | bit : ok_bits & ~bit;
          copy_tile<D>(ring_addr + stage * TileBytes<D>::kTileBytes + sub * TileBytes<D>::kBytes,
                       a.cache + (static_cast<long>(ok ? id : 0) * a.kv_heads + kvh) * blk.bytes,
                       a.page_size, page_shift == 4 ? 0 : row + sub * kSub, lane);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    int t = tA + warp;
    int2 ids[kStages - 1];
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) ids[i] = pages_of(t + i * kWarps);
    // The queries' rows (padding rows are zero) are on the way while the first
    // tiles are asked for.
    constexpr int kQWords = D / 4 * static_cast<int>(sizeof(T)) / 4;
    Words<kQWords> raw[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = row0 + nt * 8 + (kBoth ? g & 3 : g);
      if (r < rows) {
        const int tok = token_of(r), h = kvh * group + (r - tok * group);
        raw[nt] = load_words<kQWords>(reinterpret_cast<const uint8_t*>(
            static_cast<const T*>(a.q.p) + (sq.q0 + tok) * a.q.token + h * a.q.head + c * (D / 4)));
      } else {
#pragma unroll
        for (int i = 0; i < kQWords; ++i) raw[nt].w[i] = 0;
      }
    }
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) copy(t + i * kWarps, i, ids[i]);
    int2 next_ids = pages_of(t + (kStages - 1) * kWarps);
    // (where the prefix's sums lie is known before they are there)
    __shared__ RowPieces s_pieces[kPart == kOwn ? kRows : 1];
    if constexpr (kPart == kOwn) {
      const int r = row0 + lane, tok = token_of(r);
      if (warp == kWarps - 1 && lane < kRows && r < rows) {  // it has the fewest tiles
        const OwnPrefix own = part.p.own[b];
        s_pieces[lane] = find_pieces(
            part.p, part.p.head->per, own, own.tok0 * group + r, kvh, a.kv_heads,
            static_cast<long>(sq.q0 + tok) * a.heads + kvh * group + r - tok * group, D / 4);
      }
    }

    // q^T as the B operand: column g (+ 8 nt), channels c*D/4 ..
    uint32_t qf[kTerms][NT][D / 8];
    float q_gain[NT];  // 2^-x of the row g (+ 8 nt) this lane loads
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float x[D / 4];
      if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          x[2 * i] = __uint_as_float(raw[nt].w[i] << 16);
          x[2 * i + 1] = __uint_as_float(raw[nt].w[i] & 0xffff0000u);
        }
      } else {
#pragma unroll
        for (int i = 0; i < D / 4; ++i) x[i] = __uint_as_float(raw[nt].w[i]);
      }
      float top = 0.0f;
#pragma unroll
      for (int i = 0; i < D / 4; ++i) top = fmaxf(top, fabsf(x[i]));
      top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
      top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
      float up;
      row_power(top, up, q_gain[nt]);
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        const float lo = x[2 * i] * up, hi = x[2 * i + 1] * up;
        qf[0][nt][i] = pack_f16(lo, hi);
        if constexpr (kTerms == 2) {
          const float2 f = unpack_f16(qf[0][nt][i]);
          qf[1][nt][i] = pack_f16(lo - f.x, hi - f.y);
        }
      }
    }
    // the gains of this lane's score columns, with the softmax scale
    float gain[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        gain[nt][j] = score_gain(__shfl_sync(~0u, q_gain[nt], (2 * c + j) * 4), a.scale_log2);

    float o[D / 32][NP][4];
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int np = 0; np < NP; ++np)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][np][j] = 0.0f;
    float m[NT][2], base[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) m[nt][j] = -INFINITY, base[nt][j] = -kLift, l[nt][j] = 0.0f;

    for (int stage = 0; t < tB; t += kWarps, stage = stage + 1 == kStages ? 0 : stage + 1) {
      __syncwarp();  // every lane has read the stage that is copied to next
      copy(t + (kStages - 1) * kWarps, stage == 0 ? kStages - 1 : stage - 1, next_ids);
      next_ids = pages_of(t + kStages * kWarps);
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
      __syncwarp();  // every lane's copies of this tile have landed
      const uint32_t oks = (ok_bits >> (stage * kSubs)) & ((1u << kSubs) - 1u);
      const uint8_t* here = ring + stage * TileBytes<D>::kTileBytes;
      const int tok0 = (t + first_tile) * kTile;
      const bool whole =
          oks == (1u << kSubs) - 1u && tok0 >= all_first && tok0 + kTile - 1 <= all_last;

      float s[kSubs][NT][4];
#pragma unroll
      for (int sub = 0; sub < kSubs; ++sub) {
        KeyRegs<D> cur;
        load_keys<D>(cur, here + sub * TileBytes<D>::kBytes, g, c);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[sub][nt][j] = 0.0f;
        uint32_t ks2[2][(D + 127) / 128];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < (D + 127) / 128; ++j) ks2[i][j] = e4m3x2_to_f16(cur.s[i] >> (16 * j));
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {  // 8 channels of each row: two k steps
          uint32_t k0[4], k1[4];
          e2m1_to_f16(cur.k[0].w[w], k0);
          e2m1_to_f16(cur.k[1].w[w], k1);
          const int sc = w / 2;  // the scale these channels fall under
          const uint32_t s0 =
              sc & 1 ? f16_high_twice(ks2[0][sc / 2]) : f16_low_twice(ks2[0][sc / 2]);
          const uint32_t s1 =
              sc & 1 ? f16_high_twice(ks2[1][sc / 2]) : f16_low_twice(ks2[1][sc / 2]);
          uint32_t af[2][4];
#pragma unroll
          for (int hstep = 0; hstep < 2; ++hstep) {
            af[hstep][0] = hmul2(k0[2 * hstep], s0), af[hstep][1] = hmul2(k1[2 * hstep], s1);
            af[hstep][2] = hmul2(k0[2 * hstep + 1], s0), af[hstep][3] = hmul2(k1[2 * hstep + 1], s1);
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float(&acc)[4] = s[sub][nt];
            if constexpr (kTerms == 1) {
#pragma unroll
              for (int hstep = 0; hstep < 2; ++hstep)
                mma(acc, af[hstep], qf[0][nt][4 * w + 2 * hstep], qf[0][nt][4 * w + 2 * hstep + 1]);
            } else {
              float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
              for (int term = kTerms - 1; term >= 0; --term)
#pragma unroll
                for (int hstep = 0; hstep < 2; ++hstep)
                  mma(d, af[hstep], qf[term][nt][4 * w + 2 * hstep],
                      qf[term][nt][4 * w + 2 * hstep + 1]);
#pragma unroll
              for (int j = 0; j < 4; ++j) acc[j] += d[j];
            }
          }
        }
      }
      if (!whole) {
#pragma unroll
        for (int sub = 0; sub < kSubs; ++sub)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int tok = tok0 + sub * kSub + g + 8 * (j >> 1);
              if (!((oks >> sub) & 1u) || tok < first[nt][j & 1] || tok > last[nt][j & 1])
                s[sub][nt][j] = -INFINITY;
            }
      }
      // [j]: column 2c + (j & 1), token g + 8 (j >> 1)
      bool grow = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float x = fmaxf(s[0][nt][j], s[0][nt][j + 2]);
#pragma unroll
          for (int sub = 1; sub < kSubs; ++sub)
            x = fmaxf(x, fmaxf(s[sub][nt][j], s[sub][nt][j + 2]));
          grow |= x * gain[nt][j] > m[nt][j] + kLag;
        }
      if (__any_sync(~0u, grow)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float f[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float x = fmaxf(s[0][nt][j], s[0][nt][j + 2]);
#pragma unroll
            for (int sub = 1; sub < kSubs; ++sub)
              x = fmaxf(x, fmaxf(s[sub][nt][j], s[sub][nt][j + 2]));
            x = fmaxf(x * gain[nt][j], m[nt][j]);
            x = fmaxf(x, __shfl_xor_sync(~0u, x, 4));
            x = fmaxf(x, __shfl_xor_sync(~0u, x, 8));
            x = fmaxf(x, __shfl_xor_sync(~0u, x, 16));
            const float nb = x == -INFINITY ? -kLift : x - kLift;
            f[j] = m[nt][j] == -INFINITY ? 0.0f : ex2(base[nt][j] - nb);
            l[nt][j] *= f[j];
            m[nt][j] = x;
            base[nt][j] = nb;
          }
          // sums' columns are the scores' columns
#pragma unroll
          for (int i = 0; i < D / 32; ++i)
#pragma unroll
            for (int np = nt * (NP / NT); np < (nt + 1) * (NP / NT); ++np)
#pragma unroll
              for (int j = 0; j < 4; ++j) o[i][np][j] *= f[j & 1];
        }
      }
#pragma unroll
      for (int sub = 0; sub < kSubs; ++sub) {
        // P in powers of two over the base, transposed to the B operand
        uint32_t pf[kTerms][NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float p[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            p[j] = ex2(fmaf(s[sub][nt][j], gain[nt][j & 1], -base[nt][j & 1]));
            l[nt][j & 1] += p[j];
          }
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint32_t w = pack_f16(p[2 * half], p[2 * half + 1]);
            pf[0][nt][half] = transpose8x8(w);
            if constexpr (kTerms == 2) {
              const float2 f = unpack_f16(w);
              pf[1][nt][half] = transpose8x8(pack_f16(p[2 * half] - f.x, p[2 * half + 1] - f.y));
            }
          }
        }
        // V^T as the A operand. A token that no row sees may be uninitialised
        // memory: its scale is zeroed, so that 0 * NaN cannot enter the sum.
        ValueRegs<D> cur;
        load_values<D>(cur, here + sub * TileBytes<D>::kBytes, g, c);
        uint32_t vs[4][kVs];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (!whole) {
            const int tok = tok0 + sub * kSub + 2 * c + (i & 1) + 8 * (i >> 1);
            if (!((oks >> sub) & 1u) || tok < tile_first || tok > tile_last) cur.s[i] = 0;
          }
#pragma unroll
          for (int j = 0; j < kVs; ++j)
            vs[i][j] = e4m3x2_to_f16(((cur.s[i] >> (8 * j)) & 0xffu) * 0x101u);
        }
        // P at the columns of one parity: of the even channels, then of the odd
        uint32_t pb[kTerms][2][NP][2];  // [term][half of the tokens][column tile][token 2c, 2c + 1]
#pragma unroll
        for (int term = 0; term < kTerms; ++term)
#pragma unroll
          for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int np = 0; np < NP; ++np) {
              const uint32_t w = pf[term][kBoth ? 0 : np / 2][half];
              const bool odd = kBoth ? g >= 4 : np & 1;
              pb[term][half][np][0] = __byte_perm(w, 0, odd ? 0x1044 : 0x4410);
              pb[term][half][np][1] = __byte_perm(w, 0, odd ? 0x3244 : 0x4432);
            }
#pragma unroll
        for (int w = 0; w < D / 64; ++w) {  // 8 channels: two m tiles
          uint32_t h[4][4];
          const int sc = D == 256 ? w / 2 : 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            e2m1_to_f16(cur.v[i].w[w], h[i]);
#pragma unroll
            for (int q = 0; q < 4; ++q) h[i][q] = hmul2(h[i][q], vs[i][sc]);
          }
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const uint32_t af[2][4] = {
                {h[0][2 * q], h[0][2 * q + 1], h[1][2 * q], h[1][2 * q + 1]},
                {h[2][2 * q], h[2][2 * q + 1], h[3][2 * q], h[3][2 * q + 1]}};
#pragma unroll
            for (int np = 0; np < NP; ++np) {
              float(&acc)[4] = o[2 * w + q][np];
              if constexpr (kTerms == 1) {
                mma(acc, af[0], pb[0][0][np][0], pb[0][0][np][1]);
                mma(acc, af[1], pb[0][1][np][0], pb[0][1][np][1]);
              } else {
                float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int term = kTerms - 1; term >= 0; --term) {
                  mma(d, af[0], pb[term][0][np][0], pb[term][0][np][1]);
                  mma(d, af[1], pb[term][1][np][0], pb[term][1][np][1]);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[j] += d[j];
              }
            }
          }
        }
      }
    }

    // Sums over prefixes are read and written with rows on neighbouring lanes; four
    // channels of a row then move within it, so that the rows use other banks.
    constexpr bool by_rows = kPart != kWhole;
    auto place = [](int r, int ch) { return by_rows ? ch ^ (4 * (r & 7)) : ch; };
    // join the warps: sums [row][channel] and statistics (base, l) in shared
    // memory, in the place of the stages
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (!entered) pdl_enter();
    entered = true;
    __syncthreads();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float x = l[nt][j];
        x += __shfl_xor_sync(~0u, x, 4);
        x += __shfl_xor_sync(~0u, x, 8);
        x += __shfl_xor_sync(~0u, x, 16);
        const int r = kBoth ? (2 * c + j) & 3 : nt * 8 + 2 * c + j;
        if (g == 0 && (!kBoth || c < 2)) {
          s_stat[(warp * kRows + r) * 2] = m[nt][j] == -INFINITY ? -INFINITY : base[nt][j];
          s_stat[(warp * kRows + r) * 2 + 1] = x;
        }
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
#pragma unroll
          for (int up = 0; up < 2; ++up) {
            float* dst = smem + (warp * kRows + r) * D + place(r, g * (D / 8) + 4 * i) + 2 * up;
            if constexpr (kBoth)
              dst[c >> 1] = o[i][0][2 * up + j];
            else
              *reinterpret_cast<float2*>(dst) =
                  make_float2(o[i][2 * nt][2 * up + j], o[i][2 * nt + 1][2 * up + j]);
          }
      }
    __syncthreads();
    const bool alone = p0 == 0 && p1 == per_seg;
    // four channels of a row: the sum of its P V, its base and its sum of P
    auto finish = [&](int r, int ch, float4 sum, float top, float den) {
      const int tok = token_of(row0 + r), h = kvh * group + (row0 + r) - tok * group;
      const long at_row = static_cast<long>(sq.q0 + tok) * a.heads + h;
      if constexpr (kPart == kPrefix) {
        part.p.row_sums[sums_at(at_row, ch / 4, D / 4)] = sum;
        if (ch == 0) part.p.row_stats[at_row] = make_float2(top, den);
        return;
      }
      if constexpr (kPart == kOwn) add_pieces(s_pieces[r], D / 4, ch / 4, sum, top, den);
      const float f = out_factor(den, a.v_scale);
      store4(static_cast<T*>(a.out) + at_row * D + ch,
             make_float4(sum.x * f, sum.y * f, sum.z * f, sum.w * f));
      if (a.lse && ch == 0) a.lse[at_row] = log_sum(top, den);
    };
    // pieces of a segment: the CTA it begins in keeps its piece in slot 1 (its
    // range ends inside the segment), later ones in slot 0
    const long my_slot = 2l * blockIdx.x + (p0 == 0 ? 1 : 0);
    for (int i = threadIdx.x; i < kRows * (D / 4); i += kThreads) {
      const int r = by_rows ? i % kRows : i / (D / 4);
      const int ch = (by_rows ? i / kRows : i % (D / 4)) * 4;
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_stat[(w * kRows + r) * 2]);
      float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      float den = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float b2 = s_stat[(w * kRows + r) * 2];
        const float f = b2 == -INFINITY ? 0.0f : ex2(b2 - top);
        const float4 v = *reinterpret_cast<const float4*>(smem + (w * kRows + r) * D + place(r, ch));
        den += f * s_stat[(w * kRows + r) * 2 + 1];
        sum.x += f * v.x, sum.y += f * v.y, sum.z += f * v.z, sum.w += f * v.w;
      }
      if (alone) {
        if (row0 + r < rows) finish(r, ch, sum, top, den);
      } else {
        if constexpr (kPart == kPrefix)
          reinterpret_cast<float4*>(partial)[sums_at(my_slot * kRows + r, ch / 4, D / 4)] = sum;
        else
          *reinterpret_cast<float4*>(partial + (my_slot * kRows + r) * D + ch) = sum;
        if (ch == 0) {
          stats[(my_slot * kRows + r) * 2] = top;
          stats[(my_slot * kRows + r) * 2 + 1] = den;
        }
      }
    }
    if (kPart != kPrefix && !alone) {
      const int cta0 = static_cast<int>((seg_start + max(0, setup - 1)) / per);
      const int cta1 = static_cast<int>((seg_end - 1) / per);
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0)
        s_last = ptx::add_acq_rel(counters + cta0, 1) == cta1 - cta0;
      __syncthreads();
      if (s_last) {
        __threadfence();
        const int n = cta1 - cta0 + 1;
        const float* first_sum = partial + 2l * cta0 * kRows * D;
        const float* first_stat = stats + 4l * cta0 * kRows;
        auto slot_of = [](int k) { return (2l * k + (k == 0)) * kRows; };
        if (n <= kJoin) {  // statistics and sums are fetched together
          for (int i = threadIdx.x; i < kRows * (D / 4); i += kThreads) {
            const int r = by_rows ? i % kRows : i / (D / 4);
            const int ch = (by_rows ? i / kRows : i % (D / 4)) * 4;
            if (row0 + r >= rows) continue;
            float2 st[kJoin];
            float4 v[kJoin];
#pragma unroll
            for (int k = 0; k < kJoin; ++k) {
              st[k] = make_float2(-INFINITY, 0.0f);
              v[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
              if (k < n) {
                st[k] = __ldcg(reinterpret_cast<const float2*>(first_stat + (slot_of(k) + r) * 2));
                v[k] = __ldcg(reinterpret_cast<const float4*>(first_sum + (slot_of(k) + r) * D + ch));
              }
            }
            float top = -INFINITY, den = 0.0f;
            float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int k = 0; k < kJoin; ++k) top = fmaxf(top, st[k].x);
#pragma unroll
            for (int k = 0; k < kJoin; ++k) {
              const float f = st[k].x == -INFINITY ? 0.0f : ex2(st[k].x - top);
              den += f * st[k].y;
              sum.x += f * v[k].x, sum.y += f * v[k].y, sum.z += f * v[k].z, sum.w += f * v[k].w;
            }
            finish(r, ch, sum, top, den);
          }
        } else {
          // every piece's statistics into shared memory, then its weight
          float* w = smem;                 // [kRows][n] bases, then weights
          float* dens = smem + kRows * n;  // [kRows][n]
          for (int i = threadIdx.x; i < kRows * n; i += kThreads) {
            const int r = i / n, k = i - r * n;
            const float2 st =
                __ldcg(reinterpret_cast<const float2*>(first_stat + (slot_of(k) + r) * 2));
            w[i] = st.x;
            dens[i] = st.y;
          }
          __syncthreads();
          for (int r = warp; r < kRows; r += kWarps) {
            float top = -INFINITY, den = 0.0f;
            for (int k = lane; k < n; k += 32) top = fmaxf(top, w[r * n + k]);
#pragma unroll
            for (int d = 16; d > 0; d /= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
            for (int k = lane; k < n; k += 32) {
              const float b2 = w[r * n + k];
              const float f = b2 == -INFINITY ? 0.0f : ex2(b2 - top);
              w[r * n + k] = f;
              den += f * dens[r * n + k];
            }
#pragma unroll
            for (int d = 16; d > 0; d /= 2) den += __shfl_xor_sync(~0u, den, d);
            __syncwarp();
            if (lane == 0) s_stat[2 * r] = top, s_stat[2 * r + 1] = den;
          }
          __syncthreads();
          for (int i = threadIdx.x; i < kRows * (D / 4); i += kThreads) {
            const int r = by_rows ? i % kRows : i / (D / 4);
            const int ch = (by_rows ? i / kRows : i % (D / 4)) * 4;
            if (row0 + r >= rows) continue;
            float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            for (int k0 = 0; k0 < n; k0 += kJoin) {  // kJoin pieces on the way at a time
              float4 v[kJoin];
#pragma unroll
              for (int j = 0; j < kJoin; ++j) {
                const int k = k0 + j;
                v[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (k < n)
                  v[j] = __ldcg(
                      reinterpret_cast<const float4*>(first_sum + (slot_of(k) + r) * D + ch));
              }
#pragma unroll
              for (int j = 0; j < kJoin; ++j) {
                const float f = k0 + j < n ? w[r * n + k0 + j] : 0.0f;
                sum.x += f * v[j].x, sum.y += f * v[j].y, sum.z += f * v[j].z, sum.w += f * v[j].w;
              }
            }
            finish(r, ch, sum, s_stat[2 * r], s_stat[2 * r + 1]);
          }
        }
      }
    }
    __syncthreads();
    at = seg_start + p1;
    if (p1 == per_seg) {
      seg_start = at;
      if (++kvh == a.kv_heads) kvh = 0, ++row_tile;
      if (at < end && at == starts[b + 1]) {
        while (starts[b + 1] <= at) ++b;
        row_tile = kvh = 0;
      }
    }
  }
  if (!entered) pdl_enter();
  if (flags) atomicOr(status, flags);
}

}  // namespace split
}  // namespace
}  // namespace moe
