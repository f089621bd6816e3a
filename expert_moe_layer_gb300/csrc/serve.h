// Host-side launch helpers of the norms around a layer's blocks and of the
// pages of a shared cache. See include/moe.h for the contracts.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "moe.h"

namespace moe {

struct NormArgs {
  int T = 0, H = 0;
  const void* y = nullptr;  // nullptr: no block output
  const void* x = nullptr;
  long y_stride = 0, x_stride = 0;  // elements per row
  const float *post_w = nullptr, *post_b = nullptr, *pre_w = nullptr, *pre_b = nullptr;
  const void* gate = nullptr;
  long gate_token = 0;
  int gate_channel = 0;  // 0 or 1
  void *x_out = nullptr, *h = nullptr;
  int layer = 0, post = 0, sigmoid = 0;
  float scale = 1.0f, offset = 0.0f, eps = 0.0f;
};
cudaError_t launch_norm(bool act_bf16, bool res_bf16, const NormArgs& a, int sms, cudaStream_t st);

// The caches (one per layer) that one set of page ids indexes.
struct CacheList {
  int n = 0;
  long page_bytes = 0;
  uint8_t* p[MOE_KV_MAX_CACHES] = {};
};

struct PoolArgs {
  int32_t* table = nullptr;  // [rows, max_pages]
  int32_t* held = nullptr;   // [rows]
  int32_t* refs = nullptr;   // [pages]
  int rows = 0, max_pages = 0, page_shift = 0;  // log2 of the page size
  long pages = 0;
  unsigned* status = nullptr;  // nullptr where a call has no workspace
};

// Pages are looked through in chunks of kScan times a power of two pages, at
// most kMaxChunks of them.
constexpr int kScan = 8192, kMaxChunks = 1024;
inline long pool_chunk(long pages) {
  long c = kScan;
  while ((pages + c - 1) / c > kMaxChunks) c *= 2;
  return c;
}

// Words at the start of the workspace, behind the status.
struct PoolHeader {
  unsigned status;
  int done;    // CTAs that have looked through their chunk
  int free;    // free pages
  int used;    // pages in use
  int moves;   // free pages below `used`: pages that compaction moves
  int copies;  // pages that a reservation copies
};

struct PoolLayout {
  size_t claims, items, copies, prefix, list, ranks, total;
};
PoolLayout pool_layout(long pages, int rows, int n);

// Up to so many items the kernels of fork and release clear the status themselves.
constexpr int kFewItems = 32;
// Clears n words, the first of which is a call's status.
cudaError_t launch_clear(void* words, long n, cudaStream_t st);

// Callers clear the header (and the claims where `rows` is given) first, unless
// pool_clears says that the kernel does so itself.
bool pool_clears(long pages);
cudaError_t launch_reserve(const PoolArgs& a, const CacheList& caches, int n, const int32_t* rows,
                           const int32_t* start, const int32_t* end, void* ws, const PoolLayout& L,
                           int sms, cudaStream_t st);
cudaError_t launch_compact(const PoolArgs& a, const CacheList& caches, int32_t* used, void* ws,
                           const PoolLayout& L, int sms, cudaStream_t st);
cudaError_t launch_fork(const PoolArgs& a, int n, const int32_t* parents, const int32_t* children,
                        const int32_t* tokens, cudaStream_t st);
cudaError_t launch_release(const PoolArgs& a, int n, const int32_t* rows, const int32_t* keep,
                           cudaStream_t st);
cudaError_t launch_copy_pages(const CacheList& from, long from_pages, const CacheList& to,
                              long to_pages, int n, const int32_t* src, const int32_t* dst,
                              unsigned* status, int sms, cudaStream_t st);

}  // namespace moe
