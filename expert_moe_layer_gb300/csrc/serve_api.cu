// C ABI of the shared pages of a cache and of the norms: host validation,
// workspace layout and launches. See include/moe.h for the contract of each.
#include <cuda_runtime.h>

#include <cmath>

#include "internal.h"
#include "kv4.cuh"
#include "moe.h"
#include "serve.h"

namespace moe {
namespace {

constexpr int kMaxItems = 1 << 18, kMaxRows = 1 << 18, kMaxWidth = 1 << 20;
constexpr int64_t kMaxPoolPages = int64_t{1} << 30;
constexpr int kMaxHidden = 16384, kMaxNormRows = 1 << 24;

#define MOE_TRY(x)                 \
  do {                             \
    const int _rc = (x);           \
    if (_rc != MOE_OK) return _rc; \
  } while (0)

int cuda_ok(cudaError_t e) { return e == cudaSuccess ? MOE_OK : fail_cuda(static_cast<int>(e)); }
bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
bool ints(const int32_t* p) { return p && aligned(p, 4); }

int validate_caches(const moe_attn_config* cfg, const moe_kv_caches* c) {
  const size_t bytes = moe_kv_page_bytes(cfg);
  if (bytes == 0) {
    const int rc = moe_validate_attn_config(cfg);
    return rc == MOE_OK ? MOE_ERR_UNSUPPORTED : rc;  // a head_dim without cache kernels
  }
  if (!c || c->num_caches < 1 || c->num_caches > MOE_KV_MAX_CACHES || !c->caches ||
      c->num_pages < 1 || c->num_pages > (int64_t{1} << 31))
    return MOE_ERR_INVALID_ARG;
  for (int i = 0; i < c->num_caches; ++i)
    if (!c->caches[i] || !aligned(c->caches[i], 16)) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

int validate_pool(const moe_attn_config* cfg, const moe_kv_pool* p) {
  if (!p) return MOE_ERR_INVALID_ARG;
  MOE_TRY(validate_caches(cfg, &p->caches));
  if (p->num_rows < 1 || p->num_rows > kMaxRows || p->max_pages < 1 || p->max_pages > kMaxWidth ||
      p->caches.num_pages > kMaxPoolPages)
    return MOE_ERR_INVALID_ARG;
  return ints(p->page_table) && ints(p->held) && ints(p->refs) ? MOE_OK : MOE_ERR_INVALID_ARG;
}
int validate_items(int n) { return n < 0 || n > kMaxItems ? MOE_ERR_INVALID_ARG : MOE_OK; }

CacheList cache_list(const moe_attn_config* cfg, const moe_kv_caches& c) {
  CacheList l;
  l.n = c.num_caches;
  l.page_bytes = static_cast<long>(moe_kv_page_bytes(cfg));
  for (int i = 0; i < l.n; ++i) l.p[i] = static_cast<uint8_t*>(c.caches[i]);
  return l;
}
PoolArgs pool_args(const moe_attn_config* cfg, const moe_kv_pool* p, void* status) {
  PoolArgs a;
  a.table = p->page_table, a.held = p->held, a.refs = p->refs;
  a.rows = p->num_rows, a.max_pages = p->max_pages, a.page_shift = 0;
  while ((1 << a.page_shift) < cfg->page_size) ++a.page_shift;
  a.pages = static_cast<long>(p->caches.num_pages);
  a.status = static_cast<unsigned*>(status);
  return a;
}

int validate_status_ws(const void* ws, size_t ws_bytes) {
  return ws && (ws_bytes < 4 || !aligned(ws, 4)) ? MOE_ERR_WORKSPACE : MOE_OK;
}
int clear_status(void* ws, cudaStream_t st) {
  return ws ? cuda_ok(launch_clear(ws, 1, st)) : MOE_OK;
}
int sms_or_fail(int* sms) {
  *sms = sm_count();
  return *sms < 1 ? MOE_ERR_CUDA : MOE_OK;
}

bool dtype_ok(moe_dtype d) { return d == MOE_F32 || d == MOE_BF16; }
int ebytes(moe_dtype d) { return d == MOE_BF16 ? 2 : 4; }

int validate_norm(const moe_norm_config* c) {
  if (!c || c->hidden_size < 1 || !dtype_ok(c->act_dtype) || !dtype_ok(c->residual_dtype))
    return MOE_ERR_INVALID_ARG;
  if (c->kind != MOE_NORM_RMS && c->kind != MOE_NORM_LAYER) return MOE_ERR_INVALID_ARG;
  if (c->gate != MOE_GATE_LINEAR && c->gate != MOE_GATE_SIGMOID) return MOE_ERR_INVALID_ARG;
  if (!std::isfinite(c->residual_scale) || !std::isfinite(c->weight_offset) ||
      !std::isfinite(c->eps) || c->eps <= 0.0f)
    return MOE_ERR_INVALID_ARG;
  return c->hidden_size > kMaxHidden ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

// Rows of H elements: they do not overlap, and stay within 64-bit byte offsets.
int validate_rows(const void* p, int64_t stride, int H, int T, int bytes) {
  if (!aligned(p, bytes) || stride < 0 || stride > (int64_t{1} << 38)) return MOE_ERR_INVALID_ARG;
  return T > 1 && stride < H ? MOE_ERR_INVALID_ARG : MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_kv_pool_workspace_size(const moe_attn_config* cfg, const moe_kv_pool* pool, int n) {
  if (validate_pool(cfg, pool) != MOE_OK || validate_items(n) != MOE_OK) return 0;
  return pool_layout(static_cast<long>(pool->caches.num_pages), pool->num_rows, n).total;
}

int moe_kv_fork(const moe_attn_config* cfg, const moe_kv_pool* pool, int n, const int32_t* parents,
                const int32_t* children, const int32_t* tokens, void* ws, size_t ws_bytes,
                void* stream) {
  MOE_TRY(validate_pool(cfg, pool));
  MOE_TRY(validate_items(n));
  if (n == 0) return MOE_OK;
  if (!ints(parents) || !ints(children) || !ints(tokens)) return MOE_ERR_INVALID_ARG;
  MOE_TRY(validate_status_ws(ws, ws_bytes));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (n > kFewItems) MOE_TRY(clear_status(ws, st));
  return cuda_ok(launch_fork(pool_args(cfg, pool, ws), n, parents, children, tokens, st));
}

int moe_kv_reserve(const moe_attn_config* cfg, const moe_kv_pool* pool, int n, const int32_t* rows,
                   const int32_t* start, const int32_t* end, void* ws, size_t ws_bytes,
                   void* stream) {
  MOE_TRY(validate_pool(cfg, pool));
  MOE_TRY(validate_items(n));
  if (n == 0) return MOE_OK;
  if (!ints(start) || !ints(end) || (rows && !aligned(rows, 4))) return MOE_ERR_INVALID_ARG;
  if (!rows && n > pool->num_rows) return MOE_ERR_INVALID_ARG;
  const PoolArgs a = pool_args(cfg, pool, ws);
  const PoolLayout L = pool_layout(a.pages, a.rows, n);
  if (!ws || ws_bytes < L.total || !aligned(ws, 16)) return MOE_ERR_WORKSPACE;
  int sms;
  MOE_TRY(sms_or_fail(&sms));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (!pool_clears(a.pages))
    MOE_TRY(cuda_ok(launch_clear(ws, static_cast<long>(L.claims) / 4 + (rows ? a.rows : 0), st)));
  return cuda_ok(
      launch_reserve(a, cache_list(cfg, pool->caches), n, rows, start, end, ws, L, sms, st));
}

int moe_kv_release(const moe_attn_config* cfg, const moe_kv_pool* pool, int n, const int32_t* rows,
                   const int32_t* keep, void* ws, size_t ws_bytes, void* stream) {
  MOE_TRY(validate_pool(cfg, pool));
  MOE_TRY(validate_items(n));
  if (n == 0) return MOE_OK;
  if ((rows && !aligned(rows, 4)) || (keep && !aligned(keep, 4))) return MOE_ERR_INVALID_ARG;
  if (!rows && n > pool->num_rows) return MOE_ERR_INVALID_ARG;
  MOE_TRY(validate_status_ws(ws, ws_bytes));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (n > kFewItems) MOE_TRY(clear_status(ws, st));
  return cuda_ok(launch_release(pool_args(cfg, pool, ws), n, rows, keep, st));
}

int moe_kv_compact(const moe_attn_config* cfg, const moe_kv_pool* pool, int32_t* used, void* ws,
                   size_t ws_bytes, void* stream) {
  MOE_TRY(validate_pool(cfg, pool));
  if (used && !aligned(used, 4)) return MOE_ERR_INVALID_ARG;
  const PoolArgs a = pool_args(cfg, pool, ws);
  const PoolLayout L = pool_layout(a.pages, a.rows, 0);
  if (!ws || ws_bytes < L.total || !aligned(ws, 16)) return MOE_ERR_WORKSPACE;
  int sms;
  MOE_TRY(sms_or_fail(&sms));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (!pool_clears(a.pages)) MOE_TRY(cuda_ok(launch_clear(ws, static_cast<long>(L.claims) / 4, st)));
  return cuda_ok(launch_compact(a, cache_list(cfg, pool->caches), used, ws, L, sms, st));
}

int moe_kv_copy_pages(const moe_attn_config* cfg, const moe_kv_caches* from,
                      const moe_kv_caches* to, int n, const int32_t* src, const int32_t* dst,
                      void* ws, size_t ws_bytes, void* stream) {
  MOE_TRY(validate_caches(cfg, from));
  MOE_TRY(validate_caches(cfg, to));
  if (from->num_caches != to->num_caches) return MOE_ERR_INVALID_ARG;
  MOE_TRY(validate_items(n));
  if (n == 0) return MOE_OK;
  if (!ints(src) || !ints(dst)) return MOE_ERR_INVALID_ARG;
  MOE_TRY(validate_status_ws(ws, ws_bytes));
  int sms;
  MOE_TRY(sms_or_fail(&sms));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  MOE_TRY(clear_status(ws, st));
  return cuda_ok(launch_copy_pages(cache_list(cfg, *from), static_cast<long>(from->num_pages),
                                   cache_list(cfg, *to), static_cast<long>(to->num_pages), n, src,
                                   dst, static_cast<unsigned*>(ws), sms, st));
}

int moe_validate_norm_config(const moe_norm_config* cfg) { return validate_norm(cfg); }

int moe_norm(const moe_norm_config* cfg, int T, const void* y, int64_t y_stride, const void* x,
             int64_t x_stride, const float* post_w, const float* post_b, const void* gate,
             int64_t gate_token_stride, int64_t gate_channel_stride, const float* pre_w,
             const float* pre_b, void* x_out, void* h, void* ws, size_t ws_bytes, void* stream) {
  MOE_TRY(validate_norm(cfg));
  if (T < 0 || T > kMaxNormRows) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  const int H = cfg->hidden_size, ab = ebytes(cfg->act_dtype), rb = ebytes(cfg->residual_dtype);
  if (!x || (!x_out && !h)) return MOE_ERR_INVALID_ARG;
  if (!y && (post_w || post_b || gate || x_out)) return MOE_ERR_INVALID_ARG;
  MOE_TRY(validate_rows(x, x_stride, H, T, rb));
  if (y) MOE_TRY(validate_rows(y, y_stride, H, T, ab));
  for (const void* p : {static_cast<const void*>(post_w), static_cast<const void*>(post_b),
                        static_cast<const void*>(pre_w), static_cast<const void*>(pre_b),
                        static_cast<const void*>(x_out), static_cast<const void*>(h)})
    if (!aligned(p, 16)) return MOE_ERR_INVALID_ARG;
  if (gate) {
    if (!aligned(gate, ab) || gate_token_stride < 0 || gate_token_stride > (int64_t{1} << 38) ||
        gate_channel_stride < 0 || gate_channel_stride > 1)
      return MOE_ERR_INVALID_ARG;
  }
  if (T > 1 && ((x_out == x && x_stride != H) || (h && h == y && y_stride != H)))
    return MOE_ERR_INVALID_ARG;
  if ((h && h == x) || (x_out && x_out == y) || (h && h == x_out)) return MOE_ERR_INVALID_ARG;
  MOE_TRY(validate_status_ws(ws, ws_bytes));
  int sms;
  MOE_TRY(sms_or_fail(&sms));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  MOE_TRY(clear_status(ws, st));
  NormArgs a;
  a.T = T, a.H = H, a.y = y, a.x = x;
  a.y_stride = static_cast<long>(y_stride), a.x_stride = static_cast<long>(x_stride);
  a.post_w = post_w, a.post_b = post_b, a.pre_w = pre_w, a.pre_b = pre_b;
  a.gate = gate, a.gate_token = static_cast<long>(gate_token_stride);
  a.gate_channel = static_cast<int>(gate_channel_stride);
  a.x_out = x_out, a.h = h;
  a.layer = cfg->kind == MOE_NORM_LAYER, a.post = cfg->post_norm != 0;
  a.sigmoid = cfg->gate == MOE_GATE_SIGMOID;
  a.scale = cfg->residual_scale, a.offset = cfg->weight_offset, a.eps = cfg->eps;
  return cuda_ok(
      launch_norm(cfg->act_dtype == MOE_BF16, cfg->residual_dtype == MOE_BF16, a, sms, st));
}

}  // extern "C"
