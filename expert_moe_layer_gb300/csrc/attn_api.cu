// C ABI of the attention entry points: host validation, rotary frequencies,
// workspace layout and launches. See include/moe.h for the contract of each.
#include <cuda_runtime.h>

#include <cmath>

#include "attn.h"
#include "internal.h"
#include "kv4.cuh"
#include "moe.h"

namespace moe {
namespace {

constexpr int kMaxT = 1 << 18;
constexpr int kMaxTableRows = 1 << 24;
constexpr int kMaxPages = 1 << 20;

#define MOE_TRY(x)                 \
  do {                             \
    const int _rc = (x);           \
    if (_rc != MOE_OK) return _rc; \
  } while (0)

int cuda_ok(cudaError_t e) { return e == cudaSuccess ? MOE_OK : fail_cuda(static_cast<int>(e)); }

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
int ebytes(const moe_attn_config* c) { return c->act_dtype == MOE_BF16 ? 2 : 4; }
int page_shift(const moe_attn_config* c) {
  int n = 0;
  while ((1 << n) < c->page_size) ++n;
  return n;
}
bool scale_ok(float s) { return std::isfinite(s) && s > 0.0f && std::isfinite(1.0f / s); }

// What the rotary calls use: everything but the head counts.
int validate_rope_cfg(const moe_attn_config* c) {
  if (!c) return MOE_ERR_INVALID_ARG;
  if (c->act_dtype != MOE_F32 && c->act_dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if (c->head_dim < 2 || c->head_dim % 2 != 0) return MOE_ERR_INVALID_ARG;
  if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1)) != 0)
    return MOE_ERR_INVALID_ARG;
  if (c->rotary_dim < 0 || c->rotary_dim > c->head_dim || c->rotary_dim % 2 != 0)
    return MOE_ERR_INVALID_ARG;
  if (c->rope_layout != MOE_ROPE_HALF && c->rope_layout != MOE_ROPE_INTERLEAVED)
    return MOE_ERR_INVALID_ARG;
  if (c->rope_positions < 0 || (c->rotary_dim > 0 && c->rope_positions < 1))
    return MOE_ERR_INVALID_ARG;
  if (c->window < 0) return MOE_ERR_INVALID_ARG;
  if (!std::isfinite(c->softmax_scale) || c->softmax_scale < 0.0f) return MOE_ERR_INVALID_ARG;
  if (!scale_ok(c->k_scale) || !scale_ok(c->v_scale)) return MOE_ERR_INVALID_ARG;
  return c->head_dim > 2 * kMaxPairs ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

int validate_cfg(const moe_attn_config* c) {
  const int rc = validate_rope_cfg(c);
  if (rc == MOE_ERR_INVALID_ARG) return rc;
  if (c->num_heads < 1 || c->num_kv_heads < 1 || c->num_heads % c->num_kv_heads != 0)
    return MOE_ERR_INVALID_ARG;
  return c->num_heads > 512 ? MOE_ERR_UNSUPPORTED : rc;
}

bool cache_dim(int D) { return D == 64 || D == 128 || D == 256; }

int validate_cache_cfg(const moe_attn_config* c) {
  MOE_TRY(validate_cfg(c));
  return cache_dim(c->head_dim) ? MOE_OK : MOE_ERR_UNSUPPORTED;
}

// Strides of [T, heads, D] rows: heads and tokens may lie anywhere but must
// not overlap, and stay in the range that 64-bit byte offsets cover.
int validate_rows(const moe_attn_config* c, const void* p, int64_t token, int64_t head,
                  int heads) {
  if (!p || !aligned(p, ebytes(c))) return MOE_ERR_INVALID_ARG;
  const int64_t most = int64_t{1} << 40;
  if (token < 0 || head < 0 || token > most || head > most) return MOE_ERR_INVALID_ARG;
  if (heads > 1 && head < c->head_dim) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

int validate_cache(const void* cache, int64_t num_pages) {
  if (!cache || !aligned(cache, 16)) return MOE_ERR_INVALID_ARG;
  if (num_pages < 1 || num_pages > (int64_t{1} << 31)) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

// The optional status workspace: cleared here, nullptr if there is none.
int clear_status(void* ws, size_t ws_bytes, cudaStream_t st, unsigned** status) {
  *status = nullptr;
  if (!ws) return MOE_OK;
  *status = static_cast<unsigned*>(ws);
  return cuda_ok(cudaMemsetAsync(ws, 0, 4, st));
}
int validate_status_ws(const void* ws, size_t ws_bytes) {
  return ws && (ws_bytes < 4 || !aligned(ws, 4)) ? MOE_ERR_WORKSPACE : MOE_OK;
}

// Radians per position of each pair, and the factor on the table.
int frequencies(int R, const moe_rope_scaling* s, double* f, double* gain) {
  constexpr double kPi = 3.14159265358979323846;
  if (!s || !std::isfinite(s->base) || s->base <= 1.0) return MOE_ERR_INVALID_ARG;
  if (s->kind < MOE_ROPE_SCALE_NONE || s->kind > MOE_ROPE_SCALE_YARN) return MOE_ERR_INVALID_ARG;
  const bool scaled = s->kind != MOE_ROPE_SCALE_NONE;
  if (scaled && (!std::isfinite(s->factor) || s->factor < 1.0)) return MOE_ERR_INVALID_ARG;
  if (!std::isfinite(s->attention_factor) || s->attention_factor < 0.0)
    return MOE_ERR_INVALID_ARG;
  const bool mixed = s->kind == MOE_ROPE_SCALE_PARTS || s->kind == MOE_ROPE_SCALE_YARN;
  const double slow = s->slow_turns == 0.0 ? 1.0 : s->slow_turns;
  const double fast = s->fast_turns != 0.0                  ? s->fast_turns
                      : s->kind == MOE_ROPE_SCALE_YARN ? 32.0
                                                            : 4.0;
  if (mixed && (!std::isfinite(s->original_positions) || s->original_positions <= 0.0 ||
                !std::isfinite(fast) || !(slow > 0.0) || !(fast > slow)))
    return MOE_ERR_INVALID_ARG;
  if (s->kind == MOE_ROPE_SCALE_NTK && R <= 2) return MOE_ERR_INVALID_ARG;
  double base = s->base;
  if (s->kind == MOE_ROPE_SCALE_NTK) base *= std::pow(s->factor, R / (R - 2.0));
  double low = 0.0, high = 1.0;
  if (s->kind == MOE_ROPE_SCALE_YARN) {
    auto pair = [&](double turns) {
      return R * std::log(s->original_positions / (turns * 2.0 * kPi)) / (2.0 * std::log(base));
    };
    low = std::floor(pair(fast));
    high = std::ceil(pair(slow));
    if (high < 0.0) {  // no pair turns as often as slow_turns: f / s for all
      low = -1.0, high = 0.0;
    } else if (low > R - 1.0) {  // every pair turns more often than fast_turns: f for all
      high = low + 1.0;
    } else {
      low = std::fmax(low, 0.0);
      high = std::fmin(high, R - 1.0);
      if (low == high) high += 0.001;
    }
  }
  for (int i = 0; i < R / 2; ++i) {
    const double own = std::pow(base, -2.0 * i / R);
    double keep = 1.0;
    if (s->kind == MOE_ROPE_SCALE_LINEAR) keep = 0.0;
    if (s->kind == MOE_ROPE_SCALE_PARTS)
      keep = (s->original_positions * own / (2.0 * kPi) - slow) / (fast - slow);
    if (s->kind == MOE_ROPE_SCALE_YARN) keep = 1.0 - (i - low) / (high - low);
    keep = std::fmin(std::fmax(keep, 0.0), 1.0);
    f[i] = keep == 1.0 ? own : own * keep + own / s->factor * (1.0 - keep);
  }
  *gain = s->attention_factor != 0.0                 ? s->attention_factor
          : s->kind == MOE_ROPE_SCALE_YARN ? 0.1 * std::log(s->factor) + 1.0
                                                     : 1.0;
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_validate_attn_config(const moe_attn_config* cfg) { return validate_cfg(cfg); }

size_t moe_kv_page_bytes(const moe_attn_config* cfg) {
  if (validate_cache_cfg(cfg) != MOE_OK) return 0;
  return static_cast<size_t>(cfg->num_kv_heads) * kv_block(cfg->page_size, cfg->head_dim).bytes;
}

int moe_rope_table(const moe_attn_config* cfg, int n, const int32_t* positions,
                   const moe_rope_scaling* scaling, float* table, void* ws, size_t ws_bytes,
                   void* stream) {
  MOE_TRY(validate_rope_cfg(cfg));
  const int R = cfg->rotary_dim;
  if (n < 0 || n > kMaxTableRows || R == 0) return MOE_ERR_INVALID_ARG;
  double f[kMaxPairs], gain;
  MOE_TRY(frequencies(R, scaling, f, &gain));
  if (n == 0) return MOE_OK;
  if (!table || !aligned(table, 16) || (positions && !aligned(positions, 4)))
    return MOE_ERR_INVALID_ARG;
  MOE_TRY(validate_status_ws(ws, ws_bytes));
  RopeTurns turns = {};
  for (int i = 0; i < R / 2; ++i) {
    // f < 2 pi (base > 1), so this is below one turn: 64 bits of fraction
    const double part = f[i] / 6.28318530717958647693;
    turns.f[i] = static_cast<unsigned long long>(std::ldexp(part, 64));
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  unsigned* status;
  MOE_TRY(clear_status(ws, ws_bytes, st, &status));
  return cuda_ok(
      launch_rope_table(turns, R / 2, static_cast<float>(gain), n, positions, table, st));
}

int moe_rope(const moe_attn_config* cfg, int T, int num_heads, const void* x,
             int64_t x_token_stride, int64_t x_head_stride, const int32_t* positions,
             const float* table, int inverse, void* out, void* ws, size_t ws_bytes,
             void* stream) {
  MOE_TRY(validate_rope_cfg(cfg));
  if (T < 0 || T > kMaxT || num_heads < 1 || num_heads > 512) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  MOE_TRY(validate_rows(cfg, x, x_token_stride, x_head_stride, num_heads));
  if (!out || !aligned(out, 16)) return MOE_ERR_INVALID_ARG;
  if (out == x && ((T > 1 && x_token_stride != int64_t{num_heads} * cfg->head_dim) ||
                   (num_heads > 1 && x_head_stride != cfg->head_dim)))
    return MOE_ERR_INVALID_ARG;
  if (cfg->rotary_dim > 0 &&
      (!positions || !table || !aligned(positions, 4) || !aligned(table, 16)))
    return MOE_ERR_INVALID_ARG;
  MOE_TRY(validate_status_ws(ws, ws_bytes));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  RopeArgs a;
  MOE_TRY(clear_status(ws, ws_bytes, st, &a.status));
  a.T = T, a.D = cfg->head_dim, a.R = cfg->rotary_dim, a.q_heads = num_heads;
  a.q = {x, static_cast<long>(x_token_stride), static_cast<long>(x_head_stride)};
  a.positions = positions, a.table = table, a.table_rows = cfg->rope_positions;
  a.interleaved = cfg->rope_layout == MOE_ROPE_INTERLEAVED, a.inverse = inverse != 0;
  a.q_out = out;
  return cuda_ok(launch_rope(cfg->act_dtype == MOE_BF16, a, st));
}

int moe_kv_append(const moe_attn_config* cfg, int T, const void* q, int64_t q_token_stride,
                  int64_t q_head_stride, const void* k, int64_t k_token_stride,
                  int64_t k_head_stride, const void* v, int64_t v_token_stride,
                  int64_t v_head_stride, const int32_t* positions, const int64_t* slots,
                  const float* table, void* q_out, void* cache, int64_t num_pages, void* ws,
                  size_t ws_bytes, void* stream) {
  MOE_TRY(validate_cache_cfg(cfg));
  if (T < 0 || T > kMaxT) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  MOE_TRY(validate_rows(cfg, k, k_token_stride, k_head_stride, cfg->num_kv_heads));
  MOE_TRY(validate_rows(cfg, v, v_token_stride, v_head_stride, cfg->num_kv_heads));
  if (q) {
    MOE_TRY(validate_rows(cfg, q, q_token_stride, q_head_stride, cfg->num_heads));
    if (!q_out || !aligned(q_out, 16)) return MOE_ERR_INVALID_ARG;
    if (q_out == q &&
        ((T > 1 && q_token_stride != int64_t{cfg->num_heads} * cfg->head_dim) ||
         (cfg->num_heads > 1 && q_head_stride != cfg->head_dim)))
      return MOE_ERR_INVALID_ARG;
  }
  if (!slots || !aligned(slots, 8)) return MOE_ERR_INVALID_ARG;
  if (cfg->rotary_dim > 0 &&
      (!positions || !table || !aligned(positions, 4) || !aligned(table, 16)))
    return MOE_ERR_INVALID_ARG;
  MOE_TRY(validate_cache(cache, num_pages));
  MOE_TRY(validate_status_ws(ws, ws_bytes));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  RopeArgs a;
  MOE_TRY(clear_status(ws, ws_bytes, st, &a.status));
  a.T = T, a.D = cfg->head_dim, a.R = cfg->rotary_dim;
  a.q_heads = q ? cfg->num_heads : 0, a.kv_heads = cfg->num_kv_heads;
  a.q = {q, static_cast<long>(q_token_stride), static_cast<long>(q_head_stride)};
  a.k = {k, static_cast<long>(k_token_stride), static_cast<long>(k_head_stride)};
  a.v = {v, static_cast<long>(v_token_stride), static_cast<long>(v_head_stride)};
  a.positions = positions, a.slots = slots, a.table = table;
  a.table_rows = cfg->rope_positions;
  a.interleaved = cfg->rope_layout == MOE_ROPE_INTERLEAVED;
  a.q_out = q_out, a.cache = static_cast<uint8_t*>(cache);
  a.page_shift = page_shift(cfg), a.n_slots = static_cast<long>(num_pages) * cfg->page_size;
  a.k_inv = 1.0f / cfg->k_scale, a.v_inv = 1.0f / cfg->v_scale;
  return cuda_ok(launch_rope(cfg->act_dtype == MOE_BF16, a, st));
}

int moe_kv_read(const moe_attn_config* cfg, int N, const int64_t* slots, const void* cache,
                int64_t num_pages, void* k_out, void* v_out, void* ws, size_t ws_bytes,
                void* stream) {
  MOE_TRY(validate_cache_cfg(cfg));
  if (N < 0 || N > kMaxT) return MOE_ERR_INVALID_ARG;
  if (N == 0) return MOE_OK;
  if (!slots || !aligned(slots, 8) || !k_out || !v_out || !aligned(k_out, 16) ||
      !aligned(v_out, 16))
    return MOE_ERR_INVALID_ARG;
  MOE_TRY(validate_cache(cache, num_pages));
  MOE_TRY(validate_status_ws(ws, ws_bytes));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  unsigned* status;
  MOE_TRY(clear_status(ws, ws_bytes, st, &status));
  return cuda_ok(launch_kv_read(cfg->act_dtype == MOE_BF16, N, slots,
                                static_cast<const uint8_t*>(cache),
                                static_cast<long>(num_pages) * cfg->page_size, cfg->num_kv_heads,
                                cfg->head_dim, page_shift(cfg), cfg->k_scale, cfg->v_scale, k_out,
                                v_out, status, st));
}

static int validate_attention(const moe_attn_config* cfg, int num_seqs, int T, int max_q_len) {
  MOE_TRY(validate_cache_cfg(cfg));
  if (T < 0 || T > kMaxT || num_seqs < 0 || num_seqs > kMaxT || max_q_len < 0)
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

size_t moe_kv_attention_workspace_size(const moe_attn_config* cfg, int num_seqs, int T,
                                       int max_q_len) {
  if (validate_attention(cfg, num_seqs, T, max_q_len) != MOE_OK) return 0;
  return attn_layout(cfg, num_seqs, T, max_q_len).total;
}

// What moe_kv_attention and moe_kv_attention_shared are handed alike, checked;
// the workspace aside.
static int attention_args(const moe_attn_config* cfg, int num_seqs, int T, int max_q_len,
                          const void* q, int64_t q_token_stride, int64_t q_head_stride,
                          const int32_t* q_offsets, const int32_t* seq_lens,
                          const int32_t* page_table, int max_pages, const void* cache,
                          int64_t num_pages, void* out, float* lse, AttnArgs* args) {
  const int eb = ebytes(cfg);
  MOE_TRY(validate_rows(cfg, q, q_token_stride, q_head_stride, cfg->num_heads));
  if (!aligned(q, 16) || q_token_stride * eb % 16 != 0 || q_head_stride * eb % 16 != 0)
    return MOE_ERR_INVALID_ARG;
  if (num_seqs < 1 || max_q_len < 1 || max_pages < 1 || max_pages > kMaxPages)
    return MOE_ERR_INVALID_ARG;
  if (!q_offsets && num_seqs != T) return MOE_ERR_INVALID_ARG;
  if (!seq_lens || !page_table || !out || !aligned(out, 16) || !aligned(seq_lens, 4) ||
      !aligned(page_table, 4) || !aligned(q_offsets, 4) || !aligned(lse, 4))
    return MOE_ERR_INVALID_ARG;
  MOE_TRY(validate_cache(cache, num_pages));
  AttnArgs& a = *args;
  a.B = num_seqs, a.T = T, a.max_q = max_q_len;
  a.heads = cfg->num_heads, a.kv_heads = cfg->num_kv_heads;
  a.D = cfg->head_dim, a.page_size = cfg->page_size;
  // A request has at most a table row's tokens, so that a window of as many is no
  // limit. Positions lie between -2^18 and 2^28 and so do the windows left: a
  // position less a window stays within 32 bits in the kernels.
  a.window = cfg->window < int64_t{max_pages} * cfg->page_size ? cfg->window : 0;
  const float scale =
      cfg->softmax_scale > 0.0f ? cfg->softmax_scale
                                : 1.0f / std::sqrt(static_cast<float>(cfg->head_dim));
  a.scale_log2 = static_cast<float>(1.4426950408889634 * scale * cfg->k_scale);
  a.v_scale = cfg->v_scale;
  a.q = {q, static_cast<long>(q_token_stride), static_cast<long>(q_head_stride)};
  a.q_offsets = q_offsets, a.seq_lens = seq_lens, a.page_table = page_table;
  a.max_pages = max_pages;
  a.cache = static_cast<const uint8_t*>(cache), a.num_pages = static_cast<long>(num_pages);
  a.out = out, a.lse = lse;
  return MOE_OK;
}

static int attention_sms(AttnArgs* a) {
  a->sms = sm_count();
  if (a->sms < 1) return MOE_ERR_CUDA;
  if (a->sms > kAttnMaxSms) a->sms = kAttnMaxSms;
  return MOE_OK;
}

int moe_kv_attention(const moe_attn_config* cfg, int num_seqs, int T, int max_q_len,
                     const void* q, int64_t q_token_stride, int64_t q_head_stride,
                     const int32_t* q_offsets, const int32_t* seq_lens,
                     const int32_t* page_table, int max_pages, const void* cache,
                     int64_t num_pages, void* out, float* lse, void* ws, size_t ws_bytes,
                     void* stream) {
  MOE_TRY(validate_attention(cfg, num_seqs, T, max_q_len));
  if (T == 0) return MOE_OK;
  AttnArgs a;
  MOE_TRY(attention_args(cfg, num_seqs, T, max_q_len, q, q_token_stride, q_head_stride, q_offsets,
                         seq_lens, page_table, max_pages, cache, num_pages, out, lse, &a));
  const AttnLayout L = attn_layout(cfg, num_seqs, T, max_q_len);
  if (!ws || ws_bytes < L.total || !aligned(ws, 16)) return MOE_ERR_WORKSPACE;
  MOE_TRY(attention_sms(&a));
  return cuda_ok(launch_kv_attention(cfg, a, ws, L, static_cast<cudaStream_t>(stream)));
}

static int validate_groups(int num_groups, int max_group_len) {
  return num_groups < 0 || num_groups > kMaxT || max_group_len < 0 ? MOE_ERR_INVALID_ARG : MOE_OK;
}

size_t moe_kv_attention_shared_workspace_size(const moe_attn_config* cfg, int num_seqs, int T,
                                              int max_q_len, int num_groups, int max_group_len) {
  if (validate_attention(cfg, num_seqs, T, max_q_len) != MOE_OK ||
      validate_groups(num_groups, max_group_len) != MOE_OK)
    return 0;
  const size_t plain = attn_layout(cfg, num_seqs, T, max_q_len).total;
  if (!can_share(cfg, max_q_len, num_groups)) return plain;
  const size_t shared = shared_layout(cfg, num_seqs, T, num_groups, max_group_len).total;
  return shared > plain ? shared : plain;
}

int moe_kv_attention_shared(const moe_attn_config* cfg, int num_seqs, int T, int max_q_len,
                            int num_groups, int max_group_len, const void* q,
                            int64_t q_token_stride, int64_t q_head_stride,
                            const int32_t* q_offsets, const int32_t* seq_lens,
                            const int32_t* page_table, int max_pages,
                            const int32_t* group_offsets, const int32_t* prefix_lens,
                            const void* cache, int64_t num_pages, void* out, float* lse, void* ws,
                            size_t ws_bytes, void* stream) {
  MOE_TRY(validate_attention(cfg, num_seqs, T, max_q_len));
  MOE_TRY(validate_groups(num_groups, max_group_len));
  if (T == 0) return MOE_OK;
  AttnArgs a;
  MOE_TRY(attention_args(cfg, num_seqs, T, max_q_len, q, q_token_stride, q_head_stride, q_offsets,
                         seq_lens, page_table, max_pages, cache, num_pages, out, lse, &a));
  if (num_groups > 0 && (!group_offsets || !prefix_lens || !aligned(group_offsets, 4) ||
                         !aligned(prefix_lens, 4) || max_group_len < 1))
    return MOE_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (!ws || !aligned(ws, 16) ||
      ws_bytes < moe_kv_attention_shared_workspace_size(cfg, num_seqs, T, max_q_len, num_groups,
                                                        max_group_len))
    return MOE_ERR_WORKSPACE;
  MOE_TRY(attention_sms(&a));
  if (!can_share(cfg, max_q_len, num_groups) ||
      !worth_sharing(cfg, num_seqs, max_q_len, max_pages))
    return cuda_ok(
        launch_kv_attention(cfg, a, ws, attn_layout(cfg, num_seqs, T, max_q_len), st));
  const SharedLayout L = shared_layout(cfg, num_seqs, T, num_groups, max_group_len);
  return cuda_ok(launch_kv_attention_shared(cfg, a, num_groups, group_offsets, prefix_lens,
                                            max_group_len, ws, L, st));
}

}  // extern "C"
