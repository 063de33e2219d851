// The C ABI of the attention side (declared in include/nvfp4_attn.h): argument
// validation, status codes and dispatch to the kernel launchers, as abi.cpp does
// for the weight products.  Nothing here allocates or synchronises.
#include <hip/hip_runtime_api.h>

#include <cmath>
#include <cstdint>

#include "../../include/nvfp4_attn.h"
#include "abi_common.h"
#include "attn_launchers.h"

namespace {

using nvfp4::aligned;
using nvfp4::aligned16;
using nvfp4::aligned4;
using nvfp4::fail;
using nvfp4::hip_status;
using nvfp4::ok;

constexpr int64_t kMaxTokens = int64_t(1) << 24;  // rows of one call: grids stay below 2^32 threads
constexpr int64_t kMaxHeads = 32768;

static_assert(NVFP4_KV_BF16 == nvfp4::kKvBf16 && NVFP4_KV_E4M3 == nvfp4::kKvE4m3 && NVFP4_KV_NVFP4 == nvfp4::kKvNvfp4,
              "formats");
static_assert(NVFP4_ATTN_COUNTER_BYTES == nvfp4::kAttnCounterBytes, "counters");

int check_head_dim(int64_t d) {
  if (d < 16 || d > 256 || d % 16 != 0)
    return fail(NVFP4_ERR_SHAPE, "head_dim=%lld must be a multiple of 16 in [16, 256]", (long long)d);
  return NVFP4_OK;
}

int check_tokens(int64_t tokens) {
  if (tokens < 0 || tokens > kMaxTokens) return fail(NVFP4_ERR_SHAPE, "tokens=%lld out of range", (long long)tokens);
  return NVFP4_OK;
}

int check_dtype(int dtype, const char* what) {
  if (dtype != NVFP4_F32 && dtype != NVFP4_BF16) return fail(NVFP4_ERR_DTYPE, "unknown %s %d", what, dtype);
  return NVFP4_OK;
}

// A leading dimension of rows of `n` elements.
int check_ld(int64_t ld, int64_t n, const char* what) {
  if (ld < n || ld % 8 != 0 || ld > nvfp4::kMaxDim)
    return fail(NVFP4_ERR_SHAPE, "%s=%lld must be >= %lld, a multiple of 8 and at most 2^30", what, (long long)ld,
                (long long)n);
  return NVFP4_OK;
}

int check_rope(int64_t rot_dim, int64_t head_dim, int layout, float magnitude) {
  if (rot_dim < 0 || rot_dim > head_dim || rot_dim % 16 != 0)
    return fail(NVFP4_ERR_SHAPE, "rot_dim=%lld must be a multiple of 16 in [0, head_dim=%lld]", (long long)rot_dim,
                (long long)head_dim);
  if (layout != NVFP4_ROPE_HALF && layout != NVFP4_ROPE_INTERLEAVED)
    return fail(NVFP4_ERR_ARG, "unknown rotary layout %d", layout);
  if (!std::isfinite(magnitude)) return fail(NVFP4_ERR_ARG, "magnitude must be finite");
  return NVFP4_OK;
}

int check_cache(const nvfp4_kv_cache* c, bool need_pool) {
  if (!c) return fail(NVFP4_ERR_NULL, "cache is NULL");
  if (c->format != NVFP4_KV_BF16 && c->format != NVFP4_KV_E4M3 && c->format != NVFP4_KV_NVFP4)
    return fail(NVFP4_ERR_DTYPE, "unknown cache format %d", c->format);
  NVFP4_TRY(check_head_dim(c->head_dim));
  if (c->page_size < 16 || c->page_size > 65536 || c->page_size % 16 != 0)
    return fail(NVFP4_ERR_SHAPE, "page_size=%lld must be a multiple of 16 in [16, 65536]", (long long)c->page_size);
  if (c->kv_heads < 1 || c->kv_heads > 1024)
    return fail(NVFP4_ERR_SHAPE, "kv_heads=%lld must be in [1, 1024]", (long long)c->kv_heads);
  if (c->pages < 1 || c->pages > (int64_t(1) << 34) / c->page_size / c->kv_heads)
    return fail(NVFP4_ERR_SHAPE, "pages=%lld must be >= 1, and pages * page_size * kv_heads at most 2^34",
                (long long)c->pages);
  const float lo = 5.42101086e-20f, hi = 1.84467441e19f;  // 2^-64, 2^64: no product of scales leaves fp32's normal range
  if (c->format == NVFP4_KV_NVFP4) {
    if (!(c->k_scale >= lo && c->k_scale <= hi && c->v_scale >= lo && c->v_scale <= hi))
      return fail(NVFP4_ERR_ARG, "k_scale and v_scale must be in [2^-64, 2^64]");
  } else if (c->k_scale != 1.0f || c->v_scale != 1.0f) {
    return fail(NVFP4_ERR_ARG, "k_scale and v_scale must be 1 for this cache format");
  }
  if (!need_pool) return NVFP4_OK;
  if (!c->pool) return fail(NVFP4_ERR_NULL, "cache->pool is NULL");
  if (!aligned16(c->pool)) return fail(NVFP4_ERR_ALIGN, "cache->pool must be 16-byte aligned");
  return NVFP4_OK;
}

int64_t groups_of(const nvfp4_kv_cache* c) { return c->pages * c->kv_heads * (c->page_size / nvfp4::kKvGroup); }

nvfp4::KvCache cache_of(const nvfp4_kv_cache* c) {
  nvfp4::KvCache r;
  const int db = (int)((c->head_dim + 63) / 64);
  const size_t code_bytes = nvfp4::kv_code_bytes(c->format, db);
  r.codes = static_cast<uint8_t*>(c->pool);
  r.scales = r.codes ? r.codes + (size_t)groups_of(c) * code_bytes : nullptr;  // no pool: sizes only
  r.slots = c->pages * c->page_size;
  r.pages = (int32_t)c->pages;
  r.heads = (int32_t)c->kv_heads;
  r.head_dim = (int32_t)c->head_dim;
  r.gpp = (int32_t)(c->page_size / nvfp4::kKvGroup);
  r.page_size = (int32_t)c->page_size;
  r.k_scale = c->k_scale;
  r.v_scale = c->v_scale;
  return r;
}

nvfp4::AttnLaunch attn_of(const nvfp4_attn_args* a) {
  nvfp4::AttnLaunch l;
  l.cache = cache_of(a->cache);
  l.format = a->cache->format;
  l.batch = a->batch;
  l.q_heads = (int32_t)a->q_heads;
  l.q = a->q;
  l.ldq = a->ldq;
  l.table = a->page_table;
  l.table_width = a->table_width;
  l.lens = a->seq_lens;
  l.scale = a->scale;
  l.window = (int32_t)(a->window < nvfp4::kMaxDim ? a->window : nvfp4::kMaxDim);
  l.out = a->out;
  l.ldo = a->ldo;
  l.lse = a->lse;
  l.ws = a->workspace;
  return l;
}

int check_attn(const nvfp4_attn_args* a, bool need_buffers) {
  if (!a) return fail(NVFP4_ERR_NULL, "args is NULL");
  NVFP4_TRY(check_cache(a->cache, need_buffers && a->batch > 0));
  if (a->batch < 0 || a->batch > 65536) return fail(NVFP4_ERR_SHAPE, "batch=%lld must be in [0, 65536]", (long long)a->batch);
  if (a->q_heads < 1 || a->q_heads > kMaxHeads || a->q_heads % a->cache->kv_heads != 0)
    return fail(NVFP4_ERR_SHAPE, "q_heads=%lld must be a multiple of kv_heads=%lld, at most %lld", (long long)a->q_heads,
                (long long)a->cache->kv_heads, (long long)kMaxHeads);
  if (a->table_width < 0 || a->table_width > nvfp4::kMaxDim / a->cache->page_size)
    return fail(NVFP4_ERR_SHAPE, "table_width=%lld must be >= 0, and table_width * page_size at most 2^30",
                (long long)a->table_width);
  if (a->window < 0) return fail(NVFP4_ERR_ARG, "window=%lld is negative", (long long)a->window);
  if (!nvfp4::attn_fits(attn_of(a)))
    return fail(NVFP4_ERR_SHAPE, "batch x query rows x table too large: the call would have 2^31 tiles of 32 tokens or more");
  if (!need_buffers || a->batch == 0) return NVFP4_OK;
  if (!(a->scale > 0.0f && a->scale <= 0x1p127f)) return fail(NVFP4_ERR_ARG, "scale must be positive and at most 2^127");
  NVFP4_TRY(check_ld(a->ldq, a->q_heads * a->cache->head_dim, "ldq"));
  NVFP4_TRY(check_ld(a->ldo, a->q_heads * a->cache->head_dim, "ldo"));
  if (!a->q || !a->out || !a->seq_lens || (a->table_width > 0 && !a->page_table))
    return fail(NVFP4_ERR_NULL, "q, page_table, seq_lens and out must be non-NULL");
  if (!aligned16(a->q) || !aligned16(a->out)) return fail(NVFP4_ERR_ALIGN, "q and out must be 16-byte aligned");
  if (!aligned4(a->page_table) || !aligned4(a->seq_lens) || !aligned4(a->lse))
    return fail(NVFP4_ERR_ALIGN, "page_table, seq_lens and lse must be 4-byte aligned");
  return NVFP4_OK;
}

}  // namespace

extern "C" {

int nvfp4_rope_freqs(const nvfp4_rope_config* c, uint64_t* freqs, float* magnitude) {
  NVFP4_GUARD_BEGIN
  if (!c || !magnitude) return fail(NVFP4_ERR_NULL, "config and magnitude must be non-NULL");
  if (c->rot_dim < 0 || c->rot_dim > 256 || c->rot_dim % 16 != 0)
    return fail(NVFP4_ERR_SHAPE, "rot_dim=%lld must be a multiple of 16 in [0, 256]", (long long)c->rot_dim);
  if (!freqs && c->rot_dim != 0) return fail(NVFP4_ERR_NULL, "freqs must be non-NULL");
  if (c->scaling != NVFP4_ROPE_NONE && c->scaling != NVFP4_ROPE_LINEAR && c->scaling != NVFP4_ROPE_YARN)
    return fail(NVFP4_ERR_ARG, "unknown rotary scaling %d", c->scaling);
  if (!(c->base > 1.0) || !std::isfinite(c->base)) return fail(NVFP4_ERR_ARG, "base must be finite and above 1");
  if (c->scaling != NVFP4_ROPE_NONE && (!(c->factor >= 1.0) || !std::isfinite(c->factor)))
    return fail(NVFP4_ERR_ARG, "factor must be finite and at least 1");
  const bool yarn = c->scaling == NVFP4_ROPE_YARN;
  if (yarn && !(c->original_max > 0.0 && std::isfinite(c->original_max) && c->beta_slow > 0.0 &&
                c->beta_fast > c->beta_slow && std::isfinite(c->beta_fast)))
    return fail(NVFP4_ERR_ARG, "YaRN needs original_max > 0 and beta_fast > beta_slow > 0");
  const long double two_pi = 6.283185307179586476925286766559L;
  const long double rot = (long double)c->rot_dim, log_base = logl((long double)c->base);
  long double low = 0.0L, high = 0.0L;
  bool slow = false;  // every pair turns less than beta_slow times
  if (yarn && c->rot_dim > 0) {
    // The (fractional) pair that makes `turns` turns over the original positions.
    const auto pair = [&](double turns) { return rot * logl((long double)c->original_max / (turns * two_pi)) / (2.0L * log_base); };
    low = floorl(pair(c->beta_fast));
    high = ceill(pair(c->beta_slow));
    slow = pair(c->beta_slow) < 0.0L;
    low = low < 0.0L ? 0.0L : low;
    high = high > rot - 1.0L ? rot - 1.0L : high;
  }
  for (int64_t i = 0; i < c->rot_dim / 2; ++i) {
    long double f = expl(-2.0L * (long double)i / rot * log_base) / two_pi;
    if (c->scaling == NVFP4_ROPE_LINEAR) f /= (long double)c->factor;
    if (yarn) {
      long double width = high - low, ramp;
      width = width < 0.001L ? 0.001L : width;
      ramp = ((long double)i - low) / width;
      ramp = slow ? 1.0L : ramp < 0.0L ? 0.0L : ramp > 1.0L ? 1.0L : ramp;
      f = f * (1.0L - ramp) + f / (long double)c->factor * ramp;
    }
    freqs[i] = (uint64_t)roundl(f * 18446744073709551616.0L);  // f < 0.16
  }
  *magnitude = yarn && c->factor > 1.0 ? (float)(0.1 * std::log(c->factor) + 1.0) : 1.0f;
  return ok();
  NVFP4_GUARD_END
}

int nvfp4_rope(const nvfp4_rope_args* a, void* stream) {
  NVFP4_GUARD_BEGIN
  if (!a) return fail(NVFP4_ERR_NULL, "args is NULL");
  NVFP4_TRY(check_tokens(a->tokens));
  NVFP4_TRY(check_head_dim(a->head_dim));
  if (a->heads < 0 || a->heads > kMaxHeads) return fail(NVFP4_ERR_SHAPE, "heads=%lld out of range", (long long)a->heads);
  NVFP4_TRY(check_rope(a->rot_dim, a->head_dim, a->layout, a->magnitude));
  NVFP4_TRY(check_dtype(a->x_dtype, "x_dtype"));
  NVFP4_TRY(check_dtype(a->y_dtype, "y_dtype"));
  if (a->tokens == 0 || a->heads == 0) return ok();
  NVFP4_TRY(check_ld(a->ldx, a->heads * a->head_dim, "ldx"));
  NVFP4_TRY(check_ld(a->ldy, a->heads * a->head_dim, "ldy"));
  if (!a->x || !a->y || (a->rot_dim > 0 && (!a->positions || !a->freqs)))
    return fail(NVFP4_ERR_NULL, "x, y, positions and freqs must be non-NULL");
  if (!aligned16(a->x) || !aligned16(a->y)) return fail(NVFP4_ERR_ALIGN, "x and y must be 16-byte aligned");
  if (!aligned4(a->positions) || !aligned(a->freqs, 8))
    return fail(NVFP4_ERR_ALIGN, "positions must be 4-byte and freqs 8-byte aligned");
  if (a->x == a->y && (a->x_dtype != a->y_dtype || a->ldx != a->ldy))
    return fail(NVFP4_ERR_ARG, "in place, x and y must have the same dtype and leading dimension");
  nvfp4::RopeLaunch l;
  l.rope = nvfp4::Rope{a->freqs, a->positions, (int32_t)a->rot_dim, a->layout == NVFP4_ROPE_INTERLEAVED, a->magnitude,
                       a->inverse ? -1.0f : 1.0f};
  l.tokens = a->tokens;
  l.heads = (int32_t)a->heads;
  l.head_dim = (int32_t)a->head_dim;
  l.x = a->x;
  l.y = a->y;
  l.ldx = a->ldx;
  l.ldy = a->ldy;
  l.x_bf16 = a->x_dtype == NVFP4_BF16;
  l.y_bf16 = a->y_dtype == NVFP4_BF16;
  return hip_status(nvfp4::launch_rope(l, (hipStream_t)stream), "rope launch");
  NVFP4_GUARD_END
}

int nvfp4_kv_cache_bytes(const nvfp4_kv_cache* c, size_t* bytes) {
  NVFP4_GUARD_BEGIN
  if (!bytes) return fail(NVFP4_ERR_NULL, "bytes is NULL");
  NVFP4_TRY(check_cache(c, false));
  *bytes = (size_t)groups_of(c) * nvfp4::kv_group_bytes(c->format, (int)((c->head_dim + 63) / 64));
  return ok();
  NVFP4_GUARD_END
}

int nvfp4_kv_append(const nvfp4_kv_append_args* a, void* stream) {
  NVFP4_GUARD_BEGIN
  if (!a) return fail(NVFP4_ERR_NULL, "args is NULL");
  NVFP4_TRY(check_cache(a->cache, a->tokens > 0));
  NVFP4_TRY(check_tokens(a->tokens));
  NVFP4_TRY(check_dtype(a->dtype, "dtype"));
  const int64_t d = a->cache->head_dim, n = a->cache->kv_heads * d;
  if (a->freqs) NVFP4_TRY(check_rope(a->rot_dim, d, a->layout, a->magnitude));
  if (a->q) {
    if (!a->freqs) return fail(NVFP4_ERR_ARG, "q is turned into q_out: it needs freqs");
    if (a->q_heads < 1 || a->q_heads > kMaxHeads) return fail(NVFP4_ERR_SHAPE, "q_heads=%lld out of range", (long long)a->q_heads);
  }
  if (a->tokens == 0) return ok();
  NVFP4_TRY(check_ld(a->ldk, n, "ldk"));
  NVFP4_TRY(check_ld(a->ldv, n, "ldv"));
  if (!a->slots || !a->k || !a->v) return fail(NVFP4_ERR_NULL, "slots, k and v must be non-NULL");
  if (!aligned16(a->k) || !aligned16(a->v)) return fail(NVFP4_ERR_ALIGN, "k and v must be 16-byte aligned");
  if (!aligned(a->slots, 8)) return fail(NVFP4_ERR_ALIGN, "slots must be 8-byte aligned");
  if (a->freqs) {
    if (!a->positions) return fail(NVFP4_ERR_NULL, "positions must be non-NULL with freqs");
    if (!aligned4(a->positions) || !aligned(a->freqs, 8))
      return fail(NVFP4_ERR_ALIGN, "positions must be 4-byte and freqs 8-byte aligned");
  }
  if (a->q) {
    NVFP4_TRY(check_ld(a->ldq, a->q_heads * d, "ldq"));
    NVFP4_TRY(check_ld(a->ldqo, a->q_heads * d, "ldqo"));
    if (!a->q_out) return fail(NVFP4_ERR_NULL, "q_out must be non-NULL with q");
    if (!aligned16(a->q) || !aligned16(a->q_out)) return fail(NVFP4_ERR_ALIGN, "q and q_out must be 16-byte aligned");
    if (a->q == a->q_out && (a->dtype != NVFP4_BF16 || a->ldq != a->ldqo))
      return fail(NVFP4_ERR_ARG, "in place, q must be bf16 and ldqo equal ldq");
  }
  nvfp4::KvAppendLaunch l;
  l.cache = cache_of(a->cache);
  l.format = a->cache->format;
  l.rope = nvfp4::Rope{a->freqs, a->positions, (int32_t)(a->freqs ? a->rot_dim : 0), a->layout == NVFP4_ROPE_INTERLEAVED,
                       a->magnitude, 1.0f};
  l.tokens = a->tokens;
  l.slots = a->slots;
  l.k = a->k;
  l.v = a->v;
  l.q = a->q;
  l.q_out = a->q_out;
  l.ldk = a->ldk;
  l.ldv = a->ldv;
  l.ldq = a->ldq;
  l.ldqo = a->ldqo;
  l.q_heads = (int32_t)a->q_heads;
  l.bf16 = a->dtype == NVFP4_BF16;
  return hip_status(nvfp4::launch_kv_append(l, (hipStream_t)stream), "kv append launch");
  NVFP4_GUARD_END
}

int nvfp4_kv_read(const nvfp4_kv_cache* c, const int64_t* slots, int64_t tokens, void* k_out, int64_t ldk, void* v_out,
                  int64_t ldv, int out_dtype, void* stream) {
  NVFP4_GUARD_BEGIN
  NVFP4_TRY(check_cache(c, tokens > 0));
  NVFP4_TRY(check_tokens(tokens));
  NVFP4_TRY(check_dtype(out_dtype, "out_dtype"));
  if (tokens == 0 || (!k_out && !v_out)) return ok();
  const int64_t n = c->kv_heads * c->head_dim;
  if (k_out) NVFP4_TRY(check_ld(ldk, n, "ldk"));
  if (v_out) NVFP4_TRY(check_ld(ldv, n, "ldv"));
  if (!slots) return fail(NVFP4_ERR_NULL, "slots must be non-NULL");
  if (!aligned16(k_out) || !aligned16(v_out)) return fail(NVFP4_ERR_ALIGN, "k_out and v_out must be 16-byte aligned");
  if (!aligned(slots, 8)) return fail(NVFP4_ERR_ALIGN, "slots must be 8-byte aligned");
  nvfp4::KvReadLaunch l;
  l.cache = cache_of(c);
  l.format = c->format;
  l.tokens = tokens;
  l.slots = slots;
  l.k = k_out;
  l.v = v_out;
  l.ldk = ldk;
  l.ldv = ldv;
  l.bf16 = out_dtype == NVFP4_BF16;
  return hip_status(nvfp4::launch_kv_read(l, (hipStream_t)stream), "kv read launch");
  NVFP4_GUARD_END
}

int nvfp4_attn_decode_workspace_bytes(const nvfp4_attn_args* a, size_t* bytes) {
  NVFP4_GUARD_BEGIN
  if (!bytes) return fail(NVFP4_ERR_NULL, "bytes is NULL");
  NVFP4_TRY(check_attn(a, false));
  *bytes = a->batch == 0 ? 0 : nvfp4::attn_workspace_bytes(attn_of(a));
  return ok();
  NVFP4_GUARD_END
}

int nvfp4_attn_decode(const nvfp4_attn_args* a, void* stream) {
  NVFP4_GUARD_BEGIN
  NVFP4_TRY(check_attn(a, true));
  if (a->batch == 0) return ok();
  const nvfp4::AttnLaunch l = attn_of(a);
  const size_t need = nvfp4::attn_workspace_bytes(l);
  if (!a->workspace || a->workspace_bytes < need)
    return fail(NVFP4_ERR_WORKSPACE, "workspace of %zu bytes required, %zu given", need, a->workspace ? a->workspace_bytes : 0);
  if (!aligned16(a->workspace)) return fail(NVFP4_ERR_ALIGN, "workspace must be 16-byte aligned");
  return hip_status(nvfp4::launch_attn_decode(l, (hipStream_t)stream), "attention launch");
  NVFP4_GUARD_END
}

}  // extern "C"
