// Checks of arguments and descriptors that the files of the attention side's C ABI share.
#pragma once

#include <cmath>
#include <cstdint>

#include "../../include/nvfp4_attn.h"
#include "abi_common.h"
#include "attn_launchers.h"

namespace nvfp4 {

constexpr int64_t kMaxTokens = int64_t(1) << 24;  // rows of one call: grids stay below 2^32 threads
constexpr int64_t kMaxHeads = 32768;

inline int check_head_dim(int64_t d) {
  if (d < 16 || d > 256 || d % 16 != 0)
    return fail(NVFP4_ERR_SHAPE, "head_dim=%lld must be a multiple of 16 in [16, 256]", (long long)d);
  return NVFP4_OK;
}

inline int check_tokens(int64_t tokens) {
  if (tokens < 0 || tokens > kMaxTokens) return fail(NVFP4_ERR_SHAPE, "tokens=%lld out of range", (long long)tokens);
  return NVFP4_OK;
}

inline int check_dtype(int dtype, const char* what) {
  if (dtype != NVFP4_F32 && dtype != NVFP4_BF16) return fail(NVFP4_ERR_DTYPE, "unknown %s %d", what, dtype);
  return NVFP4_OK;
}

// A leading dimension of rows of `n` elements.
inline int check_ld(int64_t ld, int64_t n, const char* what) {
  if (ld < n || ld % 8 != 0 || ld > kMaxDim)
    return fail(NVFP4_ERR_SHAPE, "%s=%lld must be >= %lld, a multiple of 8 and at most 2^30", what, (long long)ld,
                (long long)n);
  return NVFP4_OK;
}

inline int check_rope(int64_t rot_dim, int64_t head_dim, int layout, float magnitude) {
  if (rot_dim < 0 || rot_dim > head_dim || rot_dim % 16 != 0)
    return fail(NVFP4_ERR_SHAPE, "rot_dim=%lld must be a multiple of 16 in [0, head_dim=%lld]", (long long)rot_dim,
                (long long)head_dim);
  if (layout != NVFP4_ROPE_HALF && layout != NVFP4_ROPE_INTERLEAVED)
    return fail(NVFP4_ERR_ARG, "unknown rotary layout %d", layout);
  if (!std::isfinite(magnitude)) return fail(NVFP4_ERR_ARG, "magnitude must be finite");
  return NVFP4_OK;
}

inline int check_cache(const nvfp4_kv_cache* c, bool need_pool) {
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

inline int64_t groups_of(const nvfp4_kv_cache* c) { return c->pages * c->kv_heads * (c->page_size / kKvGroup); }

inline KvCache cache_of(const nvfp4_kv_cache* c) {
  KvCache r;
  const int db = (int)((c->head_dim + 63) / 64);
  const size_t code_bytes = kv_code_bytes(c->format, db);
  r.codes = static_cast<uint8_t*>(c->pool);
  r.scales = r.codes ? r.codes + (size_t)groups_of(c) * code_bytes : nullptr;  // no pool: sizes only
  r.slots = c->pages * c->page_size;
  r.pages = (int32_t)c->pages;
  r.heads = (int32_t)c->kv_heads;
  r.head_dim = (int32_t)c->head_dim;
  r.gpp = (int32_t)(c->page_size / kKvGroup);
  r.page_size = (int32_t)c->page_size;
  r.k_scale = c->k_scale;
  r.v_scale = c->v_scale;
  return r;
}

inline AttnLaunch attn_of(const nvfp4_attn_args* a) {
  AttnLaunch l;
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
  l.window = (int32_t)(a->window < kMaxDim ? a->window : kMaxDim);
  l.out = a->out;
  l.ldo = a->ldo;
  l.lse = a->lse;
  l.ws = a->workspace;
  return l;
}

inline int check_attn(const nvfp4_attn_args* a, bool need_buffers) {
  if (!a) return fail(NVFP4_ERR_NULL, "args is NULL");
  NVFP4_TRY(check_cache(a->cache, need_buffers && a->batch > 0));
  if (a->batch < 0 || a->batch > 65536) return fail(NVFP4_ERR_SHAPE, "batch=%lld must be in [0, 65536]", (long long)a->batch);
  if (a->q_heads < 1 || a->q_heads > kMaxHeads || a->q_heads % a->cache->kv_heads != 0)
    return fail(NVFP4_ERR_SHAPE, "q_heads=%lld must be a multiple of kv_heads=%lld, at most %lld", (long long)a->q_heads,
                (long long)a->cache->kv_heads, (long long)kMaxHeads);
  if (a->table_width < 0 || a->table_width > kMaxDim / a->cache->page_size)
    return fail(NVFP4_ERR_SHAPE, "table_width=%lld must be >= 0, and table_width * page_size at most 2^30",
                (long long)a->table_width);
  if (a->window < 0) return fail(NVFP4_ERR_ARG, "window=%lld is negative", (long long)a->window);
  if (!attn_fits(attn_of(a)))
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

}  // namespace nvfp4
