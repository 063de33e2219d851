// The C ABI of reading less of a long cache (declared in include/nvfp4_attn_long.h): argument validation,
// status codes and dispatch, as attn_abi.cpp does.  Nothing here allocates or synchronises.
#include <hip/hip_runtime_api.h>

#include <cmath>
#include <cstdint>

#include "../../include/nvfp4_attn_long.h"
#include "attn_checks.h"

namespace {

using namespace nvfp4;

constexpr int64_t kMaxBatch = 65536;
static_assert(NVFP4_SELECT_COUNTER_BYTES == kSelectCounterBytes, "counters");

int check_batch(int64_t batch) {
  if (batch < 0 || batch > kMaxBatch) return fail(NVFP4_ERR_SHAPE, "batch=%lld must be in [0, 65536]", (long long)batch);
  return NVFP4_OK;
}

// A count of pages: `low` or more, and no more than 2^30 tokens.
int check_width(int64_t n, int64_t low, int64_t page_size, const char* what) {
  if (n < low || n > kMaxDim / page_size)
    return fail(NVFP4_ERR_SHAPE, "%s=%lld must be >= %lld, and %s * page_size at most 2^30", what, (long long)n, (long long)low, what);
  return NVFP4_OK;
}

int check_workspace(const void* ws, size_t given, size_t need) {
  if (need == 0) return NVFP4_OK;
  if (!ws || given < need)
    return fail(NVFP4_ERR_WORKSPACE, "workspace of %zu bytes required, %zu given", need, ws ? given : 0);
  if (!aligned16(ws)) return fail(NVFP4_ERR_ALIGN, "workspace must be 16-byte aligned");
  return NVFP4_OK;
}

AttnSharedLaunch shared_of(const nvfp4_attn_shared_args* a) {
  return AttnSharedLaunch{attn_of(&a->attn), a->prefix_table, a->prefix_width, a->prefix_len};
}

int check_shared(const nvfp4_attn_shared_args* a, bool need_buffers) {
  if (!a) return fail(NVFP4_ERR_NULL, "args is NULL");
  NVFP4_TRY(check_attn(&a->attn, need_buffers));
  if (a->attn.window != 0) return fail(NVFP4_ERR_ARG, "window=%lld: a shared prefix takes none", (long long)a->attn.window);
  NVFP4_TRY(check_width(a->prefix_width, 0, a->attn.cache->page_size, "prefix_width"));
  if (a->attn.batch == 0) return NVFP4_OK;
  if (!attn_shared_fits(shared_of(a)))
    return fail(NVFP4_ERR_SHAPE, "batch x query heads above 2^30, or 2^31 tiles of the prefix or more");
  if (!need_buffers) return NVFP4_OK;
  if (!a->prefix_len || (a->prefix_width > 0 && !a->prefix_table))
    return fail(NVFP4_ERR_NULL, "prefix_table and prefix_len must be non-NULL");
  if (!aligned4(a->prefix_table) || !aligned4(a->prefix_len))
    return fail(NVFP4_ERR_ALIGN, "prefix_table and prefix_len must be 4-byte aligned");
  return NVFP4_OK;
}

int check_weigh(const nvfp4_attn_weigh_args* a, bool need_buffers) {
  if (!a) return fail(NVFP4_ERR_NULL, "args is NULL");
  NVFP4_TRY(check_attn(&a->attn, need_buffers));
  if (a->attn.batch * a->attn.cache->kv_heads > (int64_t(1) << 31) / (a->attn.table_width > 0 ? a->attn.table_width : 1))
    return fail(NVFP4_ERR_SHAPE, "batch * kv_heads * table_width must be at most 2^31");
  if (!need_buffers || a->attn.batch == 0) return NVFP4_OK;
  if (!std::isfinite(a->decay) || a->decay < 0.0f) return fail(NVFP4_ERR_ARG, "decay must be finite and at least 0");
  if (a->attn.table_width > 0 && (!a->weights_out || (a->decay != 0.0f && !a->weights)))
    return fail(NVFP4_ERR_NULL, "weights and weights_out must be non-NULL");
  if (!aligned4(a->weights) || !aligned4(a->weights_out))
    return fail(NVFP4_ERR_ALIGN, "weights and weights_out must be 4-byte aligned");
  return NVFP4_OK;
}

AttnWeighLaunch weigh_of(const nvfp4_attn_weigh_args* a) {
  return AttnWeighLaunch{attn_of(&a->attn), a->weights, a->decay, a->weights_out};
}

KvSelectLaunch select_of(const nvfp4_kv_select_args* a) {
  KvSelectLaunch l;
  l.batch = a->batch;
  l.heads = (int32_t)a->cache->kv_heads;
  l.head_dim = (int32_t)a->cache->head_dim;
  l.group = (int32_t)(a->q_heads / a->cache->kv_heads);
  l.pages = (int32_t)a->cache->pages;
  l.page_size = (int32_t)a->cache->page_size;
  l.q = a->q;
  l.ldq = a->ldq;
  l.bounds = a->bounds;
  l.table = a->page_table;
  l.table_width = a->table_width;
  l.lens = a->seq_lens;
  l.budget = a->budget;
  l.pages_out = a->pages_out;
  l.lens_out = a->lens_out;
  l.ws = a->workspace;
  return l;
}

int check_select(const nvfp4_kv_select_args* a, bool need_buffers) {
  if (!a) return fail(NVFP4_ERR_NULL, "args is NULL");
  NVFP4_TRY(check_cache(a->cache, false));
  NVFP4_TRY(check_batch(a->batch));
  if (a->q_heads < 1 || a->q_heads > kMaxHeads || a->q_heads % a->cache->kv_heads != 0)
    return fail(NVFP4_ERR_SHAPE, "q_heads=%lld must be a multiple of kv_heads=%lld, at most %lld", (long long)a->q_heads,
                (long long)a->cache->kv_heads, (long long)kMaxHeads);
  NVFP4_TRY(check_width(a->table_width, 0, a->cache->page_size, "table_width"));
  NVFP4_TRY(check_width(a->budget, 1, a->cache->page_size, "budget"));
  if (a->batch * a->cache->kv_heads > (int64_t(1) << 23))
    return fail(NVFP4_ERR_SHAPE, "batch * kv_heads must be at most 2^23");
  if (!need_buffers || a->batch == 0) return NVFP4_OK;
  NVFP4_TRY(check_ld(a->ldq, a->q_heads * a->cache->head_dim, "ldq"));
  if (!a->q || !a->bounds || !a->seq_lens || (a->table_width > 0 && !a->page_table) || !a->pages_out || !a->lens_out)
    return fail(NVFP4_ERR_NULL, "q, bounds, page_table, seq_lens, pages_out and lens_out must be non-NULL");
  if (!aligned16(a->q) || !aligned16(a->bounds)) return fail(NVFP4_ERR_ALIGN, "q and bounds must be 16-byte aligned");
  if (!aligned4(a->page_table) || !aligned4(a->seq_lens) || !aligned4(a->pages_out) || !aligned4(a->lens_out))
    return fail(NVFP4_ERR_ALIGN, "page_table, seq_lens, pages_out and lens_out must be 4-byte aligned");
  return NVFP4_OK;
}

KvEvictLaunch evict_of(const nvfp4_kv_evict_args* a) {
  KvEvictLaunch l;
  l.batch = a->batch;
  l.heads = (int32_t)a->kv_heads;
  l.page_size = (int32_t)a->page_size;
  l.weights = a->weights;
  l.table = a->page_table;
  l.table_width = a->table_width;
  l.lens = a->seq_lens;
  l.budget = a->budget;
  l.sink = a->sink;
  l.recent = a->recent;
  l.table_out = a->table_out;
  l.lens_out = a->lens_out;
  l.freed = a->freed;
  l.weights_out = a->weights_out;
  l.ws = a->workspace;
  return l;
}

int check_evict(const nvfp4_kv_evict_args* a, bool need_buffers) {
  if (!a) return fail(NVFP4_ERR_NULL, "args is NULL");
  NVFP4_TRY(check_batch(a->batch));
  if (a->kv_heads < 1 || a->kv_heads > 1024)
    return fail(NVFP4_ERR_SHAPE, "kv_heads=%lld must be in [1, 1024]", (long long)a->kv_heads);
  if (a->page_size < 16 || a->page_size > 65536 || a->page_size % 16 != 0)
    return fail(NVFP4_ERR_SHAPE, "page_size=%lld must be a multiple of 16 in [16, 65536]", (long long)a->page_size);
  NVFP4_TRY(check_width(a->table_width, 0, a->page_size, "table_width"));
  NVFP4_TRY(check_width(a->budget, 1, a->page_size, "budget"));
  if (a->sink < 0) return fail(NVFP4_ERR_ARG, "sink=%lld is negative", (long long)a->sink);
  if (a->recent < 1) return fail(NVFP4_ERR_ARG, "recent=%lld must be at least 1", (long long)a->recent);
  if (!need_buffers || a->batch == 0) return NVFP4_OK;
  if (!a->seq_lens || !a->table_out || !a->lens_out || (a->table_width > 0 && (!a->page_table || !a->weights)))
    return fail(NVFP4_ERR_NULL, "weights, page_table, seq_lens, table_out and lens_out must be non-NULL");
  if (!aligned4(a->weights) || !aligned4(a->page_table) || !aligned4(a->seq_lens) || !aligned4(a->table_out) ||
      !aligned4(a->lens_out) || !aligned4(a->weights_out) || !aligned4(a->freed))
    return fail(NVFP4_ERR_ALIGN, "weights, page_table, seq_lens and the outputs must be 4-byte aligned");
  return NVFP4_OK;
}

}  // namespace

extern "C" {

int nvfp4_attn_shared_workspace_bytes(const nvfp4_attn_shared_args* a, size_t* bytes) {
  NVFP4_GUARD_BEGIN
  if (!bytes) return fail(NVFP4_ERR_NULL, "bytes is NULL");
  NVFP4_TRY(check_shared(a, false));
  *bytes = a->attn.batch == 0 ? 0 : attn_shared_workspace_bytes(shared_of(a));
  return ok();
  NVFP4_GUARD_END
}

int nvfp4_attn_shared(const nvfp4_attn_shared_args* a, void* stream) {
  NVFP4_GUARD_BEGIN
  NVFP4_TRY(check_shared(a, true));
  if (a->attn.batch == 0) return ok();
  const AttnSharedLaunch l = shared_of(a);
  NVFP4_TRY(check_workspace(a->attn.workspace, a->attn.workspace_bytes, attn_shared_workspace_bytes(l)));
  return hip_status(launch_attn_shared(l, (hipStream_t)stream), "shared attention launch");
  NVFP4_GUARD_END
}

int nvfp4_kv_bounds(const nvfp4_kv_cache* c, const int32_t* pages, int64_t n, uint16_t* bounds, void* stream) {
  NVFP4_GUARD_BEGIN
  NVFP4_TRY(check_cache(c, n > 0));
  NVFP4_TRY(check_tokens(n));
  if (n * c->kv_heads > (int64_t(1) << 32)) return fail(NVFP4_ERR_SHAPE, "n * kv_heads must be at most 2^32");
  if (n == 0) return ok();
  if (!pages || !bounds) return fail(NVFP4_ERR_NULL, "pages and bounds must be non-NULL");
  if (!aligned4(pages)) return fail(NVFP4_ERR_ALIGN, "pages must be 4-byte aligned");
  if (!aligned16(bounds)) return fail(NVFP4_ERR_ALIGN, "bounds must be 16-byte aligned");
  return hip_status(launch_kv_bounds(KvBoundsLaunch{cache_of(c), c->format, n, pages, bounds}, (hipStream_t)stream),
                    "kv bounds launch");
  NVFP4_GUARD_END
}

int nvfp4_kv_select_workspace_bytes(const nvfp4_kv_select_args* a, size_t* bytes) {
  NVFP4_GUARD_BEGIN
  if (!bytes) return fail(NVFP4_ERR_NULL, "bytes is NULL");
  NVFP4_TRY(check_select(a, false));
  *bytes = a->batch == 0 ? 0 : kv_select_workspace_bytes(select_of(a));
  return ok();
  NVFP4_GUARD_END
}

int nvfp4_kv_select(const nvfp4_kv_select_args* a, void* stream) {
  NVFP4_GUARD_BEGIN
  NVFP4_TRY(check_select(a, true));
  if (a->batch == 0) return ok();
  const KvSelectLaunch l = select_of(a);
  NVFP4_TRY(check_workspace(a->workspace, a->workspace_bytes, kv_select_workspace_bytes(l)));
  return hip_status(launch_kv_select(l, (hipStream_t)stream), "kv select launch");
  NVFP4_GUARD_END
}

int nvfp4_attn_decode_heads(const nvfp4_attn_args* a, void* stream) {
  NVFP4_GUARD_BEGIN
  NVFP4_TRY(check_attn(a, true));
  if (a->batch == 0) return ok();
  const AttnLaunch l = attn_of(a);
  NVFP4_TRY(check_workspace(a->workspace, a->workspace_bytes, attn_workspace_bytes(l)));
  return hip_status(launch_attn_heads(l, (hipStream_t)stream), "attention launch");
  NVFP4_GUARD_END
}

int nvfp4_attn_weigh_workspace_bytes(const nvfp4_attn_weigh_args* a, size_t* bytes) {
  NVFP4_GUARD_BEGIN
  if (!bytes) return fail(NVFP4_ERR_NULL, "bytes is NULL");
  NVFP4_TRY(check_weigh(a, false));
  *bytes = a->attn.batch == 0 ? 0 : attn_weigh_workspace_bytes(weigh_of(a));
  return ok();
  NVFP4_GUARD_END
}

int nvfp4_attn_weigh(const nvfp4_attn_weigh_args* a, void* stream) {
  NVFP4_GUARD_BEGIN
  NVFP4_TRY(check_weigh(a, true));
  if (a->attn.batch == 0) return ok();
  const AttnWeighLaunch l = weigh_of(a);
  NVFP4_TRY(check_workspace(a->attn.workspace, a->attn.workspace_bytes, attn_weigh_workspace_bytes(l)));
  return hip_status(launch_attn_weigh(l, (hipStream_t)stream), "weighing attention launch");
  NVFP4_GUARD_END
}

int nvfp4_kv_evict_workspace_bytes(const nvfp4_kv_evict_args* a, size_t* bytes) {
  NVFP4_GUARD_BEGIN
  if (!bytes) return fail(NVFP4_ERR_NULL, "bytes is NULL");
  NVFP4_TRY(check_evict(a, false));
  *bytes = a->batch == 0 ? 0 : kv_evict_workspace_bytes(evict_of(a));
  return ok();
  NVFP4_GUARD_END
}

int nvfp4_kv_evict(const nvfp4_kv_evict_args* a, void* stream) {
  NVFP4_GUARD_BEGIN
  NVFP4_TRY(check_evict(a, true));
  if (a->batch == 0) return ok();
  const KvEvictLaunch l = evict_of(a);
  NVFP4_TRY(check_workspace(a->workspace, a->workspace_bytes, kv_evict_workspace_bytes(l)));
  return hip_status(launch_kv_evict(l, (hipStream_t)stream), "kv evict launch");
  NVFP4_GUARD_END
}

}  // extern "C"
