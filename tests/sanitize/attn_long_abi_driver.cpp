// Drives the entry points of nvfp4_attn_long.h with arguments that they must refuse, or answer, before any launch:
// built with the sanitizers on the host side, on a machine without a GPU.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>

#include "nvfp4_attn_long.h"

namespace {

int g_failed = 0;
void expect(int got, int want, const char* what) {
  if (got != want) {
    std::printf("%s: %d, expected %d (%s)\n", what, got, want, nvfp4_last_error());
    ++g_failed;
  }
}

template <class T>
T* at(uintptr_t a) { return reinterpret_cast<T*>(a); }   // placeholders: never dereferenced

nvfp4_kv_cache cache(bool pool) {
  nvfp4_kv_cache c{};
  c.pool = pool ? at<void>(0x10000) : nullptr;
  c.pages = 8, c.page_size = 64, c.kv_heads = 8, c.head_dim = 128, c.format = NVFP4_KV_NVFP4, c.k_scale = c.v_scale = 1.0f;
  return c;
}

nvfp4_attn_args attn(const nvfp4_kv_cache* c) {
  nvfp4_attn_args a{};
  a.cache = c, a.batch = 4, a.q_heads = 40, a.q = at<uint16_t>(0x10000), a.ldq = 5120, a.page_table = at<int32_t>(0x10000);
  a.table_width = 4, a.seq_lens = at<int32_t>(0x10000), a.scale = 0.1f, a.out = at<uint16_t>(0x20000), a.ldo = 5120;
  return a;   // no workspace: every call stops there at the latest
}

}  // namespace

int main() {
  const nvfp4_kv_cache full = cache(true), sizes = cache(false);
  size_t n = 0;

  nvfp4_attn_shared_args s{};
  expect(nvfp4_attn_shared(nullptr, nullptr), NVFP4_ERR_NULL, "shared NULL");
  expect(nvfp4_attn_shared(&s, nullptr), NVFP4_ERR_NULL, "shared blank");
  s.attn = attn(&full), s.prefix_table = at<int32_t>(0x10000), s.prefix_width = 100, s.prefix_len = at<int32_t>(0x10000);
  expect(nvfp4_attn_shared(&s, nullptr), NVFP4_ERR_WORKSPACE, "shared without workspace");
  s.attn.window = 5;
  expect(nvfp4_attn_shared(&s, nullptr), NVFP4_ERR_ARG, "shared window");
  s.attn.window = 0;
  for (int64_t width : {INT64_MIN, int64_t(-1), int64_t(1) << 25, INT64_MAX}) {
    s.prefix_width = width;
    expect(nvfp4_attn_shared(&s, nullptr), NVFP4_ERR_SHAPE, "prefix_width");
  }
  s.attn = attn(&sizes), s.prefix_width = 1 << 24;
  expect(nvfp4_attn_shared_workspace_bytes(&s, &n), NVFP4_OK, "shared sizes without a pool");
  s.attn.batch = 65536, s.attn.table_width = 0;
  expect(nvfp4_attn_shared_workspace_bytes(&s, &n), NVFP4_ERR_SHAPE, "shared tiles");
  s.attn.q_heads = 32768;
  expect(nvfp4_attn_shared_workspace_bytes(&s, &n), NVFP4_ERR_SHAPE, "shared rows");
  s.attn.batch = 0;
  expect(nvfp4_attn_shared(&s, nullptr), NVFP4_OK, "shared of nothing");

  nvfp4_attn_weigh_args w{};
  expect(nvfp4_attn_weigh(nullptr, nullptr), NVFP4_ERR_NULL, "weigh NULL");
  expect(nvfp4_attn_weigh(&w, nullptr), NVFP4_ERR_NULL, "weigh blank");
  w.attn = attn(&full), w.weights = at<float>(0x10000), w.weights_out = at<float>(0x10000), w.decay = 1.0f;
  expect(nvfp4_attn_weigh(&w, nullptr), NVFP4_ERR_WORKSPACE, "weigh without workspace");
  for (float decay : {-1.0f, NAN, INFINITY}) {
    w.decay = decay;
    expect(nvfp4_attn_weigh(&w, nullptr), NVFP4_ERR_ARG, "decay");
  }
  w.attn = attn(&sizes), w.attn.batch = 65536, w.attn.table_width = 1 << 24, w.attn.window = 1;
  expect(nvfp4_attn_weigh_workspace_bytes(&w, &n), NVFP4_ERR_SHAPE, "weights past 2^31");
  w.attn.window = INT64_MAX, w.attn.batch = 4;
  expect(nvfp4_attn_weigh_workspace_bytes(&w, &n), NVFP4_OK, "weigh window");

  nvfp4_attn_args heads = attn(&full);
  expect(nvfp4_attn_decode_heads(nullptr, nullptr), NVFP4_ERR_NULL, "heads NULL");
  expect(nvfp4_attn_decode_heads(&heads, nullptr), NVFP4_ERR_WORKSPACE, "heads without workspace");

  expect(nvfp4_kv_bounds(nullptr, nullptr, 1, nullptr, nullptr), NVFP4_ERR_NULL, "bounds NULL");
  expect(nvfp4_kv_bounds(&full, nullptr, INT64_MAX, nullptr, nullptr), NVFP4_ERR_SHAPE, "bounds of too many");
  expect(nvfp4_kv_bounds(&full, nullptr, 1, nullptr, nullptr), NVFP4_ERR_NULL, "bounds pages");
  expect(nvfp4_kv_bounds(&sizes, nullptr, 0, nullptr, nullptr), NVFP4_OK, "bounds of nothing");

  nvfp4_kv_select_args k{};
  expect(nvfp4_kv_select(nullptr, nullptr), NVFP4_ERR_NULL, "select NULL");
  expect(nvfp4_kv_select(&k, nullptr), NVFP4_ERR_NULL, "select blank");
  k.cache = &sizes, k.batch = 4, k.q_heads = 40, k.q = at<uint16_t>(0x10000), k.ldq = 5120, k.bounds = at<uint16_t>(0x10000);
  k.page_table = at<int32_t>(0x10000), k.table_width = 5000, k.seq_lens = at<int32_t>(0x10000), k.budget = 9;
  k.pages_out = at<int32_t>(0x10000), k.lens_out = at<int32_t>(0x10000);
  expect(nvfp4_kv_select(&k, nullptr), NVFP4_ERR_WORKSPACE, "select without workspace");
  for (int64_t budget : {INT64_MIN, int64_t(0), int64_t(1) << 25, INT64_MAX}) {
    k.budget = budget;
    expect(nvfp4_kv_select(&k, nullptr), NVFP4_ERR_SHAPE, "budget");
  }
  k.budget = 1;
  for (int64_t batch : {int64_t(1), int64_t(127), int64_t(128), int64_t(65536)})
    for (int64_t width : {int64_t(0), int64_t(1), int64_t(65), int64_t(4097), int64_t(1) << 24}) {
      k.batch = batch, k.table_width = width;
      expect(nvfp4_kv_select_workspace_bytes(&k, &n), NVFP4_OK, "select sizes");
    }

  nvfp4_kv_evict_args e{};
  expect(nvfp4_kv_evict(nullptr, nullptr), NVFP4_ERR_NULL, "evict NULL");
  expect(nvfp4_kv_evict(&e, nullptr), NVFP4_ERR_SHAPE, "evict blank");
  e.batch = 4, e.kv_heads = 8, e.page_size = 64, e.weights = at<float>(0x10000), e.page_table = at<int32_t>(0x10000);
  e.table_width = 9000, e.seq_lens = at<int32_t>(0x10000), e.budget = 9, e.recent = INT64_MAX, e.sink = INT64_MAX;
  e.table_out = at<int32_t>(0x10000), e.lens_out = at<int32_t>(0x10000);
  expect(nvfp4_kv_evict(&e, nullptr), NVFP4_ERR_WORKSPACE, "evict without workspace");
  e.sink = INT64_MIN;
  expect(nvfp4_kv_evict(&e, nullptr), NVFP4_ERR_ARG, "sink");
  e.sink = 0, e.recent = 0;
  expect(nvfp4_kv_evict(&e, nullptr), NVFP4_ERR_ARG, "recent");
  e.recent = 1, e.page_size = INT64_MIN;
  expect(nvfp4_kv_evict(&e, nullptr), NVFP4_ERR_SHAPE, "page size");
  e.page_size = 64, e.batch = 65536, e.table_width = 1 << 24;
  expect(nvfp4_kv_evict_workspace_bytes(&e, &n), NVFP4_OK, "evict sizes");
  expect(nvfp4_kv_evict_workspace_bytes(&e, nullptr), NVFP4_ERR_NULL, "evict sizes NULL");

  if (g_failed) return 1;
  std::puts("ok");
  return 0;
}
