// The attention side's calls that are allowed without a pool -- sizes, workspace queries and calls with
// nothing to do -- with cache->pool NULL, for a build of the library's host code under the
// sanitizers.  No call here reaches a kernel launch.  Exit status 0 and a final "ok" line on success.
#include <cstdint>
#include <cstdio>

#include "nvfp4_attn.h"

static int failures = 0;
static void expect(int got, int want, const char* what) {
  if (got != want) {
    std::printf("%s: status %d, expected %d\n", what, got, want);
    ++failures;
  }
}

int main() {
  for (int format : {NVFP4_KV_BF16, NVFP4_KV_E4M3, NVFP4_KV_NVFP4}) {
    for (int64_t d : {16, 128, 192, 256}) {
      nvfp4_kv_cache c{nullptr, 8, 64, 8, d, format, 1.0f, 1.0f};
      size_t sz = 0;
      expect(nvfp4_kv_cache_bytes(&c, &sz), NVFP4_OK, "cache bytes");
      nvfp4_attn_args t{};
      t.cache = &c; t.batch = 3; t.q_heads = 16; t.table_width = 4;
      expect(nvfp4_attn_decode_workspace_bytes(&t, &sz), NVFP4_OK, "workspace");
      expect(sz > NVFP4_ATTN_COUNTER_BYTES ? 0 : 1, 0, "workspace bytes");
      t.batch = 0;
      expect(nvfp4_attn_decode_workspace_bytes(&t, &sz), NVFP4_OK, "workspace of nothing");
      expect(nvfp4_attn_decode(&t, nullptr), NVFP4_OK, "attention of nothing");
      nvfp4_kv_append_args a{};
      a.cache = &c; a.dtype = NVFP4_F32;
      expect(nvfp4_kv_append(&a, nullptr), NVFP4_OK, "append of nothing");
      expect(nvfp4_kv_read(&c, nullptr, 0, nullptr, 0, nullptr, 0, NVFP4_F32, nullptr), NVFP4_OK, "read of nothing");
      t.batch = 3; t.scale = 1.0f; t.ldq = t.ldo = 16 * d;
      expect(nvfp4_attn_decode(&t, nullptr), NVFP4_ERR_NULL, "attention without a pool");
    }
  }
  std::printf(failures ? "FAILED %d\n" : "ok\n", failures);
  return failures ? 1 : 0;
}
