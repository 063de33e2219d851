// Calls every entry point of the attention side's C ABI with arguments it must
// refuse before any launch, and the host-only ones with host buffers of exactly
// the documented sizes, for an AddressSanitizer / UndefinedBehaviorSanitizer
// build of the library's host code.  No call here reaches a kernel launch.
// Exit status 0 and a final "ok" line on success.
#include <cstdint>
#include <cstdio>
#include <vector>

#include "nvfp4_attn.h"

static int failures = 0;
static void expect(int got, int want, const char* what) {
  if (got != want) {
    std::printf("%s: status %d, expected %d\n", what, got, want);
    ++failures;
  }
}

int main() {
  void* A = reinterpret_cast<void*>(0x10000);  // placeholders: never dereferenced on these paths
  size_t sz = 0;
  float mag = 0.0f;
  for (int64_t rot : {0, 16, 128, 256}) {
    for (int scaling : {NVFP4_ROPE_NONE, NVFP4_ROPE_LINEAR, NVFP4_ROPE_YARN}) {
      nvfp4_rope_config c{rot, 1e6, scaling, 8.0, 4096.0, 32.0, 1.0};
      std::vector<uint64_t> f((size_t)rot / 2);
      expect(nvfp4_rope_freqs(&c, f.data(), &mag), NVFP4_OK, "freqs");
    }
  }
  for (double original : {1e-300, 1e300}) {
    nvfp4_rope_config c{64, 1.0000001, NVFP4_ROPE_YARN, 1e30, original, 1e300, 1e-300};
    std::vector<uint64_t> f(32);
    expect(nvfp4_rope_freqs(&c, f.data(), &mag), NVFP4_OK, "freqs, far ends");
  }
  nvfp4_rope_config bad{64, 0.5, 0, 1.0, 0.0, 0.0, 0.0};
  uint64_t one[32];
  expect(nvfp4_rope_freqs(&bad, one, &mag), NVFP4_ERR_ARG, "freqs base");

  nvfp4_rope_args r{};
  r.tokens = 4; r.heads = 2; r.head_dim = 64; r.rot_dim = 64; r.magnitude = 1.0f; r.x_dtype = r.y_dtype = NVFP4_BF16;
  r.ldx = r.ldy = 128;
  expect(nvfp4_rope(&r, nullptr), NVFP4_ERR_NULL, "rope null");
  r.ldx = INT64_MAX;
  expect(nvfp4_rope(&r, nullptr), NVFP4_ERR_SHAPE, "rope ld");
  r.tokens = INT64_MIN;
  expect(nvfp4_rope(&r, nullptr), NVFP4_ERR_SHAPE, "rope tokens");

  nvfp4_kv_cache c{A, 8, 64, 8, 128, NVFP4_KV_NVFP4, 1.0f, 1.0f};
  expect(nvfp4_kv_cache_bytes(&c, &sz), NVFP4_OK, "cache bytes");
  for (int64_t big : {INT64_MAX, INT64_MIN, (int64_t)1 << 60}) {
    nvfp4_kv_cache d = c;
    d.pages = big;
    expect(nvfp4_kv_cache_bytes(&d, &sz), NVFP4_ERR_SHAPE, "pages");
    d = c;
    d.page_size = big;
    expect(nvfp4_kv_cache_bytes(&d, &sz), NVFP4_ERR_SHAPE, "page_size");
    d = c;
    d.kv_heads = big;
    expect(nvfp4_kv_cache_bytes(&d, &sz), NVFP4_ERR_SHAPE, "kv_heads");
    d = c;
    d.head_dim = big;
    expect(nvfp4_kv_cache_bytes(&d, &sz), NVFP4_ERR_SHAPE, "head_dim");
  }
  nvfp4_kv_append_args a{};
  a.cache = &c; a.tokens = 4; a.dtype = NVFP4_F32; a.ldk = a.ldv = 1024;
  expect(nvfp4_kv_append(&a, nullptr), NVFP4_ERR_NULL, "append null");
  a.q = A; a.freqs = static_cast<uint64_t*>(A); a.q_heads = INT64_MAX;
  expect(nvfp4_kv_append(&a, nullptr), NVFP4_ERR_SHAPE, "append q_heads");
  expect(nvfp4_kv_read(&c, nullptr, 4, A, 1024, A, 1024, NVFP4_F32, nullptr), NVFP4_ERR_NULL, "read null");
  expect(nvfp4_kv_read(&c, nullptr, INT64_MAX, A, 1024, A, 1024, NVFP4_F32, nullptr), NVFP4_ERR_SHAPE, "read tokens");

  nvfp4_attn_args t{};
  t.cache = &c; t.batch = 65536; t.q_heads = 32768; t.table_width = ((int64_t)1 << 30) / 64; t.window = INT64_MAX;
  t.scale = 1.0f; t.ldq = t.ldo = 32768 * 128;
  expect(nvfp4_attn_decode_workspace_bytes(&t, &sz), NVFP4_ERR_SHAPE, "attention of 2^31 tiles");
  t.batch = 1;  // 8 kv heads x 256 row tiles x 2^20 tiles
  expect(nvfp4_attn_decode_workspace_bytes(&t, &sz), NVFP4_ERR_SHAPE, "attention of 2^31 tiles");
  t.batch = 65536; t.q_heads = 8; t.window = 1000;  // 8 kv heads x 35 tiles a sequence
  expect(nvfp4_attn_decode_workspace_bytes(&t, &sz), NVFP4_OK, "attention workspace");
  expect(nvfp4_attn_decode(&t, nullptr), NVFP4_ERR_NULL, "attention null");
  t.q = t.out = static_cast<uint16_t*>(A);
  t.seq_lens = t.page_table = static_cast<int32_t*>(A);
  t.workspace = A; t.workspace_bytes = sz - 1;
  expect(nvfp4_attn_decode(&t, nullptr), NVFP4_ERR_WORKSPACE, "attention workspace size");
  for (int64_t big : {INT64_MAX, INT64_MIN}) {
    nvfp4_attn_args u = t;
    u.batch = big;
    expect(nvfp4_attn_decode(&u, nullptr), NVFP4_ERR_SHAPE, "attention batch");
    u = t;
    u.table_width = big;
    expect(nvfp4_attn_decode(&u, nullptr), NVFP4_ERR_SHAPE, "attention table");
    u = t;
    u.q_heads = big;
    expect(nvfp4_attn_decode(&u, nullptr), NVFP4_ERR_SHAPE, "attention heads");
  }
  std::printf(failures ? "FAILED %d\n" : "ok\n", failures);
  return failures ? 1 : 0;
}
