// Host-side launchers of the attention side's kernels; called only by
// attn_abi.cpp and attn_long_abi.cpp after they have validated every argument.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

#include "kv_layout.h"

namespace nvfp4 {

// Rotary positions of one call.
struct Rope {
  const uint64_t* freqs;   // nullptr: none
  const int32_t* pos;
  int32_t rot;             // rotated values of a head
  bool interleaved;
  float magnitude;
  float sign;              // -1: the inverse turn
};

struct RopeLaunch {
  Rope rope;
  int64_t tokens;
  int32_t heads, head_dim;
  const void* x;
  void* y;
  int64_t ldx, ldy;
  bool x_bf16, y_bf16;
};
hipError_t launch_rope(const RopeLaunch& a, hipStream_t s);

struct KvAppendLaunch {
  KvCache cache;
  int format;
  Rope rope;
  int64_t tokens;
  const int64_t* slots;
  const void* k;
  const void* v;
  const void* q;           // nullptr: none
  uint16_t* q_out;
  int64_t ldk, ldv, ldq, ldqo;
  int32_t q_heads;
  bool bf16;               // k, v and q
};
hipError_t launch_kv_append(const KvAppendLaunch& a, hipStream_t s);

struct KvReadLaunch {
  KvCache cache;
  int format;
  int64_t tokens;
  const int64_t* slots;
  void* k;
  void* v;
  int64_t ldk, ldv;
  bool bf16;
};
hipError_t launch_kv_read(const KvReadLaunch& a, hipStream_t s);

struct AttnLaunch {
  KvCache cache;
  int format;
  int64_t batch;
  int32_t q_heads;
  const uint16_t* q;
  int64_t ldq;
  const int32_t* table;
  int64_t table_width;
  const int32_t* lens;
  float scale;
  int32_t window;          // 0: none
  uint16_t* out;
  int64_t ldo;
  float* lse;              // nullptr: none
  void* ws;
};
constexpr size_t kAttnCounterBytes = 1024;     // one counter a workgroup
constexpr size_t kSelectCounterBytes = 4096;   // one counter a (sequence, kv head) whose scores are cut
// In front of every workspace of the attention side: the counters of attention and of selection, from its first byte on, zero
// between calls of either.  What else a call keeps lies behind, so that one workspace serves both.
constexpr size_t kCounterBytes = kSelectCounterBytes;
// Whether the call's tiles can be numbered in 31 bits (at the longest lengths its table allows).
bool attn_fits(const AttnLaunch& a);
size_t attn_workspace_bytes(const AttnLaunch& a);
hipError_t launch_attn_decode(const AttnLaunch& a, hipStream_t s);

// ---- reading less of a long cache (attn_long_abi.cpp) ----

// Page tables of [batch][kv_heads][table_width].
hipError_t launch_attn_heads(const AttnLaunch& a, hipStream_t s);

// A grid of so many workgroups, or a few more: one dimension of a grid has fewer than 2^32 threads.
inline dim3 grid_of(int64_t workgroups) {
  const int64_t x = workgroups < 65536 ? workgroups : 65536;
  return dim3((unsigned)x, (unsigned)((workgroups + x - 1) / x));
}

struct AttnSharedLaunch {
  AttnLaunch attn;         // of the sequences' own tokens, its workspace the call's
  const int32_t* prefix_table;
  int64_t prefix_width;
  const int32_t* prefix_len;
};
// Whether the prefix's tiles can be numbered in 31 bits too.
bool attn_shared_fits(const AttnSharedLaunch& a);
size_t attn_shared_workspace_bytes(const AttnSharedLaunch& a);
hipError_t launch_attn_shared(const AttnSharedLaunch& a, hipStream_t s);

struct AttnWeighLaunch {
  AttnLaunch attn;
  const float* weights;    // [batch][kv_heads][table_width]; nullptr if decay == 0
  float decay;
  float* weights_out;
};
size_t attn_weigh_workspace_bytes(const AttnWeighLaunch& a);
hipError_t launch_attn_weigh(const AttnWeighLaunch& a, hipStream_t s);

struct KvBoundsLaunch {
  KvCache cache;
  int format;
  int64_t n;
  const int32_t* pages;
  uint16_t* bounds;        // [pages][heads][2][head_dim]
};
hipError_t launch_kv_bounds(const KvBoundsLaunch& a, hipStream_t s);

struct KvSelectLaunch {
  int64_t batch;
  int32_t heads, head_dim, group, pages, page_size;
  const uint16_t* q;
  int64_t ldq;
  const uint16_t* bounds;
  const int32_t* table;
  int64_t table_width;
  const int32_t* lens;
  int64_t budget;
  int32_t* pages_out;      // [batch][heads][budget]
  int32_t* lens_out;       // [batch]
  void* ws;
};
size_t kv_select_workspace_bytes(const KvSelectLaunch& a);
hipError_t launch_kv_select(const KvSelectLaunch& a, hipStream_t s);

struct KvEvictLaunch {
  int64_t batch;
  int32_t heads, page_size;
  const float* weights;    // [batch][heads][table_width]
  const int32_t* table;
  int64_t table_width;
  const int32_t* lens;
  int64_t budget, sink, recent;
  int32_t* table_out;      // [batch][budget]
  int32_t* lens_out;       // [batch]
  int32_t* freed;          // nullptr, or [batch][table_width]
  float* weights_out;      // nullptr, or [batch][heads][budget]
  void* ws;
};
size_t kv_evict_workspace_bytes(const KvEvictLaunch& a);
hipError_t launch_kv_evict(const KvEvictLaunch& a, hipStream_t s);

}  // namespace nvfp4
