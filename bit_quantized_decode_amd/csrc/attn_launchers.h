// Host-side launchers of the attention side's kernels; called only by
// attn_abi.cpp after it has validated every argument.
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
constexpr size_t kAttnCounterBytes = 1024;  // one counter a workgroup
// Whether the call's tiles can be numbered in 31 bits (at the longest lengths its table allows).
bool attn_fits(const AttnLaunch& a);
size_t attn_workspace_bytes(const AttnLaunch& a);
hipError_t launch_attn_decode(const AttnLaunch& a, hipStream_t s);

}  // namespace nvfp4
