// The private layout of the paged key-value cache, shared by the kernels that
// write it, read it back and attend over it.
//
// The pool is an array of groups: 16 consecutive tokens of one page and one
// kv head.  Group (page, head, g) has index (page * heads + head) * gpp + g,
// gpp = page_size / 16.  First come the codes of all groups, then the scales of
// all groups, so that a group's codes start on their own cache lines.
//
// Inside a group everything is laid out by the wavefront lane that needs it in
// attention, on 16x16x32 matrix instructions (A operand: lane l holds row l % 16
// and eight k's numbered by l / 16).  With the head padded to 64*DB values and
// E = 16*DB, lane l = 16 h + r holds E values of K and E of V:
//   K   token r, values d = E h + e                    (rows = tokens, k = d)
//   V   tokens 4h + i, values d = W r + w, e = i W + w  (rows = d, k = tokens),
//       W = E / 4
// so that neither operand crosses lanes: the queries are loaded with the same
// split of d, and the scores of a 16-token tile come out of the instruction with
// lane 16 h + q holding tokens 4h + i of query q, which is the k split of V.
// A lane's bytes are cut into 16-byte planes (and one 8-byte plane if E codes end
// on one), each plane 64 lanes in order: every wavefront load is contiguous.
//
// Scales.  E4M3: one exponent byte (2^(byte - 127)) a token, 16 of K then 16 of
// V.  NVFP4: K, SB bytes a lane (one per 16 of its values, padded to 1, 2 or 4);
// V, for each h and block of 16 d, the four tokens' bytes as one word.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace nvfp4 {

enum { kKvBf16 = 0, kKvE4m3 = 1, kKvNvfp4 = 2 };

constexpr int kKvGroup = 16;  // tokens of a group
constexpr int kKvE4m3Bias = 127;
constexpr int kKvE4m3MinExp = -110;  // the smallest exponent of an E4M3 row: every value stays a normal bf16
constexpr int kKvE4m3MaxExp = 120;   // the largest: that of a row up to fp32's maximum

template <int FMT, int DB>
struct KvLayout {
  static constexpr int kE = 16 * DB;                                        // values a lane holds of K, and of V
  static constexpr int kW = 4 * DB;                                         // consecutive d of a V lane
  static constexpr int kBits = FMT == kKvBf16 ? 16 : FMT == kKvE4m3 ? 8 : 4;
  static constexpr int kLaneBytes = kE * kBits / 8;
  static constexpr int kPlanes16 = kLaneBytes / 16;
  static constexpr bool kPlane8 = kLaneBytes % 16 != 0;
  static constexpr int kSideBytes = 64 * kLaneBytes;                        // K or V codes of a group
  static constexpr int kCodeBytes = 2 * kSideBytes;
  static constexpr int kKScaleLane = DB == 3 ? 4 : DB;                      // NVFP4: K scale bytes a lane
  static constexpr int kKScaleBytes = FMT == kKvBf16 ? 0 : FMT == kKvE4m3 ? 16 : 64 * kKScaleLane;
  static constexpr int kVScaleBytes = FMT == kKvBf16 ? 0 : FMT == kKvE4m3 ? 16 : 64 * DB;
  static constexpr int kScaleBytes = kKScaleBytes + kVScaleBytes;
  // Byte `b` of lane `l` within K's or V's codes.
  static constexpr int lane_byte(int l, int b) {
    return b / 16 < kPlanes16 ? (b / 16) * 1024 + l * 16 + b % 16 : kPlanes16 * 1024 + l * 8 + b % 16;
  }
};

// A group's codes, and its codes and scales.
inline size_t kv_code_bytes(int format, int db) {
  return (size_t)1024 * db * (format == kKvBf16 ? 4 : format == kKvE4m3 ? 2 : 1);
}
inline size_t kv_group_bytes(int format, int db) {
  const size_t scales = format == kKvBf16 ? 0 : format == kKvE4m3 ? 32 : 64 * (size_t)(db == 3 ? 4 : db) + 64 * (size_t)db;
  return kv_code_bytes(format, db) + scales;
}
static_assert(KvLayout<kKvBf16, 2>::kCodeBytes == 1024 * 2 * 4 && KvLayout<kKvE4m3, 3>::kCodeBytes == 1024 * 3 * 2 &&
                  KvLayout<kKvNvfp4, 4>::kCodeBytes == 1024 * 4 && KvLayout<kKvNvfp4, 3>::kScaleBytes == 64 * 4 + 64 * 3,
              "the host's sizes are the layout's");

// A cache as the kernels see it.
struct KvCache {
  uint8_t* codes;
  uint8_t* scales;
  int64_t slots;      // pages * page_size
  int32_t pages, heads, head_dim;
  int32_t gpp;        // groups a page
  int32_t page_size;
  float k_scale, v_scale;
};

}  // namespace nvfp4
