// Attention of one new token per sequence over the paged cache (nvfp4_attn_decode).
//
//   s_j = scale q.k_j,   o = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m)
//
// in one pass over the cache with a running reference r in place of the maximum
// (softmax does not depend on it): p_j = 2^(s_j log2 e - r), l = sum p_j.
//
// Tiles.  The query heads of one kv head (up to 16, more in further row tiles) are
// the columns of 16x16x32 matrix instructions.  A wavefront takes 32 tokens at a
// time: scores S = K Q^T come out with lane 16 h + q holding tokens 4h + i of
// query q, which is exactly the k split of the second product O^T = V^T P^T, so
// probabilities go from one to the other inside their lane.  Because a lane belongs to
// one query, the reference and the sum are lane values; the reference only
// moves when a term would pass 2^kSlack times the one that it was set by, and only
// then do lanes talk.
//
// Operands.  bf16 and E4M3 caches multiply as bf16 (every E4M3 value times its
// power of two is a bf16 number), NVFP4 as f16 (E2M1 times E4M3 is an f16
// number); the queries, bf16, are shifted into f16's range by a power of two
// per row.  Probabilities enter as one f16 number (half a step: 2^-11, an eighth
// of the output's own rounding) or as the sum of two bf16 numbers (2^-17; one
// alone would add as much as the output's rounding); everything else is fp32.
// (Two f16 numbers would take 2^-22.  Against one: 32 users of 8192 NVFP4 tokens 52.8-53.4 us
// against 50.6-50.9, 256 of up to 512 tokens 24.1-24.5 against 22.0-23.3, and an output no
// nearer to 64 bits, as its rounding to bf16 is the larger by far.)
//
// Work split.  The 32-token tiles of all units (sequence, kv head, row tile) form
// one line, each unit led by kLead blank places for what starting it costs.
// The line is cut evenly over the workgroups (one a CU, fewer if little is to be done), cuts
// inside a short unit moved to its nearer end, and each share over the wavefronts, whatever
// the lengths are.  A wavefront walks its run of the line by itself: it writes the units
// that lie inside its run, leaves the end of a unit begun by an earlier wavefront in
// LDS, and keeps the beginning of one that goes on in registers.  Once all are
// through, each beginning is joined with what follows it in LDS.  What goes on in
// another workgroup becomes a partial sum in memory, and the last workgroup of a unit to
// arrive joins those, in order.
//
// Bound by the cache's bytes where they are many, by a fixed 8 us where they are few: the
// launch (3 us), lengths, page table and first tile, each waiting for the one before (3 us), and
// the way of partial sums through memory (2 to 4 us).  8 kv heads of 128 for 40 query heads,
// inputs cold (warm in brackets): one user over 131,072 tokens bf16 87-91 us (85-89; 537 MB, 5.9 to
// 6.3 TB/s); 32 users over up to 16,384 tokens NVFP4 51-59 us (50-57; 274-308 MB, 5.2 to 5.4 TB/s, by
// the lengths); over 8192 each 52 us (302 MB, 5.8 TB/s); one user over 100 / 1000 / 8000 tokens 7.2 /
// 9.4 / 12.9 us (7.0 / 9.2 / 12.3).  A streaming read runs at 6.65.  Dequantising NVFP4 takes 2.5 % of
// the long batches, an eighth of short users' (against a copy with a trivial conversion).
// Non-temporal loads: 32 users of 16,384 NVFP4 tokens 96 us against 112, one of 131,072 bf16
// tokens 90 against 100 (a cache that still lies in the MALL reads up to 5 % slower).  Page
// sizes of 16 to 2048 tokens, in order or not, read alike.
#include <cmath>

#include "attn_launchers.h"
#include "device_common.h"

namespace nvfp4 {
namespace {

constexpr int kTile = 32;                  // tokens of a wavefront's step
constexpr int kRows = 16;                  // query heads of a row tile
constexpr int kCus = 256;
// Places before a unit's tiles.  (With 2: 32 ragged users of NVFP4 52-56 us against 50-55;
// with 4: 256 users of up to 512 tokens 23.0-24.4 us against 21.8-23.0.)
constexpr int kLead = 3;
// Places of a workgroup's share, at least, if units are cut: a part for each adds to the
// join what the share saves, so that the longest unit gets about as many parts as its join
// reads in one round trip, within bounds; powers of two, for shifts.  (NVFP4, one kv head of
// 128, shares of 4 / 9 / 16 / 32 / 64 places for 8 query heads: 4000 tokens 11.0 / 12.0 / 12.5 /
// 14.3 / 17.9 us, 16,000 tokens 18.0 / 15.6 / 14.5 / 15.7 / 19.8, 131,072 tokens 32.1 / 32.3 /
// 31.9 / 23.4 / 22.7.  Parts of 16 / 32 / 64 / 96 over 16,000 tokens: 1 query head 15.6 / 14.9 /
// 13.0 / 12.8 us, 4 heads 14.8 / 13.5 / 13.3 / 14.3, 16 heads 16.6 / 17.4 / 21.5 / 26.5.)
constexpr int kShareMinLog = 2, kShareMaxLog = 5, kPartsMinLog = 4, kPartsMaxLog = 6;
constexpr int kJoinBatch = 12;             // parts that a thread of a join reads at once
static_assert(kCus * 4 <= (int)kAttnCounterBytes, "one counter a workgroup");
constexpr double kLog2e = 1.4426950408889634;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -__builtin_inff();
constexpr float kFltMax = 3.40282347e38f;

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

struct AttnParams {
  KvCache cache;
  const uint16_t* q;
  const int32_t* table;
  const int32_t* lens;
  uint16_t* out;
  float* lse;
  unsigned* counters;
  float* part;         // partial sums, see part_offset()
  int64_t ldq, ldo, table_width;
  int32_t batch, q_heads, group, row_tiles, window, part_rows, part_bytes, parts_log;
  float score_factor;  // score_factor * 2^score_exp = scale * log2 e * the keys' tensor scale
  int score_exp;
};

// The tokens that a row attends to.
struct Span {
  int begin, end;      // [begin, end)
  int base;            // begin rounded down to a group
  int tiles;           // at least one, so that an empty row is written too
};
__device__ __forceinline__ Span span_of(const AttnParams& a, int len) {
  Span s;
  const int64_t most = a.table_width * a.cache.page_size;
  s.end = len < 0 ? 0 : (int64_t)len > most ? (int)most : len;
  s.begin = a.window > 0 && s.end > a.window ? s.end - a.window : 0;
  s.base = s.begin & ~(kKvGroup - 1);
  const int n = (s.end - s.base + kTile - 1) / kTile;
  s.tiles = n > 1 ? n : 1;
  return s;
}

// The partial sums that workgroup w leaves of a unit that starts before its share
// (side 0) or in it (side 1): rows of reference, sum and the padded head's sums.
// They are written through to memory and read from it (sc1), whichever XCDs the
// workgroups run on; offsets are bytes, below 2^31 for every workspace.
template <int DP>
__device__ __forceinline__ int part_offset(const AttnParams& a, int w, int side, int row) {
  return ((2 * w + side) * a.part_rows + row) * (DP + 4) * 4;
}
constexpr int kThroughMemory = 16;  // cache policy sc1
__device__ __forceinline__ __amdgpu_buffer_rsrc_t part_buffer(const AttnParams& a) {
  return __builtin_amdgcn_make_buffer_rsrc(a.part, 0, a.part_bytes, 0x00020000);
}
__device__ __forceinline__ f32x4 load_part(__amdgpu_buffer_rsrc_t r, int offset) {
  return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, offset, 0, kThroughMemory));
}
__device__ __forceinline__ void store_part(__amdgpu_buffer_rsrc_t r, int offset, f32x4 v) {
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), r, offset, 0, kThroughMemory);
}

template <int FMT, int DB>
struct Tile {
  using L = KvLayout<FMT, DB>;
  static constexpr int kWords = L::kLaneBytes / 4;
  static constexpr int kVScales = FMT == kKvNvfp4 && DB == 3 ? 3 : 1;
  uint32_t k[2][kWords], v[2][kWords];
  uint32_t ks[2], vs[2][kVScales];
};

// Where a group's codes and scales lie.  The codes are a buffer: that of a group that
// is not there (below 0) is empty, and loads from it give zeros without reading.
// (Its scales are the pool's first, a few bytes that every wavefront finds in the
// cache; as a second buffer they cost 0.2 us of 15 in scalar registers.)
struct GroupBuffers {
  __amdgpu_buffer_rsrc_t codes;
  const uint8_t* scales;
};
template <int FMT, int DB>
__device__ __forceinline__ GroupBuffers group_buffers(const KvCache& c, int group) {
  using L = KvLayout<FMT, DB>;
  const int64_t g = max(group, 0);
  GroupBuffers r;
  r.codes = __builtin_amdgcn_make_buffer_rsrc(c.codes + g * L::kCodeBytes, 0, group < 0 ? 0 : L::kCodeBytes, 0x00020000);
  r.scales = c.scales + g * L::kScaleBytes;
  return r;
}

constexpr int kStreamed = 2;  // cache policy nt
template <int FMT, int DB>
__device__ __forceinline__ void load_side(__amdgpu_buffer_rsrc_t r, int side, int lane, uint32_t* w) {
  using L = KvLayout<FMT, DB>;
#pragma unroll
  for (int i = 0; i < L::kPlanes16; ++i) {
    const u32x4 x =
        __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, lane * 16, side + i * 1024, kStreamed));
#pragma unroll
    for (int j = 0; j < 4; ++j) w[4 * i + j] = x[j];
  }
  if constexpr (L::kPlane8) {
    const u32x2 x = __builtin_bit_cast(
        u32x2, __builtin_amdgcn_raw_buffer_load_b64(r, lane * 8, side + L::kPlanes16 * 1024, kStreamed));
    w[4 * L::kPlanes16] = x[0];
    w[4 * L::kPlanes16 + 1] = x[1];
  }
}

template <int FMT, int DB>
__device__ __forceinline__ void load_k(const GroupBuffers (&g)[2], int lane, Tile<FMT, DB>& t) {
  using L = KvLayout<FMT, DB>;
#pragma unroll
  for (int a = 0; a < 2; ++a) {
    load_side<FMT, DB>(g[a].codes, 0, lane, t.k[a]);
    if constexpr (FMT == kKvE4m3) t.ks[a] = g[a].scales[lane & 15];
    else if constexpr (FMT == kKvNvfp4) {
      if constexpr (L::kKScaleLane == 1) t.ks[a] = g[a].scales[lane];
      else if constexpr (L::kKScaleLane == 2) t.ks[a] = *reinterpret_cast<const uint16_t*>(g[a].scales + 2 * lane);
      else t.ks[a] = *reinterpret_cast<const uint32_t*>(g[a].scales + 4 * lane);
    }
  }
}

template <int FMT, int DB>
__device__ __forceinline__ void load_v(const GroupBuffers (&g)[2], int lane, Tile<FMT, DB>& t) {
  using L = KvLayout<FMT, DB>;
#pragma unroll
  for (int a = 0; a < 2; ++a) {
    load_side<FMT, DB>(g[a].codes, L::kSideBytes, lane, t.v[a]);
    if constexpr (FMT == kKvE4m3)
      t.vs[a][0] = *reinterpret_cast<const uint32_t*>(g[a].scales + L::kKScaleBytes + 4 * (lane >> 4));
    else if constexpr (FMT == kKvNvfp4) {
#pragma unroll
      for (int u = 0; u < Tile<FMT, DB>::kVScales; ++u)
        t.vs[a][u] = *reinterpret_cast<const uint32_t*>(
            g[a].scales + L::kKScaleBytes + 16 * DB * (lane >> 4) + 4 * ((L::kW * (lane & 15) + 4 * u) / 16));
    }
  }
}

// E4M3 byte `i` of w as an f16 pair of that value.
__device__ __forceinline__ f16x2 scale_pair(uint32_t w, int i) {
  const f16x2 p = __builtin_bit_cast(f16x2, i >= 2 ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true)
                                                   : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false));
  return (i & 1) ? f16x2{p[1], p[1]} : f16x2{p[0], p[0]};
}

// Two E2M1 codes (byte `sel`) times a scale pair: exact in f16.
template <int SEL>
__device__ __forceinline__ uint32_t e2m1_scaled(uint32_t w, f16x2 s) {
  const f16x2 p = __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, SEL)) * s;
  return __builtin_bit_cast(uint32_t, p);
}
// Two E4M3 codes (half HI of w) times a power of two: exact in bf16.
template <bool HI>
__device__ __forceinline__ uint32_t e4m3_scaled(uint32_t w, float s) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, HI));
}
__device__ __forceinline__ float byte_exp2(uint32_t w, int i) { return __uint_as_float(((w >> (8 * i)) & 0xffu) << 23); }

template <int FMT>
__device__ __forceinline__ f32x4 mma(const uint32_t* a, const uint32_t* b, f32x4 acc) {
  const u32x4 x{a[0], a[1], a[2], a[3]}, y{b[0], b[1], b[2], b[3]};
  if constexpr (FMT == kKvNvfp4)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, x), __builtin_bit_cast(f16x8, y), acc, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, y), acc, 0, 0, 0);
}

// K operand of matrix step s: the lane's values 8s .. 8s + 7 as 16-bit pairs.
template <int FMT, int DB>
__device__ __forceinline__ void k_operand(const Tile<FMT, DB>& t, int a, int s, uint32_t (&o)[4]) {
  if constexpr (FMT == kKvBf16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = t.k[a][4 * s + i];
  } else if constexpr (FMT == kKvE4m3) {
    const float x = byte_exp2(t.ks[a], 0);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      o[2 * i] = e4m3_scaled<false>(t.k[a][2 * s + i], x);
      o[2 * i + 1] = e4m3_scaled<true>(t.k[a][2 * s + i], x);
    }
  } else {
    const f16x2 x = scale_pair(t.ks[a], s / 2);
    o[0] = e2m1_scaled<0>(t.k[a][s], x);
    o[1] = e2m1_scaled<1>(t.k[a][s], x);
    o[2] = e2m1_scaled<2>(t.k[a][s], x);
    o[3] = e2m1_scaled<3>(t.k[a][s], x);
  }
}

// The lane's V values of token i as 16-bit pairs: o[j] holds d = W r + 2j, + 1.
template <int FMT, int DB>
__device__ __forceinline__ void v_token(const Tile<FMT, DB>& t, int a, int i, uint32_t (&o)[2 * DB]) {
  constexpr int kPairs = 2 * DB;
  if constexpr (FMT == kKvBf16) {
#pragma unroll
    for (int j = 0; j < kPairs; ++j) o[j] = t.v[a][kPairs * i + j];
  } else if constexpr (FMT == kKvE4m3) {
    const float x = byte_exp2(t.vs[a][0], i);
#pragma unroll
    for (int j = 0; j < kPairs; j += 2) {
      o[j] = e4m3_scaled<false>(t.v[a][(kPairs * i + j) / 2], x);
      o[j + 1] = e4m3_scaled<true>(t.v[a][(kPairs * i + j) / 2], x);
    }
  } else {
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
      const f16x2 x = scale_pair(t.vs[a][DB == 3 ? j / 2 : 0], i);
      const int byte = kPairs * i + j;
      const uint32_t w = t.v[a][byte / 4];
      switch (byte % 4) {
        case 0: o[j] = e2m1_scaled<0>(w, x); break;
        case 1: o[j] = e2m1_scaled<1>(w, x); break;
        case 2: o[j] = e2m1_scaled<2>(w, x); break;
        default: o[j] = e2m1_scaled<3>(w, x); break;
      }
    }
  }
}

// Clears what masked tokens hold, so that garbage (NaN codes, infinities) times
// a zero probability stays zero.  ok: bit 4a + i, tokens 4h + i of group a.
template <int FMT, int DB>
__device__ __forceinline__ void clear_masked(Tile<FMT, DB>& t, uint32_t ok) {
  constexpr int kTokenWords = Tile<FMT, DB>::kWords / 4;
#pragma unroll
  for (int a = 0; a < 2; ++a)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool keep = (ok >> (4 * a + i)) & 1u;
      if constexpr (FMT == kKvNvfp4) {  // a zero scale: every code is finite
#pragma unroll
        for (int u = 0; u < Tile<FMT, DB>::kVScales; ++u) t.vs[a][u] &= keep ? ~0u : ~(0xffu << (8 * i));
      } else {
#pragma unroll
        for (int j = 0; j < kTokenWords; ++j) t.v[a][kTokenWords * i + j] = keep ? t.v[a][kTokenWords * i + j] : 0u;
        if constexpr (FMT == kKvE4m3)
          t.vs[a][0] = keep ? t.vs[a][0] : (t.vs[a][0] & ~(0xffu << (8 * i))) | (127u << (8 * i));
      }
    }
}

// Rounded as written: a fused product and difference would take p from a score that is
// not rounded, against a reference that is, and at scores past 2^25 give it any size.
__device__ __forceinline__ float rounded_product(float a, float b) {
#pragma clang fp contract(off)
  return a * b;
}

__device__ __forceinline__ float lane_xor(float v, int off) { return __shfl_xor(v, off); }

// The largest term is set to 2^kOffset, and none passes 2^(kOffset + kSlack).  f16: 2^15;
// terms under 2^-14 lose bits: one below 2^-25 of the largest is taken to within 2^-36 of that
// (half of f16's last step, 2^-25, under the offset).  bf16 has fp32's range: no term passes 1,
// so that sums of n terms stay below n times the largest value, as the definition's do
// (with terms up to 2^8, values from 2^119 / n on gave infinity; same times).
template <int FMT>
struct Softmax {
  static constexpr float kOffset = FMT == kKvNvfp4 ? 11.0f : -8.0f;
  static constexpr float kSlack = FMT == kKvNvfp4 ? 4.0f : 8.0f;
};

// Four outputs of row `qh` of sequence b from their sums, and (d == 0) its lse.
__device__ __forceinline__ void write_out(const AttnParams& a, int b, int qh, int d, float ref, float l, f32x4 acc) {
  const bool some = l > 0.0f || l != l;  // NaN stays NaN
  const float f = some ? a.cache.v_scale / l : 0.0f;
  if (d < a.cache.head_dim) {
    uint16_t* to = a.out + (int64_t)b * a.ldo + (int64_t)qh * a.cache.head_dim + d;
    *reinterpret_cast<uint2*>(to) = make_uint2(pack_bf16x2(acc[0] * f, acc[1] * f), pack_bf16x2(acc[2] * f, acc[3] * f));
  }
  if (d == 0 && a.lse) a.lse[(int64_t)b * a.q_heads + qh] = some ? (ref + __builtin_amdgcn_logf(l)) * kLn2 : kNegInf;
}

// Adds (m, l, v) to running sums under the larger reference.
__device__ __forceinline__ void add_part(float& top, float& sum, f32x4& acc, float m, float l, f32x4 v) {
  const float next = fmaxf(top, m);
  const float fo = top == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(top - next);
  const float fi = m == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(m - next);
  sum = sum * fo + l * fi;
  acc = acc * fo + v * fi;
  top = next;
}

// Joins the partial sums that workgroups wfirst .. wlast left of a unit.  The parts
// are cut into runs over the threads that its values leave over; each thread adds
// its run in workgroup order, kJoinBatch parts a round trip to memory; the runs are
// then added in order through LDS (6 floats a thread).
template <int DP, int kThreads>
__device__ __forceinline__ void join_parts(const AttnParams& a, int wfirst, int wlast, int rows, int b, int q0, float* lds) {
  constexpr int kQuads = DP / 4;
  const int parts = wlast - wfirst + 1, items = rows * kQuads;
  const int runs = min(items >= kThreads ? 1 : kThreads / items, parts);
  const __amdgpu_buffer_rsrc_t buf = part_buffer(a);
  for (int e0 = 0; e0 < items; e0 += kThreads) {   // more than one round: runs == 1
    const int e = e0 + (int)threadIdx.x, run = e / items, item = runs > 1 ? e - run * items : e;
    const bool live = runs > 1 ? run < runs : e < items;
    const int r = live ? item / kQuads : 0, d = live ? 4 * (item - r * kQuads) : 0;
    const int p0 = !live ? 0 : runs > 1 ? parts * run / runs : 0, p1 = !live ? 0 : runs > 1 ? parts * (run + 1) / runs : parts;
    float top = kNegInf, l = 0.0f;
    f32x4 acc{0.0f, 0.0f, 0.0f, 0.0f};
    for (int i = p0; i < p1; i += kJoinBatch) {
      f32x4 ml[kJoinBatch], v[kJoinBatch];
#pragma unroll
      for (int j = 0; j < kJoinBatch; ++j) {
        if (i + j < p1) {
          const int from = part_offset<DP>(a, wfirst + i + j, i + j == 0 ? 1 : 0, r);
          ml[j] = load_part(buf, from);
          v[j] = load_part(buf, from + (4 + d) * 4);
        }
      }
#pragma unroll
      for (int j = 0; j < kJoinBatch; ++j)
        if (i + j < p1) add_part(top, l, acc, ml[j][0], ml[j][1], v[j]);
    }
    if (runs > 1) {
      float* mine = lds + (run * items + item) * 6;
      __syncthreads();
      if (live) {
        mine[0] = top;
        mine[1] = l;
#pragma unroll
        for (int j = 0; j < 4; ++j) mine[2 + j] = acc[j];
      }
      __syncthreads();
      if (live && run == 0) {
        for (int i = 1; i < runs; ++i) {
          const float* other = lds + (i * items + item) * 6;
          add_part(top, l, acc, other[0], other[1], f32x4{other[2], other[3], other[4], other[5]});
        }
      }
    }
    if (live && (runs == 1 || run == 0)) write_out(a, b, q0 + r, d, top, l, acc);
  }
}

// Wavefronts a SIMD; a workgroup fills a CU.  Two keep enough loads in flight, and more
// only make the joins longer: 8 users of up to 4608 tokens of 64-wide E4M3 heads 11.1 us with
// two, 11.3 with one, 12.2 with four; one user over 40,000 tokens of 128-wide NVFP4 heads 17.1,
// 20.6, 17.9 with three.  Narrow NVFP4 heads, with the fewest bytes a step, want three: 32 users over
// 16,384 tokens 61.3 us with two, 55.7 with three, 54.7 with four (and 8 users over up to
// 8192: 12.5, 13.3, 14.3).  Wide bf16 heads have registers for one.
constexpr int waves_per_simd(int fmt, int db) {
  return fmt == kKvBf16 && db == 4 ? 1 : fmt == kKvNvfp4 && db == 1 ? 3 : 2;
}

// The line cut into n runs of nearly equal length, the first `more` one longer.
struct Cut {
  int n, each, more;
};
__device__ __forceinline__ Cut cut_of(int length, int n) {
  const int each = (int)((unsigned)length / (unsigned)n);
  return Cut{n, each, length - each * n};
}
__device__ __forceinline__ int run_start(const Cut& c, int i) { return c.each * i + min(i, c.more); }
__device__ __forceinline__ int run_of(const Cut& c, int place) {
  const int longer = c.more * (c.each + 1);
  const bool in = place < longer;
  return (in ? 0 : c.more) + (int)((unsigned)(in ? place : place - longer) / (unsigned)(in ? c.each + 1 : max(c.each, 1)));
}

// A unit, as much of it as joins need: places [u0, u1) of its tiles, and where its
// rows go.
struct Unit {
  int u0, u1;
  int b, q0, rows;
};

// Inclusive sum over the lanes below: within each row of sixteen by shifts, then
// the rows' last lanes carried into the rows after them.
template <int CTRL, int ROWS>
__device__ __forceinline__ int add_lanes(int v) {
  return v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xf, true);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ int max_lanes(int v) {
  return max(v, __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xf, true));
}
__device__ __forceinline__ int lane_max(int v) {  // of values >= 0, in the last lane
  v = max_lanes<0x111, 0xf>(v);
  v = max_lanes<0x112, 0xf>(v);
  v = max_lanes<0x114, 0xf>(v);
  v = max_lanes<0x118, 0xf>(v);
  v = max_lanes<0x142, 0xa>(v);
  return max_lanes<0x143, 0xc>(v);
}
__device__ __forceinline__ int lane_scan(int v) {
  v = add_lanes<0x111, 0xf>(v);  // row_shr:1, 2, 4, 8
  v = add_lanes<0x112, 0xf>(v);
  v = add_lanes<0x114, 0xf>(v);
  v = add_lanes<0x118, 0xf>(v);
  v = add_lanes<0x142, 0xa>(v);  // row_bcast:15 into rows 1 and 3
  return add_lanes<0x143, 0xc>(v);  // row_bcast:31 into rows 2 and 3
}

// One workgroup's LDS.
template <int DP, int WAVES>
struct Staging {
  // Sums that wavefronts leave (slot: the wavefront), and the beginning of the
  // unit that goes on in another workgroup (slot WAVES).
  float ml[WAVES + 1][kRows][2];                                    // reference and sum
  float o[WAVES + 1][kRows][DP + 4] __attribute__((aligned(16)));
  Unit first, last;          // the units cut by the share's two ends
  int has_first, has_last, last_from, joins[2], from[2], to[2];
};

template <int FMT, int DB>
__global__ __launch_bounds__(256 * waves_per_simd(FMT, DB), (waves_per_simd(FMT, DB))) void attn_kernel(const AttnParams a) {
  using L = KvLayout<FMT, DB>;
  constexpr int kWaves = 4 * waves_per_simd(FMT, DB), kThreads = 64 * kWaves;
  constexpr int kDp = 64 * DB, kE = L::kE, kW = L::kW, kSteps = kE / 8, kQuads = kE / 4;
  __shared__ Staging<kDp, kWaves> lds;

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int qn = lane & 15, h = lane >> 4, d0 = kE * h;
  const int units_per_row = a.cache.heads * a.row_tiles;

  // The line's length, and each lane's stretch of it: `per` rows of the batch.
  const auto len_of = [&](int row) { return row < a.batch ? a.lens[row] : 0; };
  const auto places_in = [&](int row, int len) {
    return row < a.batch ? span_of(a, len).tiles + kLead : 0;  // of a unit
  };
  if (tid == 0) lds.has_first = lds.has_last = lds.joins[0] = lds.joins[1] = 0;
  wait_vmcnt_lgkm0<63>();
  barrier_only();
  const int per = (a.batch + 63) / 64;
  // A window of 64 rows from row `win` on, which starts at place `win_start`: the
  // lanes' lengths, places of a unit and of the row, and inclusive sums of places.
  int win = 0, win_start = 0, win_len = 0, win_unit = 0, win_mine = 0, win_upto = 0;
  const auto move_window = [&](int row, int start) {
    win = row;
    win_start = start;
    win_len = len_of(row + lane);
    win_unit = places_in(row + lane, win_len);
    win_mine = win_unit * units_per_row;
    win_upto = lane_scan(win_mine);
  };
  int mine, upto, longest;                  // of each lane's `per` rows
  if (per == 1) {
    move_window(0, 0);
    mine = win_mine;
    upto = win_upto;
    longest = win_unit;
  } else {
    mine = longest = 0;
#pragma unroll 4
    for (int i = 0; i < per; ++i) {
      const int unit = places_in(lane * per + i, len_of(lane * per + i));
      mine += unit * units_per_row;
      longest = max(longest, unit);
    }
    upto = lane_scan(mine);
  }
  const int total = __builtin_amdgcn_readlane(upto, 63);
  // (The nearest power of two, of places in one of 2^parts_log parts.)
  const unsigned longest_unit = (unsigned)__builtin_amdgcn_readlane(lane_max(longest), 63);
  const int share_log =
      min(max(31 - __builtin_clz((longest_unit + longest_unit / 2) >> a.parts_log | 1u), kShareMinLog), kShareMaxLog);
  const int w = blockIdx.x;
  const Cut shares = cut_of(total, min((int)gridDim.x, max(total >> share_log, a.batch * units_per_row)));
  if (w >= shares.n) return;
  // The row that holds a place, where it starts and how long its units are; the
  // window moves there if it is elsewhere.
  struct Row {
    int b, start, unit;
  };
  const auto row_at = [&](int place) {
    if (place < win_start || place >= win_start + __builtin_amdgcn_readlane(win_upto, 63)) {
      const int in = __builtin_ctzll(__ballot(upto > place));
      move_window(in * per, __builtin_amdgcn_readlane(upto - mine, in));
      while (place >= win_start + __builtin_amdgcn_readlane(win_upto, 63))  // (ends in the lane's own rows)
        move_window(win + 64, win_start + __builtin_amdgcn_readlane(win_upto, 63));
    }
    const int at = __builtin_ctzll(__ballot(win_start + win_upto > place));
    return Row{win + at, win_start + __builtin_amdgcn_readlane(win_upto - win_mine, at),
               __builtin_amdgcn_readlane(win_unit, at)};
  };
  // The workgroup's share [s0, s1), an end moved to a unit's end if that unit is
  // short; the wavefront's run [g0, g1) of it, and the row where that starts.  (Short:
  // where units are about as many as workgroups, up to two tiles a wavefront; where
  // they are fewer, cutting gives work to idle CUs, and short is less.  64 users of up to
  // 300 tokens, 4 kv heads of 192: 14.5 us with one tile a wavefront, 11.7 with two; 8 users of up
  // to 768 tokens: 9.7 and 12.5.  256 users of up to 512 tokens, 8 heads of 128: 24.6 and 21.8.
  // Heads of 64 are quicker to read than to join: 8 users of up to 400 tokens 7.7 and 7.0.)
  const int short_unit = kLead + (2 * a.batch * units_per_row >= kCus ? 2 * kWaves : DB == 1 ? 16 : 8);
  int s0 = 0, s1 = 0, g0 = 0, g1 = 0;
  Cut runs{kWaves, 0, 0};
  Row r0{0, 0, 1};
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    if (k == 2) {
      if (s0 >= s1) return;
      runs = cut_of(s1 - s0, kWaves);
      g0 = s0 + run_start(runs, wave);
      g1 = s0 + run_start(runs, wave + 1);
    }
    const int place = k == 2 ? g0 : run_start(shares, w + k);
    r0 = row_at(min(place, total - 1));
    const int into = (int)((unsigned)(place - r0.start) % (unsigned)r0.unit);
    const bool moved = k < 2 && place < total && r0.unit <= short_unit;
    const int end = !moved ? place : 2 * into < r0.unit ? place - into : place - into + r0.unit;
    if (k == 0) s0 = end;
    else if (k == 1) s1 = end;
  }
  int b = r0.b, row_start = r0.start;

  // What is left in registers at the end: the beginning of a unit that goes on.
  f32x4 o[kW];
  float ref = kNegInf, sum = 0.0f;
  Unit tail{0, 0, 0, 0, 0};
  // o[j][i] is d = W (4h + i) + j of query q: the lane's quad u is d0 + 4u.
  const auto quad = [&](int u) {
    const int i = 4 * u / kW, j = 4 * u % kW;
    return f32x4{o[j][i], o[j + 1][i], o[j + 2][i], o[j + 3][i]};
  };

  for (int g = g0; g < g1;) {
    if (b - win >= 64) move_window(b, row_start);
    const Span sp = span_of(a, __builtin_amdgcn_readlane(win_len, b - win));
    const int places = sp.tiles + kLead, row_end = row_start + places * units_per_row;
    if (g >= row_end) {
      row_start = row_end;
      ++b;
      continue;
    }
    const int unit = (int)((unsigned)(g - row_start) / (unsigned)places);
    const int u0 = row_start + unit * places + kLead, u1 = u0 + sp.tiles;
    g = max(g, u0);
    const int stop = min(u1, g1);
    if (g >= stop) break;                       // the run ends before the unit's first tile
    const int head = a.row_tiles > 1 ? unit / a.row_tiles : unit, rt = unit - head * a.row_tiles;
    const int rows = min(a.group - rt * kRows, kRows), q0 = head * a.group + rt * kRows;
    const int first = g - u0, count = stop - g;

    // Queries: lane (q, h) holds values E h .. E h + E - 1 of row q.
    uint32_t qv[kE / 2];
    const int d_here = a.cache.head_dim - kE * h;  // values of this lane inside the head
    const bool in_head = qn < rows && d_here > 0;  // other lanes and values: zeros, from addresses inside
    const uint16_t* qp = a.q + (int64_t)b * a.ldq + (in_head ? (q0 + qn) * a.cache.head_dim + kE * h : q0 * a.cache.head_dim);
    const int last = in_head ? d_here - 8 : 0;
#pragma unroll
    for (int i = 0; i < kE / 8; ++i) {
      const u32x4 x = load16(qp + min(8 * i, last));
#pragma unroll
      for (int j = 0; j < 4; ++j) qv[4 * i + j] = in_head && 8 * i <= last ? x[j] : 0u;
    }
    // Page lookups: lane j holds the group of step it + j / 2, half j & 1, for 32
    // steps from the last multiple of 32; -1: none there.
    int looked_up = -1;
    const auto look_up = [&](int it, int (&group)[2]) {
      if ((it & 31) == 0) {
        const int tok = sp.base + (first + it + (lane >> 1)) * kTile + (lane & 1) * kKvGroup;
        looked_up = -1;
        if (it + (lane >> 1) < count && tok < sp.end) {
          const int tg = tok / kKvGroup, pg = tg / a.cache.gpp;
          const int page = a.table[(int64_t)b * a.table_width + pg];
          if (page >= 0 && page < a.cache.pages)
            looked_up = (page * a.cache.heads + head) * a.cache.gpp + (tg - pg * a.cache.gpp);
        }
      }
      group[0] = __builtin_amdgcn_readlane(looked_up, 2 * (it & 31));
      group[1] = __builtin_amdgcn_readlane(looked_up, 2 * (it & 31) + 1);
    };
    GroupBuffers from[2];
    const auto to_load = [&](const int (&group)[2]) {
      from[0] = group_buffers<FMT, DB>(a.cache, group[0]);
      from[1] = group_buffers<FMT, DB>(a.cache, group[1]);
    };

    // K of the next step is loaded once this step's scores are formed, V of the
    // next once this step's V is in its operands: one tile of registers, and
    // loads in flight all the time.  The last step loads from empty buffers.
    Tile<FMT, DB> t;
    int group[2];
    look_up(0, group);
    to_load(group);
    // (In the loop's own order, so that its waits count the same loads on entry.)
    load_k<FMT, DB>(from, lane, t);
    __builtin_amdgcn_sched_barrier(0);
    load_v<FMT, DB>(from, lane, t);
    __builtin_amdgcn_sched_barrier(0);
    int score_exp = a.score_exp;
    if constexpr (FMT == kKvNvfp4) {
      // bf16 -> f16: a power of two per row puts its largest magnitude at
      // 2^14 .. 2^15; values down to 2^-28 of it stay exact.
      u16x2 pair{0, 0};
#pragma unroll
      for (int i = 0; i < kE / 2; ++i) pair = __builtin_elementwise_max(pair, __builtin_bit_cast(u16x2, qv[i] & 0x7fff7fffu));
      uint32_t big = (uint32_t)(pair[0] > pair[1] ? pair[0] : pair[1]) << 16;
      big = max(big, (uint32_t)__shfl_xor((int)big, 16));
      big = max(big, (uint32_t)__shfl_xor((int)big, 32));
      // (Below 2^-112 the power stays 2^126: the smallest bf16 number, 2^-133, is then 2^-7.)
      int e = (int)(big >> 23) - 127 - 14;
      e = e < -126 ? -126 : e > 112 ? 112 : e;
      const float down = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
      for (int i = 0; i < kE / 2; ++i) {
        const f16x2 p{(_Float16)(bf16_lo(qv[i]) * down), (_Float16)(bf16_hi(qv[i]) * down)};
        qv[i] = __builtin_bit_cast(uint32_t, p);
      }
      score_exp += e;
    }
    // One product of the scales, whatever their sizes; where it passes fp32's range, zero products stay zero.
    const float score_scale = fminf(__builtin_amdgcn_ldexpf(a.score_factor, score_exp), kFltMax);

#pragma unroll
    for (int i = 0; i < kW; ++i) o[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    ref = kNegInf;
    sum = 0.0f;
    float shift = 0.0f;

    for (int it = 0; it < count; ++it) {
      const int tok0 = sp.base + (first + it) * kTile;
      const bool has0 = group[0] >= 0, has1 = group[1] >= 0;
      const bool whole = has0 && has1 && tok0 >= sp.begin && tok0 + kTile <= sp.end;
      if (it + 1 < count) look_up(it + 1, group);
      else group[0] = group[1] = -1;
      to_load(group);
      uint32_t okbits = 0xffu;
      if (!whole) {
        okbits = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int tok = tok0 + (i / 4) * kKvGroup + 4 * h + i % 4;
          okbits |= ((i / 4 ? has1 : has0) && tok >= sp.begin && tok < sp.end) ? 1u << i : 0u;
        }
      }

      // Scores.
      float x[8];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        f32x4 acc{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          uint32_t op[4];
          k_operand<FMT, DB>(t, half, s, op);
          acc = mma<FMT>(op, &qv[4 * s], acc);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) x[4 * half + i] = rounded_product(acc[i], score_scale);
      }
      load_k<FMT, DB>(from, lane, t);
      if (!whole) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = (okbits >> i) & 1u ? x[i] : kNegInf;
      }
      float top = x[0];
#pragma unroll
      for (int i = 1; i < 8; ++i) top = fmaxf(top, x[i]);
      // (Differences of scores are exact where a bound on them matters; sums with the
      // reference would be rounded to the scores' own steps.)
      if (__any(top - ref > Softmax<FMT>::kOffset + Softmax<FMT>::kSlack)) {
        top = fmaxf(top, lane_xor(top, 16));
        top = fmaxf(top, lane_xor(top, 32));
        // (Scores past 2^27 have steps of 16 and more: the offset may round past the range.)
        const float below = top - Softmax<FMT>::kOffset;
        const float next = fmaxf(ref, top - below > Softmax<FMT>::kOffset + Softmax<FMT>::kSlack ? top : below);
        const float alpha = next == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(ref - next);
        ref = next;
        shift = ref == kNegInf ? 0.0f : ref;
        sum *= alpha;
#pragma unroll
        for (int i = 0; i < kW; ++i) o[i] *= alpha;
      }
      float p[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        p[i] = __builtin_amdgcn_exp2f(x[i] - shift);
        sum += p[i];
      }
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (FMT == kKvNvfp4) {
          hi[i] = __builtin_bit_cast(uint32_t, f16x2{(_Float16)p[2 * i], (_Float16)p[2 * i + 1]});
        } else {
          hi[i] = pack_bf16x2(p[2 * i], p[2 * i + 1]);
          lo[i] = pack_bf16x2(p[2 * i] - bf16_lo(hi[i]), p[2 * i + 1] - bf16_hi(hi[i]));
        }
      }

      // O^T += V^T P^T: step j takes d = W r + j, its eight tokens gathered by
      // byte permutes from the tokens' pairs.
      if (!whole) clear_masked<FMT, DB>(t, okbits);
      uint32_t vt[8][2 * DB];
#pragma unroll
      for (int i = 0; i < 8; ++i) v_token<FMT, DB>(t, i / 4, i % 4, vt[i]);
      uint32_t op[kW][4];
#pragma unroll
      for (int j = 0; j < kW; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          op[j][i] = __builtin_amdgcn_perm(vt[2 * i + 1][j / 2], vt[2 * i][j / 2], j % 2 ? 0x07060302u : 0x05040100u);
      load_v<FMT, DB>(from, lane, t);
#pragma unroll
      for (int j = 0; j < kW; ++j) {
        o[j] = mma<FMT>(op[j], hi, o[j]);
        if constexpr (FMT != kKvNvfp4) o[j] = mma<FMT>(op[j], lo, o[j]);
      }
    }

    sum += lane_xor(sum, 16);
    sum += lane_xor(sum, 32);
    if (u0 < g0 || u1 > s1) {
      // The end, or a stretch, of a unit that an earlier wavefront began; or the
      // beginning of one that goes on in another workgroup.
      const int slot = u0 < g0 ? wave : kWaves;
      if (qn < rows) {
        if (h == 0) {
          lds.ml[slot][qn][0] = ref;
          lds.ml[slot][qn][1] = sum;
        }
#pragma unroll
        for (int u = 0; u < kQuads; ++u) *reinterpret_cast<f32x4*>(&lds.o[slot][qn][d0 + 4 * u]) = quad(u);
      }
      if (lane == 0 && u0 < s0 && g == s0) {
        lds.first = Unit{u0, u1, b, q0, rows};
        lds.has_first = 1;
      }
      if (lane == 0 && u0 >= g0) {
        lds.last = Unit{u0, u1, b, q0, rows};
        lds.has_last = 1;
        lds.last_from = wave + 1;
      }
    } else if (u1 > g1) {
      tail = Unit{u0, u1, b, q0, rows};
    } else if (qn < rows) {
#pragma unroll
      for (int u = 0; u < kQuads; ++u) write_out(a, b, q0 + qn, d0 + 4 * u, ref, sum, quad(u));
    }
    g = stop;
  }
  __syncthreads();

  // One past the last wavefront with a place before u1 (runs without a place are the
  // share's last).
  const auto wave_end = [&](int u1) {
    return u1 >= s1 ? (runs.each > 0 ? kWaves : runs.more) : run_of(runs, u1 - 1 - s0) + 1;
  };
  if (tail.rows > 0) {
    // A unit inside the share: its beginning, in registers, and what the
    // wavefronts after it left.
    f32x4 acc[kQuads];
#pragma unroll
    for (int u = 0; u < kQuads; ++u) acc[u] = quad(u);
    const int from = wave + 1, end = wave_end(tail.u1);
    float top = ref;
    for (int i = from; i < end; ++i) top = fmaxf(top, lds.ml[i][qn][0]);
    const float fo = ref == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(ref - top);
    sum *= fo;
#pragma unroll
    for (int u = 0; u < kQuads; ++u) acc[u] *= fo;
#pragma unroll 2
    for (int i = from; i < end; ++i) {
      const float m = lds.ml[i][qn][0];
      const float f = m == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(m - top);
      sum += lds.ml[i][qn][1] * f;
#pragma unroll
      for (int u = 0; u < kQuads; ++u) acc[u] += *reinterpret_cast<const f32x4*>(&lds.o[i][qn][d0 + 4 * u]) * f;
    }
    if (qn < tail.rows) {
#pragma unroll
      for (int u = 0; u < kQuads; ++u) write_out(a, tail.b, tail.q0 + qn, d0 + 4 * u, top, sum, acc[u]);
    }
  }
  const int has_first = lds.has_first, has_last = lds.has_last;
  if (!has_first && !has_last) return;
  // The units cut by the share's two ends, by all threads: each four values of a
  // row, from slot kWaves (the beginning of the second) and those of the wavefronts
  // from `from` on.
  const __amdgpu_buffer_rsrc_t buf = part_buffer(a);
#pragma unroll 1
  for (int side = has_first ? 0 : 1; side <= has_last; ++side) {
    const int from = side ? lds.last_from - 1 : 0, rows = side ? lds.last.rows : lds.first.rows;
    const int end = wave_end(side ? lds.last.u1 : lds.first.u1);
    for (int e = tid; e < rows * (kDp / 4); e += kThreads) {
      const int r = e / (kDp / 4), d = 4 * (e - r * (kDp / 4));
      const auto slot = [&](int i) { return side && i == from ? kWaves : i; };
      float top = kNegInf, l = 0.0f;
#pragma unroll 1
      for (int i = from; i < end; ++i) top = fmaxf(top, lds.ml[slot(i)][r][0]);
      f32x4 acc{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
      for (int i = from; i < end; ++i) {
        const int k = slot(i);
        const float m = lds.ml[k][r][0];
        const float f = m == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(m - top);
        l += lds.ml[k][r][1] * f;
        acc += *reinterpret_cast<const f32x4*>(&lds.o[k][r][d]) * f;
      }
      const int to = part_offset<kDp>(a, w, side, r);
      if (d == 0) store_part(buf, to, f32x4{top, l, 0.0f, 0.0f});
      store_part(buf, to + (4 + d) * 4, acc);
    }
  }
  __atomic_signal_fence(__ATOMIC_SEQ_CST);  // keep the stores of partial sums above the wait
  __builtin_amdgcn_s_waitcnt(0);            // they have completed
  __syncthreads();
  if (tid < 2 && (tid ? has_last : has_first)) {
    // A unit's counter is that of the workgroup where it begins; the last to
    // arrive finds all others counted and leaves it at zero.
    const Unit u = tid ? lds.last : lds.first;
    const int from = run_of(shares, u.u0), to = run_of(shares, u.u1 - 1);
    const unsigned before = __hip_atomic_fetch_add(a.counters + from, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (before == (unsigned)(to - from)) {
      __hip_atomic_store(a.counters + from, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      lds.joins[tid] = 1;
      lds.from[tid] = from;
      lds.to[tid] = to;
    }
  }
  __syncthreads();
  const int joins[2] = {lds.joins[0], lds.joins[1]};
#pragma unroll 1
  for (int side = joins[0] ? 0 : 1; side <= joins[1]; ++side) {
    const Unit u = side ? lds.last : lds.first;
    join_parts<kDp, kThreads>(a, lds.from[side], lds.to[side], u.rows, u.b, u.q0, &lds.o[0][0][0]);
  }
}

int row_tiles_of(const AttnLaunch& a) { return (a.q_heads / a.cache.heads + kRows - 1) / kRows; }

int waves_of(const AttnLaunch& a) { return 4 * waves_per_simd(a.format, (a.cache.head_dim + 63) / 64); }

// The places of the line, at the longest possible lengths.
int64_t places_of(const AttnLaunch& a) {
  int64_t tokens = a.table_width * a.cache.page_size;
  if (a.window > 0 && a.window + kKvGroup < tokens) tokens = a.window + kKvGroup;
  const int64_t tiles = tokens > kTile ? (tokens + kTile - 1) / kTile : 1;
  return a.batch * a.cache.heads * row_tiles_of(a) * (tiles + kLead);
}

// Workgroups of a launch: one a CU, or fewer if the longest possible lengths have
// no work for them.
int workgroups_of(const AttnLaunch& a) {
  const int64_t shares = places_of(a) >> kShareMinLog, units = a.batch * a.cache.heads * row_tiles_of(a);
  const int64_t all = shares > units ? shares : units;
  return (int)(all < kCus ? all : kCus);
}

int part_rows_of(const AttnLaunch& a) {
  const int g = a.q_heads / a.cache.heads;
  return g < kRows ? g : kRows;
}

size_t part_bytes_of(const AttnLaunch& a) {
  const size_t dp = (size_t)((a.cache.head_dim + 63) / 64) * 64;
  return (size_t)workgroups_of(a) * 2 * part_rows_of(a) * (dp + 4) * sizeof(float);
}

// Of the parts that a unit is cut into (see kShareMinLog): the power of two nearest to
// those that its join reads in one round trip.
int parts_log_of(const AttnLaunch& a) {
  const int quads = (a.cache.head_dim + 63) / 64 * 16;
  const int trip = kJoinBatch * (64 * waves_of(a) / (part_rows_of(a) * quads));
  const int log = 31 - __builtin_clz((unsigned)(trip + trip / 2) | 1u);
  return log < kPartsMinLog ? kPartsMinLog : log > kPartsMaxLog ? kPartsMaxLog : log;
}

template <int FMT, int DB>
void attn_launch(const AttnLaunch& a, hipStream_t s) {
  AttnParams p;
  p.cache = a.cache;
  p.q = a.q;
  p.table = a.table;
  p.lens = a.lens;
  p.out = a.out;
  p.lse = a.lse;
  p.counters = static_cast<unsigned*>(a.ws);
  p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(a.ws) + kAttnCounterBytes);
  p.ldq = a.ldq;
  p.ldo = a.ldo;
  p.table_width = a.table_width;
  p.batch = (int32_t)a.batch;
  p.q_heads = a.q_heads;
  p.group = a.q_heads / a.cache.heads;
  p.row_tiles = row_tiles_of(a);
  p.window = a.window;
  p.part_rows = part_rows_of(a);
  p.part_bytes = (int32_t)part_bytes_of(a);
  p.parts_log = parts_log_of(a);
  p.score_factor = (float)std::frexp(a.scale * kLog2e * a.cache.k_scale, &p.score_exp);
  hipLaunchKernelGGL((attn_kernel<FMT, DB>), dim3((unsigned)workgroups_of(a)), dim3(64 * waves_of(a)), 0, s, p);
}

template <int FMT>
void attn_launch_db(const AttnLaunch& a, hipStream_t s) {
  switch ((a.cache.head_dim + 63) / 64) {
    case 1: attn_launch<FMT, 1>(a, s); break;
    case 2: attn_launch<FMT, 2>(a, s); break;
    case 3: attn_launch<FMT, 3>(a, s); break;
    default: attn_launch<FMT, 4>(a, s); break;
  }
}

}  // namespace

bool attn_fits(const AttnLaunch& a) { return places_of(a) < (int64_t(1) << 31); }

size_t attn_workspace_bytes(const AttnLaunch& a) { return kAttnCounterBytes + part_bytes_of(a); }

hipError_t launch_attn_decode(const AttnLaunch& a, hipStream_t s) {
  switch (a.format) {
    case kKvBf16: attn_launch_db<kKvBf16>(a, s); break;
    case kKvE4m3: attn_launch_db<kKvE4m3>(a, s); break;
    default: attn_launch_db<kKvNvfp4>(a, s); break;
  }
  return hipGetLastError();
}

}  // namespace nvfp4
