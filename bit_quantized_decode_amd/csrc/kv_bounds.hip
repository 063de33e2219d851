// The bounds of a page's keys (nvfp4_kv_bounds): for each kv head and channel, the smallest and the
// largest value that the page's tokens hold.
//
// Every value of every cache format is a bf16 number but for the tensor scale (E4M3 times a power of two; E2M1 times
// E4M3 has six significant bits), so that bounds in bf16 are exact.  A 16-bit float with all but the
// sign bit flipped where it is negative orders as an integer: two channels' bounds move by one packed
// minimum and one packed maximum a word.  NVFP4's products are exact in f16 too and move by packed f16 minima and
// maxima; those pass over NaN, which only a block's scale brings in, so that the scales are looked at.
//
// One wavefront takes one page of one kv head.  A lane holds E channels of every sixteenth token (kv_layout.h);
// at the end the sixteen lanes of a channel set are reduced by exchanges that halve the words each lane
// keeps, so that each ends up with its own part of the result.
//
// Bound by the cache's bytes, for NVFP4 by the arithmetic: 131,072 tokens of 8 heads of 128 in pages of 64 (8.4 MB of bounds)
// 46 us of bf16 (6.0 TB/s), 31 of E4M3 (4.6), 19 of NVFP4 (4.4; 20.4 by the ordered integers of the other formats); in pages of
// 16, with four times the bounds and the reductions, 86, 52 and 51.  Up to 512 workgroups that loop over the list are no
// faster (NVFP4 pages of 64 21, E4M3 pages of 16 58).
#include "attn_kernel.h"

namespace nvfp4 {
namespace {

typedef int16_t i16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t ordered(uint32_t w) {  // and back
  const i16x2 v = __builtin_bit_cast(i16x2, w);
  return w ^ (__builtin_bit_cast(uint32_t, v >> i16x2{15, 15}) & 0x7fff7fffu);
}
template <int FMT, bool MAX>
__device__ __forceinline__ uint32_t pick(uint32_t a, uint32_t b) {
  if constexpr (FMT == kKvNvfp4) {
    const f16x2 x = __builtin_bit_cast(f16x2, a), y = __builtin_bit_cast(f16x2, b);
    return __builtin_bit_cast(uint32_t, MAX ? __builtin_elementwise_max(x, y) : __builtin_elementwise_min(x, y));
  }
  const i16x2 x = __builtin_bit_cast(i16x2, a), y = __builtin_bit_cast(i16x2, b);
  return __builtin_bit_cast(uint32_t, MAX ? __builtin_elementwise_max(x, y) : __builtin_elementwise_min(x, y));
}

// Lane exchanges within sixteen lanes that flip bit 3, 2, 1 or 0 of the lane (and, for the first
// two, those below it, which does not matter to a reduction).
template <int STEP>
__device__ __forceinline__ uint32_t partner(uint32_t v) {
  constexpr int kCtrl = STEP == 0 ? 0x140 : STEP == 1 ? 0x141 : STEP == 2 ? 0x4e : 0xb1;
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, 0xf, 0xf, true);
}
template <int FMT, int STEP, int N, bool MAX>
__device__ __forceinline__ void reduce(uint32_t* w, int r) {
  if constexpr (STEP < 4) {
    if constexpr (N % 2 == 0) {
      const bool upper = (r >> (3 - STEP)) & 1;
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        const uint32_t mine = upper ? w[i + N / 2] : w[i], other = upper ? w[i] : w[i + N / 2];
        w[i] = pick<FMT, MAX>(mine, partner<STEP>(other));
      }
      reduce<FMT, STEP + 1, N / 2, MAX>(w, r);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] = pick<FMT, MAX>(w[i], partner<STEP>(w[i]));
      reduce<FMT, STEP + 1, N, MAX>(w, r);
    }
  }
}
// What a lane is left with: N words from word `at` on.
constexpr int words_left(int n) { return n % 16 == 0 ? n / 16 : n % 8 == 0 ? n / 8 : n; }
template <int STEP, int N>
__device__ __forceinline__ int word_at(int r) {
  if constexpr (STEP == 4 || N % 2 != 0) return 0;
  else return ((r >> (3 - STEP)) & 1) * (N / 2) + word_at<STEP + 1, N / 2>(r);
}

// An f16 pair of a few significant bits as a bf16 pair.
__device__ __forceinline__ uint32_t f16_to_bf16(uint32_t w) {
  const f16x2 v = __builtin_bit_cast(f16x2, w);
  return pack_exact_bf16x2((float)v[0], (float)v[1]);
}

template <int FMT, int DB>
__global__ __launch_bounds__(256) void bounds_kernel(const KvBoundsLaunch a) {
  using L = KvLayout<FMT, DB>;
  constexpr int kE = L::kE, kN = kE / 2, kLeft = words_left(kN);
  const int lane = threadIdx.x & 63, r = lane & 15, h = lane >> 4;
  const int64_t item = workgroup() * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t at = item / a.cache.heads;
  if (at >= a.n) return;
  const int head = (int)(item - at * a.cache.heads), page = a.pages[at];
  if (page < 0 || page >= a.cache.pages) return;
  const int first = (page * a.cache.heads + head) * a.cache.gpp;  // pages * heads * groups of a page stay below 2^30

  uint32_t low[kN], high[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    low[i] = FMT == kKvNvfp4 ? 0x7c007c00u : 0x7fff7fffu;
    high[i] = FMT == kKvNvfp4 ? 0xfc00fc00u : 0x80008000u;
  }
  uint32_t nan = 0;                     // NVFP4: byte i, whether the lane's block i has a NaN scale
  Tile<FMT, DB> t;
  // Two sixteens at a time; the second of an odd last pair is the first again, which changes nothing.
#pragma unroll 2
  for (int g = 0; g < a.cache.gpp; g += 2) {
    const GroupBuffers from[2] = {group_buffers<FMT, DB>(a.cache, first + g),
                                  group_buffers<FMT, DB>(a.cache, first + min(g + 1, a.cache.gpp - 1))};
    load_k<FMT, DB>(from, lane, t);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      // (0x7f is the one magnitude whose sum with 1 reaches a byte's top bit.)
      if constexpr (FMT == kKvNvfp4) nan |= ((t.ks[half] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
#pragma unroll
      for (int s = 0; s < kE / 8; ++s) {
        uint32_t op[4];
        k_operand<FMT, DB>(t, half, s, op);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t v = FMT == kKvNvfp4 ? op[i] : ordered(op[i]);
          low[4 * s + i] = pick<FMT, false>(low[4 * s + i], v);
          high[4 * s + i] = pick<FMT, true>(high[4 * s + i], v);
        }
      }
    }
  }
  reduce<FMT, 0, kN, false>(low, r);
  reduce<FMT, 0, kN, true>(high, r);
  if constexpr (FMT == kKvNvfp4) {
    nan |= partner<0>(nan);
    nan |= partner<1>(nan);
    nan |= partner<2>(nan);
    nan |= partner<3>(nan);
  }
  const int d = kE * h + 2 * word_at<0, kN>(r);
  uint16_t* to = a.bounds + ((int64_t)page * a.cache.heads + head) * 2 * a.cache.head_dim + d;
#pragma unroll
  for (int i = 0; i < kLeft; ++i) {
    uint32_t lo, hi;
    if constexpr (FMT == kKvNvfp4) {
      const int block = (word_at<0, kN>(r) + i) / 8;
      const bool bad = (nan >> (8 * block) & 0x80u) != 0;
      lo = bad ? 0x7fc07fc0u : f16_to_bf16(low[i]);
      hi = bad ? 0x7fc07fc0u : f16_to_bf16(high[i]);
    } else {
      lo = ordered(low[i]);
      hi = ordered(high[i]);
    }
    // A channel with a NaN has it in both bounds: ordered, NaN lies beyond infinity at one end.
    const uint32_t nan_lo = ((lo & 0x7fffu) > 0x7f80u || (hi & 0x7fffu) > 0x7f80u) ? 0x7fc0u : 0u;
    const uint32_t nan_hi = ((lo & 0x7fff0000u) > 0x7f800000u || (hi & 0x7fff0000u) > 0x7f800000u) ? 0x7fc00000u : 0u;
    if (d + 2 * i < a.cache.head_dim) {
      *reinterpret_cast<uint32_t*>(to + 2 * i) = lo | nan_lo | nan_hi;
      *reinterpret_cast<uint32_t*>(to + a.cache.head_dim + 2 * i) = hi | nan_lo | nan_hi;
    }
  }
}

template <int FMT>
void bounds_launch(const KvBoundsLaunch& a, hipStream_t s) {
  const dim3 grid = grid_of((a.n * a.cache.heads + 3) / 4), threads(256);
  switch ((a.cache.head_dim + 63) / 64) {
    case 1: hipLaunchKernelGGL((bounds_kernel<FMT, 1>), grid, threads, 0, s, a); break;
    case 2: hipLaunchKernelGGL((bounds_kernel<FMT, 2>), grid, threads, 0, s, a); break;
    case 3: hipLaunchKernelGGL((bounds_kernel<FMT, 3>), grid, threads, 0, s, a); break;
    default: hipLaunchKernelGGL((bounds_kernel<FMT, 4>), grid, threads, 0, s, a); break;
  }
}

}  // namespace

hipError_t launch_kv_bounds(const KvBoundsLaunch& a, hipStream_t s) {
  switch (a.format) {
    case kKvBf16: bounds_launch<kKvBf16>(a, s); break;
    case kKvE4m3: bounds_launch<kKvE4m3>(a, s); break;
    default: bounds_launch<kKvNvfp4>(a, s); break;
  }
  return hipGetLastError();
}

}  // namespace nvfp4
