// Rotary positions on the device: the angle of a pair, its sine and cosine, and
// the turn of eight pairs.
#pragma once

#include "device_common.h"

namespace nvfp4 {

// pos * f modulo one turn, in 2^-32 turns.  f is a 64-bit fraction of a turn, so
// the product modulo 2^64 is the exact fraction of pos * f; its upper word is
// what is kept (2^-32 turns = 1.5e-9 rad).  A negative pos is pos_u - 2^32, which
// takes f's lower word off the upper one.
__device__ __forceinline__ uint32_t rope_phase(int32_t pos, uint64_t f) {
  const uint32_t p = (uint32_t)pos, lo = (uint32_t)f, hi = (uint32_t)(f >> 32);
  const uint32_t u = __umulhi(p, lo) + p * hi;
  return pos < 0 ? u - lo : u;
}

// Sine and cosine of 2 pi phase / 2^32.  The phase splits into a quarter turn
// and a rest |x| <= pi/4, exact in integers; there the Taylor sums to x^9 and
// x^10 are within 2e-9 and 2e-10, below the fp32 rounding (6e-8) of their terms.
__device__ __forceinline__ void sincos_phase(uint32_t phase, float& s, float& c) {
  const uint32_t quarter = (phase + 0x20000000u) >> 30;
  const float x = (float)(int32_t)(phase - (quarter << 30)) * 1.46291807926715968e-9f;  // 2 pi / 2^32
  const float z = x * x;
  const float ps = x + x * z * (-1.66666667e-1f + z * (8.33333333e-3f + z * (-1.98412698e-4f + z * 2.75573192e-6f)));
  const float pc =
      1.0f + z * (-0.5f + z * (4.16666667e-2f + z * (-1.38888889e-3f + z * (2.48015873e-5f - z * 2.75573192e-7f))));
  const float a = (quarter & 1u) ? pc : ps, b = (quarter & 1u) ? ps : pc;
  s = (quarter & 2u) ? -a : a;
  c = ((quarter + 1u) & 2u) ? -b : b;
}

// Eight consecutive values at element `off` of p (16-byte aligned), in fp32.
// STREAM: read once, by a non-temporal load.
template <bool BF16, bool STREAM = false>
__device__ __forceinline__ void load8(const void* p, int64_t off, float* v) {
  if (BF16) {
    const uint16_t* q = static_cast<const uint16_t*>(p) + off;
    const u32x4 a = STREAM ? load16_stream(q) : load16(q);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_lo(a[i]);
      v[2 * i + 1] = bf16_hi(a[i]);
    }
  } else {
    const float* q = static_cast<const float*>(p) + off;
    const u32x4 a = STREAM ? load16_stream(q) : load16(q), b = STREAM ? load16_stream(q + 4) : load16(q + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = __uint_as_float(a[i]);
      v[4 + i] = __uint_as_float(b[i]);
    }
  }
}

template <bool BF16>
__device__ __forceinline__ void store8(void* p, int64_t off, const float* v) {
  if (BF16) {
    u32x4 a;
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p) + off) = a;
  } else {
    f32x4* q = reinterpret_cast<f32x4*>(static_cast<float*>(p) + off);
    q[0] = f32x4{v[0], v[1], v[2], v[3]};
    q[1] = f32x4{v[4], v[5], v[6], v[7]};
  }
}

// A head is cut into units of sixteen values.  Unit u < rot/16 is eight pairs: in
// the half layout values 8u + [0, 8) and rot/2 + 8u + [0, 8), interleaved 16u +
// [0, 16).  The other units are values 16u + [0, 16), which only move.
struct RopeUnit {
  int first, second;  // where its two runs of eight values start
  bool turned;
};
__device__ __forceinline__ RopeUnit rope_unit(int u, int rot, bool interleaved) {
  RopeUnit r;
  r.turned = 16 * u < rot;
  const bool half = r.turned && !interleaved;
  r.first = half ? 8 * u : 16 * u;
  r.second = half ? rot / 2 + 8 * u : 16 * u + 8;
  return r;
}

// The eight (cosine, sine)s of unit u at a position, times the magnitude.
__device__ __forceinline__ void rope_angles(const uint64_t* __restrict__ freqs, int u, int32_t pos, float magnitude,
                                            float sign, float (&c)[8], float (&s)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float si, co;
    sincos_phase(rope_phase(pos, freqs[8 * u + i]), si, co);
    c[i] = co * magnitude;
    s[i] = si * magnitude * sign;
  }
}

// Turns a unit's pairs in place.  (The empty statements differ, so that the
// compiler does not merge the two layouts into one code with v indexed at run
// time, which puts it into scratch memory.)
__device__ __forceinline__ void rope_turn(float (&v)[16], bool interleaved, const float (&c)[8], const float (&s)[8]) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = v[2 * i], b = v[2 * i + 1];
      v[2 * i] = a * c[i] - b * s[i];
      v[2 * i + 1] = a * s[i] + b * c[i];
      asm volatile("; interleaved pair");
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = v[i], b = v[8 + i];
      v[i] = a * c[i] - b * s[i];
      v[8 + i] = a * s[i] + b * c[i];
      asm volatile("; pair of halves");
    }
  }
}

}  // namespace nvfp4
