// Rotary positions (nvfp4_rope): every head of a row turned, pair i by
// pos * f_i turns, in fp32 with one rounding at the end.
//
// One thread takes one unit (rope_device.h: eight pairs, or sixteen values past
// the rotated part) of one token: it forms the eight sines and cosines once and
// turns that unit in every head of its share.  Bound by the bytes: 4096 tokens of
// 48 heads of 128, bf16, in 20.2 us (5.0 TB/s read and written, a large copy's
// rate; 23.8 us without non-temporal loads, 25.9 us with one head a thread besides,
// whose sines are then formed 48 times over).
#include "attn_launchers.h"
#include "rope_device.h"

namespace nvfp4 {
namespace {

constexpr int kThreads = 256;

template <bool XBF, bool YBF>
__global__ __launch_bounds__(kThreads) void rope_kernel(const RopeLaunch a, int heads_per) {
  const int units = a.head_dim / 16;
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t t = i / units;
  if (t >= a.tokens) return;
  const int u = (int)(i - t * units);
  const RopeUnit r = rope_unit(u, a.rope.rot, a.rope.interleaved);
  float c[8], s[8];
  if (r.turned) rope_angles(a.rope.freqs, u, a.rope.pos[t], a.rope.magnitude, a.rope.sign, c, s);
  const int h0 = blockIdx.y * heads_per, h1 = min(h0 + heads_per, a.heads);
  for (int h = h0; h < h1; ++h) {
    const int64_t x = t * a.ldx + (int64_t)h * a.head_dim, y = t * a.ldy + (int64_t)h * a.head_dim;
    float v[16];
    load8<XBF, true>(a.x, x + r.first, v);
    load8<XBF, true>(a.x, x + r.second, v + 8);
    if (r.turned) rope_turn(v, a.rope.interleaved, c, s);
    store8<YBF>(a.y, y + r.first, v);
    store8<YBF>(a.y, y + r.second, v + 8);
  }
}

}  // namespace

hipError_t launch_rope(const RopeLaunch& a, hipStream_t s) {
  const int64_t threads = a.tokens * (a.head_dim / 16);
  const int64_t wgs = (threads + kThreads - 1) / kThreads;
  // Heads of a thread: one while the threads do not fill the GPU, more where
  // they do, four workgroups a CU kept.
  const int64_t per = wgs * a.heads / 1024;
  const int heads_per = (int)(per < 1 ? 1 : per > 8 ? 8 : per);
  const dim3 grid((unsigned)wgs, (unsigned)((a.heads + heads_per - 1) / heads_per));
  if (a.x_bf16 && a.y_bf16) hipLaunchKernelGGL((rope_kernel<true, true>), grid, dim3(kThreads), 0, s, a, heads_per);
  else if (a.x_bf16) hipLaunchKernelGGL((rope_kernel<true, false>), grid, dim3(kThreads), 0, s, a, heads_per);
  else if (a.y_bf16) hipLaunchKernelGGL((rope_kernel<false, true>), grid, dim3(kThreads), 0, s, a, heads_per);
  else hipLaunchKernelGGL((rope_kernel<false, false>), grid, dim3(kThreads), 0, s, a, heads_per);
  return hipGetLastError();
}

}  // namespace nvfp4
