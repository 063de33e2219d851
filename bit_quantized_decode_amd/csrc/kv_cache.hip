// The paged key-value cache: writing rows of a QKV product into it, quantised,
// keys (and queries) turned on the way (nvfp4_kv_append), and reading them back
// (nvfp4_kv_read).
//
// One lane takes one block of sixteen values of one token, in each head of its
// share; the blocks of a row sit in neighbouring lanes, so that a row is read in
// one piece and the E4M3 format's row maximum is a few lane exchanges.  A
// wavefront takes the same head of consecutive tokens: its writes then fill the
// layout's 16-token pieces.  Sines and cosines are formed once per lane, for all
// its heads.
//
// Bound by the bytes.  8192 tokens of 8 heads of 128, bf16 in: written as bf16 in
// 15.9 us (67 MB read and written, 4.2 TB/s; 18.0 with ordinary stores, while E4M3
// takes 10.8 with ordinary and 11.0 with non-temporal ones: hence by format), E4M3
// 10.8 (4.7 TB/s), NVFP4 11.4 (3.8 TB/s; 18.6 with a division a value and codes by
// comparison), keys turned on the way 12.2; read back in 15.1, 10.9 and 10.7 us.
#include "attn_launchers.h"
#include "rope_device.h"

namespace nvfp4 {
namespace {

constexpr int kThreads = 256;

constexpr int lanes_per_row(int db) { return db == 1 ? 4 : db == 2 ? 8 : 16; }

// Where a slot lies.
struct Place {
  int64_t group;
  int t;       // token within the group
  bool valid;
};
__device__ __forceinline__ Place place_of(const KvCache& c, int64_t slot, int head) {
  Place p;
  p.valid = slot >= 0 && slot < c.slots;
  const uint32_t tg = p.valid ? (uint32_t)(slot >> 4) : 0u;
  const uint32_t page = tg / (uint32_t)c.gpp;
  p.t = (int)(slot & 15);
  p.group = ((int64_t)page * c.heads + head) * c.gpp + (tg - page * (uint32_t)c.gpp);
  return p;
}

__device__ __forceinline__ float e4m3_of(uint32_t byte) { return __builtin_amdgcn_cvt_f32_fp8((int)byte, 0); }
__device__ __forceinline__ float exp2_of_byte(uint32_t byte) { return __uint_as_float(byte << 23); }

// Sixteen values as codes of the format, and the scale byte.  `amax` holds the
// bits of the largest magnitude: of the row (E4M3) or of the block (NVFP4).  As
// integers, magnitudes keep their order, with NaN above infinity above the rest.
template <int FMT>
__device__ __forceinline__ void encode16(const float (&v)[16], uint32_t amax, float st, uint32_t (&w)[8], uint32_t& scale) {
  const bool finite = amax < 0x7f800000u;
  if constexpr (FMT == kKvBf16) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
    scale = 0;
  } else if constexpr (FMT == kKvE4m3) {
    int e = (int)(amax >> 23) - 127 - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);  // 448 = 1.75 * 2^8
    e = e < kKvE4m3MinExp ? kKvE4m3MinExp : e;
    if (!finite) e = 0;
    const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      int p = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i] * inv, v[4 * i + 1] * inv, 0, false);
      p = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2] * inv, v[4 * i + 3] * inv, p, true);
      w[i] = finite ? (uint32_t)p : 0x7f7f7f7fu;
    }
    // Under the largest exponent the code 0x78 (256) would stand for 2^128: it becomes 0x77 (240), the
    // largest finite value.  (No code is above 0x78 there: adding 8 carries into the sign's bit for 0x78 alone.)
    if (e == kKvE4m3MaxExp) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] -= ((w[i] & 0x7f7f7f7fu) + 0x08080808u) >> 7 & 0x01010101u;
    }
    scale = (uint32_t)(e + kKvE4m3Bias);
  } else {
    const float q = __uint_as_float(amax) / (6.0f * st);
    uint32_t sb = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(fminf(q, 448.0f), 0.0f, 0, false) & 0xffu;
    // Quotients |v| / d rounded as a division rounds them: with the correctly
    // rounded reciprocal r, q0 = a r is within a unit of the quotient, and one
    // step with the exact residual a - q0 d rounds it correctly (Markstein, "Computation
    // of elementary functions on the IBM RISC System/6000 processor", 1990).  Beyond
    // 8 d every code is the largest; the minimum keeps the steps finite.
    const float d = e4m3_of(sb) * st, r = 1.0f / d, most = 8.0f * d;
    uint32_t p[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float q2[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float a = fminf(fabsf(v[2 * i + j]), most), q0 = a * r;
        q2[j] = __builtin_copysignf(__builtin_fmaf(__builtin_fmaf(-q0, d, a), r, q0), v[2 * i + j]);
      }
      // Nearest E2M1, ties to even, +-6 beyond: the conversion's own rounding.
      switch (i % 4) {
        case 0: p[i / 4] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(p[i / 4], q2[0], q2[1], 1.0f, 0); break;
        case 1: p[i / 4] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(p[i / 4], q2[0], q2[1], 1.0f, 1); break;
        case 2: p[i / 4] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(p[i / 4], q2[0], q2[1], 1.0f, 2); break;
        default: p[i / 4] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(p[i / 4], q2[0], q2[1], 1.0f, 3); break;
      }
    }
    const bool some = sb != 0u && finite;
    w[0] = some ? p[0] : 0u;
    w[1] = some ? p[1] : 0u;
    scale = finite ? sb : 0x7fu;
  }
}

// STREAM: a non-temporal store.
template <int BYTES, bool STREAM>
__device__ __forceinline__ void store_bytes(uint8_t* p, const uint32_t* w, int shift) {
  if constexpr (BYTES == 2) *reinterpret_cast<uint16_t*>(p) = (uint16_t)(w[0] >> shift);
  else if constexpr (BYTES == 4) *reinterpret_cast<uint32_t*>(p) = w[0];
  else if constexpr (BYTES == 8) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  else if constexpr (STREAM) __builtin_nontemporal_store(u32x4{w[0], w[1], w[2], w[3]}, reinterpret_cast<u32x4*>(p));
  else *reinterpret_cast<u32x4*>(p) = u32x4{w[0], w[1], w[2], w[3]};
}
template <int BYTES>
__device__ __forceinline__ void load_bytes(const uint8_t* p, uint32_t* w, int shift) {
  if constexpr (BYTES == 2) w[0] |= (uint32_t)*reinterpret_cast<const uint16_t*>(p) << shift;
  else if constexpr (BYTES == 4) w[0] = *reinterpret_cast<const uint32_t*>(p);
  else if constexpr (BYTES == 8) {
    const uint2 a = *reinterpret_cast<const uint2*>(p);
    w[0] = a.x;
    w[1] = a.y;
  } else {
    const u32x4 a = load16(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = a[i];
  }
}

// Moves the codes w of block b of (group, token t) between registers and the
// layout, in pieces that one lane's bytes hold together.
template <int FMT, int DB, bool VSIDE, bool WRITE>
__device__ __forceinline__ void move_codes(uint8_t* codes, int64_t group, int t, int b, uint32_t (&w)[8]) {
  using L = KvLayout<FMT, DB>;
  uint8_t* base = codes + group * L::kCodeBytes + (VSIDE ? L::kSideBytes : 0);
  // Values of one piece: K, the block lies inside one lane; V, a lane holds W
  // consecutive values, and a piece is what of those falls into the block.
  constexpr int kRun = !VSIDE ? 16 : L::kW == 8 ? 8 : L::kW == 16 ? 16 : 4;
  constexpr int kRunBytes = kRun * L::kBits / 8;
  constexpr int kPiece = kRunBytes > 16 ? 16 : kRunBytes;
  constexpr int kPerRun = kRunBytes / kPiece;
#pragma unroll
  for (int n = 0; n < 16 / kRun * kPerRun; ++n) {
    const int i = n / kPerRun, j = n % kPerRun;
    const int d = 16 * b + kRun * i;
    int lane, byte;
    if (!VSIDE) {
      const int h = d / L::kE;
      lane = 16 * h + t;
      byte = (d - h * L::kE) * L::kBits / 8;
    } else {
      const int r = d / L::kW;
      lane = 16 * (t / 4) + r;
      byte = ((t % 4) * L::kW + d - r * L::kW) * L::kBits / 8;
    }
    uint8_t* p = base + L::lane_byte(lane, byte + j * kPiece);
    if (WRITE) store_bytes<kPiece, FMT == kKvBf16>(p, w + n * kPiece / 4, n * kPiece % 4 * 8);
    else load_bytes<kPiece>(p, w + n * kPiece / 4, n * kPiece % 4 * 8);
  }
}

template <int FMT, int DB, bool VSIDE>
__device__ __forceinline__ uint8_t* scale_at(uint8_t* scales, int64_t group, int t, int b) {
  using L = KvLayout<FMT, DB>;
  uint8_t* base = scales + group * L::kScaleBytes + (VSIDE ? L::kKScaleBytes : 0);
  if (FMT == kKvE4m3) return base + t;
  if (VSIDE) return base + ((t / 4) * (4 * DB) + b) * 4 + t % 4;
  const int h = 16 * b / L::kE;
  return base + (16 * h + t) * L::kKScaleLane + (16 * b - h * L::kE) / 16;
}

// ---- writing ----------------------------------------------------------------

template <int FMT, int DB, bool VSIDE>
__device__ __forceinline__ void write_block(const KvCache& c, const Place& p, int b, const float (&v)[16]) {
  constexpr int kLpr = lanes_per_row(DB);
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) amax = max(amax, __float_as_uint(v[i]) & 0x7fffffffu);
  if (FMT == kKvE4m3) {
#pragma unroll
    for (int off = kLpr / 2; off >= 1; off >>= 1) amax = max(amax, (uint32_t)__shfl_xor((int)amax, off));
  }
  if (!p.valid || b >= 4 * DB) return;
  uint32_t w[8], scale;
  encode16<FMT>(v, amax, VSIDE ? c.v_scale : c.k_scale, w, scale);
  move_codes<FMT, DB, VSIDE, true>(c.codes, p.group, p.t, b, w);
  if (FMT == kKvNvfp4 || (FMT == kKvE4m3 && b == 0)) *scale_at<FMT, DB, VSIDE>(c.scales, p.group, p.t, b) = (uint8_t)scale;
}

// blockIdx.x: a run of tokens; blockIdx.y: a chunk of the K, V or query heads.
template <int FMT, int DB, bool BF16>
__global__ __launch_bounds__(kThreads) void append_kernel(const KvAppendLaunch a, int heads_per) {
  constexpr int kLpr = lanes_per_row(DB), kRows = kThreads / kLpr, kStride = 64 * DB + 4;
  __shared__ __attribute__((aligned(16))) float s_row[kRows * kStride];
  const int row = threadIdx.x / kLpr, b = threadIdx.x % kLpr;
  const int64_t tok = (int64_t)blockIdx.x * kRows + row;
  const int kv_chunks = (a.cache.heads + heads_per - 1) / heads_per;
  const int kind = blockIdx.y < kv_chunks ? 0 : blockIdx.y < 2 * kv_chunks ? 1 : 2;
  const int h0 = (blockIdx.y - kind * kv_chunks) * heads_per;
  const int h1 = min(h0 + heads_per, kind == 2 ? a.q_heads : a.cache.heads);
  const int64_t slot = tok < a.tokens ? a.slots[tok] : -1;
  Place p = place_of(a.cache, slot, kind == 2 ? 0 : h0);
  const bool live = p.valid && 16 * b < a.cache.head_dim;
  RopeUnit r{16 * b, 16 * b + 8, false};
  float c[8], s[8];
  if (kind != 1 && a.rope.freqs) {
    r = rope_unit(b, a.rope.rot, a.rope.interleaved);
    if (live && r.turned) rope_angles(a.rope.freqs, b, a.rope.pos[tok], a.rope.magnitude, a.rope.sign, c, s);
  }
  const void* src = kind == 0 ? a.k : kind == 1 ? a.v : a.q;
  int64_t at = tok * (kind == 0 ? a.ldk : kind == 1 ? a.ldv : a.ldq) + (int64_t)h0 * a.cache.head_dim;
  int64_t to = tok * a.ldqo + (int64_t)h0 * a.cache.head_dim;
  for (int h = h0; h < h1; ++h) {
    float v[16];
    if (live) {
      load8<BF16>(src, at + r.first, v);
      load8<BF16>(src, at + r.second, v + 8);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = 0.0f;
    }
    if (r.turned) rope_turn(v, a.rope.interleaved, c, s);
    if (kind == 2) {
      if (live) {
        store8<true>(a.q_out, to + r.first, v);
        store8<true>(a.q_out, to + r.second, v + 8);
      }
      to += a.cache.head_dim;
    } else {
      if (kind == 0 && a.rope.freqs && !a.rope.interleaved) {  // units are not blocks: exchange through LDS
        float* mine = s_row + row * kStride;
        if (b < 4 * DB) {
#pragma unroll
          for (int i = 0; i < 8; i += 4) {
            *reinterpret_cast<f32x4*>(mine + r.first + i) = f32x4{v[i], v[i + 1], v[i + 2], v[i + 3]};
            *reinterpret_cast<f32x4*>(mine + r.second + i) = f32x4{v[8 + i], v[9 + i], v[10 + i], v[11 + i]};
          }
        }
        __syncthreads();
        if (b < 4 * DB) {
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            const f32x4 x = *reinterpret_cast<const f32x4*>(mine + 16 * b + i);
            v[i] = x[0], v[i + 1] = x[1], v[i + 2] = x[2], v[i + 3] = x[3];
          }
        }
        __syncthreads();
      }
      if (kind == 0) write_block<FMT, DB, false>(a.cache, p, b, v);
      else write_block<FMT, DB, true>(a.cache, p, b, v);
      p.group += a.cache.gpp;
    }
    at += a.cache.head_dim;
  }
}

// ---- reading back -----------------------------------------------------------

// Sixteen values from codes and scale byte: exact products, then the tensor scale.
template <int FMT>
__device__ __forceinline__ void decode16(const uint32_t (&w)[8], uint32_t scale, float st, float (&v)[16]) {
  if constexpr (FMT == kKvBf16) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[2 * i] = bf16_lo(w[i]);
      v[2 * i + 1] = bf16_hi(w[i]);
    }
  } else if constexpr (FMT == kKvE4m3) {
    const float s = exp2_of_byte(scale);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[4 * i] = e4m3<0>(w[i]) * s;
      v[4 * i + 1] = e4m3<1>(w[i]) * s;
      v[4 * i + 2] = e4m3<2>(w[i]) * s;
      v[4 * i + 3] = e4m3<3>(w[i]) * s;
    }
  } else {
    const float s = e4m3_of(scale);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const f32x2 p[4] = {e2m1x2<0>(w[i]), e2m1x2<1>(w[i]), e2m1x2<2>(w[i]), e2m1x2<3>(w[i])};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[8 * i + 2 * j] = p[j][0] * s * st;
        v[8 * i + 2 * j + 1] = p[j][1] * s * st;
      }
    }
  }
}

template <int FMT, int DB, bool VSIDE, bool BF16>
__device__ __forceinline__ void read_block(const KvReadLaunch& a, const Place& p, int64_t tok, int head, int b) {
  uint32_t w[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u}, scale = 0;
  move_codes<FMT, DB, VSIDE, false>(a.cache.codes, p.group, p.t, b, w);
  if (FMT != kKvBf16) scale = *scale_at<FMT, DB, VSIDE>(a.cache.scales, p.group, p.t, b);
  float v[16];
  decode16<FMT>(w, scale, VSIDE ? a.cache.v_scale : a.cache.k_scale, v);
  void* dst = VSIDE ? a.v : a.k;
  const int64_t at = tok * (VSIDE ? a.ldv : a.ldk) + (int64_t)head * a.cache.head_dim + 16 * b;
  store8<BF16>(dst, at, v);
  store8<BF16>(dst, at + 8, v + 8);
}

template <int FMT, int DB, bool BF16>
__global__ __launch_bounds__(kThreads) void read_kernel(const KvReadLaunch a) {
  constexpr int kLpr = lanes_per_row(DB), kRows = kThreads / kLpr;
  const int row = threadIdx.x / kLpr, b = threadIdx.x % kLpr;
  const int64_t tok = (int64_t)blockIdx.x * kRows + row;
  const bool vside = blockIdx.y >= a.cache.heads;
  const int head = blockIdx.y - (vside ? a.cache.heads : 0);
  if (tok >= a.tokens || 16 * b >= a.cache.head_dim || !(vside ? a.v : a.k)) return;
  const Place p = place_of(a.cache, a.slots[tok], head);
  if (!p.valid) return;
  if (vside) read_block<FMT, DB, true, BF16>(a, p, tok, head, b);
  else read_block<FMT, DB, false, BF16>(a, p, tok, head, b);
}

// Heads of a workgroup's share: one while the rows do not fill the GPU, more
// where they do (sines and addresses are then shared), four workgroups a CU kept.
template <int FMT, int DB>
void append_launch(const KvAppendLaunch& a, hipStream_t s) {
  constexpr int kRows = kThreads / lanes_per_row(DB);
  const int64_t runs = (a.tokens + kRows - 1) / kRows;
  const int64_t heads = 2 * a.cache.heads + (a.q ? a.q_heads : 0);
  const int64_t per = runs * heads / 1024;
  const int heads_per = (int)(per < 1 ? 1 : per > 8 ? 8 : per);
  const auto chunks = [&](int n) { return (n + heads_per - 1) / heads_per; };
  const dim3 grid((unsigned)runs, (unsigned)(2 * chunks(a.cache.heads) + (a.q ? chunks(a.q_heads) : 0)));
  if (a.bf16) hipLaunchKernelGGL((append_kernel<FMT, DB, true>), grid, dim3(kThreads), 0, s, a, heads_per);
  else hipLaunchKernelGGL((append_kernel<FMT, DB, false>), grid, dim3(kThreads), 0, s, a, heads_per);
}

template <int FMT, int DB>
void read_launch(const KvReadLaunch& a, hipStream_t s) {
  constexpr int kRows = kThreads / lanes_per_row(DB);
  const dim3 grid((unsigned)((a.tokens + kRows - 1) / kRows), (unsigned)(2 * a.cache.heads));
  if (a.bf16) hipLaunchKernelGGL((read_kernel<FMT, DB, true>), grid, dim3(kThreads), 0, s, a);
  else hipLaunchKernelGGL((read_kernel<FMT, DB, false>), grid, dim3(kThreads), 0, s, a);
}

// Calls fn<FMT, DB>(a, s) for the cache's format and head size.
#define NVFP4_KV_DISPATCH_DB(fn, FMT)                        \
  switch ((a.cache.head_dim + 63) / 64) {                    \
    case 1: fn<FMT, 1>(a, s); break;                         \
    case 2: fn<FMT, 2>(a, s); break;                         \
    case 3: fn<FMT, 3>(a, s); break;                         \
    default: fn<FMT, 4>(a, s); break;                        \
  }
#define NVFP4_KV_DISPATCH(fn)                                \
  switch (a.format) {                                        \
    case kKvBf16: NVFP4_KV_DISPATCH_DB(fn, kKvBf16) break;   \
    case kKvE4m3: NVFP4_KV_DISPATCH_DB(fn, kKvE4m3) break;   \
    default: NVFP4_KV_DISPATCH_DB(fn, kKvNvfp4) break;       \
  }

}  // namespace

hipError_t launch_kv_append(const KvAppendLaunch& a, hipStream_t s) {
  NVFP4_KV_DISPATCH(append_launch)
  return hipGetLastError();
}

hipError_t launch_kv_read(const KvReadLaunch& a, hipStream_t s) {
  NVFP4_KV_DISPATCH(read_launch)
  return hipGetLastError();
}

}  // namespace nvfp4
