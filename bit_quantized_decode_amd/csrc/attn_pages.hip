// Attention of one new token per sequence over pages chosen for each kv head (nvfp4_attn_decode_heads), and
// attention that adds up the weight that each page has had (nvfp4_attn_weigh).
//
// Both are attn_kernel (attn_kernel.h).  The first looks its pages up in a table of its own for each kv head.
// The second keeps the sum m of the terms of every sixteen tokens, a byproduct of the pass over the cache, with the
// reference s that they were formed under, since that may still move.  A second launch, when the rows' references R and
// sums l are final, turns the sums of a page into its weight:
//   weight_i = sum over the group's rows r and the page's sixteens t of m_rt 2^(s_rt - R_r) / l_r.
// Both references are log2 of one scale, and s <= R: the exponent is a difference of numbers as they are, so that a row's
// shares add up to 1 however large its scores.  (As one number, log2 m + s, against lse they were off by half steps of lse: 1e-4
// at 1000, up to a factor of 2 at 2^20.)  Sums of sixteen tokens are 8 bytes a row, for 16 * 2 * head_dim values of the cache;
// the second launch finds them in the L2 and the last-level cache.
//
// Bound as attn_kernel is; what weighing adds is its 5 us and up to 5 us of the pass, for which it writes 8 bytes a row and sixteen
// tokens: 32 users of up to 8192 NVFP4 tokens 43 us for both launches (152 MB, 3.5 TB/s), the attention alone 35; one of 65,536 E4M3
// tokens 34 us (135 MB, 4.0 TB/s), the attention alone 29.
#include "attn_kernel.h"

namespace nvfp4 {
namespace {

struct WeighParams {
  AttnParams attn;
  const Mass* mass;
  const Mass* rows;
  const float* weights;
  float* weights_out;
  int64_t groups;
  float decay;
};

// LANES lanes take one page of one kv head.
template <int LANES>
__global__ __launch_bounds__(256) void weigh_kernel(const WeighParams w) {
  const AttnParams& a = w.attn;
  const int64_t item = (workgroup() * 256 + threadIdx.x) / LANES;
  const int lane = threadIdx.x % LANES;
  const int64_t unit = item / a.table_width;                 // (sequence, kv head)
  if (unit >= (int64_t)a.batch * a.cache.heads) return;
  const int b = (int)(unit / a.cache.heads), head = (int)(unit - (int64_t)b * a.cache.heads);
  const int page = (int)(item - unit * a.table_width);
  const float before = lane == 0 && w.decay != 0.0f ? w.weights[item] : 0.0f;  // (on its way while the sums are)
  const Span sp = span_of(a, a.lens[b]);
  // The page's tokens inside the span (offsets up to 2^30), as sixteens from the span's base on.
  const int from = max(page * a.cache.page_size, sp.begin), to = min((page + 1) * a.cache.page_size, sp.end);
  float sum = 0.0f;
  if (from < to) {
    const int first = (from - sp.base) / kKvGroup, n = (to - 1 - sp.base) / kKvGroup + 1 - first;
    for (int rt = 0; rt < a.row_tiles; ++rt) {
      const Mass* mass = w.mass + ((unit * a.row_tiles + rt) * w.groups + first) * a.part_rows;
      const int rows = min(a.group - rt * kRows, kRows);
      const Mass* row = w.rows + (int64_t)b * a.q_heads + head * a.group + rt * kRows;
      // Both loads at once, four of each a trip.  A sum of 0 is one of no terms, or of a row that has none, but under a reference of
      // infinity, whose row is NaN.
      for (int e0 = lane; e0 < n * a.part_rows; e0 += 4 * LANES) {
        Mass m[4], l[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e = e0 + i * LANES, r = e % a.part_rows;
          const bool in = e < n * a.part_rows && r < rows;
          m[i] = in ? mass[e] : Mass{0.0f, 0.0f};
          l[i] = row[in ? r : 0];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float share = m[i].sum * __builtin_amdgcn_exp2f(m[i].ref - l[i].ref) / l[i].sum;
          sum += m[i].sum == 0.0f && m[i].ref <= kFltMax ? 0.0f : share;   // NaN stays NaN
        }
      }
    }
  }
#pragma unroll
  for (int off = LANES / 2; off >= 1; off >>= 1) sum += __shfl_xor(sum, off);
  if (lane == 0) w.weights_out[item] = w.decay == 0.0f ? sum : w.decay * before + sum;
}

int64_t mass_groups_of(const AttnLaunch& a) {
  const int64_t most = a.table_width * a.cache.gpp;
  return a.window > 0 && a.window / kKvGroup + 2 < most ? a.window / kKvGroup + 2 : most;
}

size_t rounded(size_t bytes) { return (bytes + 255) & ~(size_t)255; }

size_t mass_bytes(const AttnLaunch& a) {
  return rounded((size_t)(a.batch * a.cache.heads * row_tiles_of(a)) * (size_t)mass_groups_of(a) * part_rows_of(a) * sizeof(Mass));
}

}  // namespace

hipError_t launch_attn_heads(const AttnLaunch& a, hipStream_t s) {
  ModeParams<kHeads> p;
  fill_params(a, p);
  return attn_launch(a, p, s);
}

size_t attn_weigh_workspace_bytes(const AttnWeighLaunch& a) {
  return rounded(attn_workspace_bytes(a.attn)) + mass_bytes(a.attn) + (size_t)a.attn.batch * a.attn.q_heads * sizeof(Mass);
}

hipError_t launch_attn_weigh(const AttnWeighLaunch& a, hipStream_t s) {
  ModeParams<kWeigh> p;
  fill_params(a.attn, p);
  uint8_t* mass = static_cast<uint8_t*>(a.attn.ws) + rounded(attn_workspace_bytes(a.attn));
  p.mass = reinterpret_cast<Mass*>(mass);
  p.rows = reinterpret_cast<Mass*>(mass + mass_bytes(a.attn));
  p.groups = mass_groups_of(a.attn);
  const hipError_t e = attn_launch(a.attn, p, s);
  if (e != hipSuccess || a.attn.table_width == 0) return e;
  WeighParams w;
  w.attn = p;
  w.mass = p.mass;
  w.rows = p.rows;
  w.weights = a.weights;
  w.weights_out = a.weights_out;
  w.groups = p.groups;
  w.decay = a.decay;
  // Lanes a page: sixteen where they find fewer than eight sums each, a wavefront from there on.  (Both launches, sixteen lanes
  // against a wavefront.  One user of 131,072 NVFP4 tokens, five rows a kv head: pages of 16 45 us against 64, of 64 40 against 45, of
  // 512 42 against 41, of 1024 41.4 against 39.1; sixteen rows: of 256 47 against 46, of 1024 54.6 against 45.8, of 4096 86 against
  // 53.  32 users of 4096, sixteen rows: of 64 37.7 against 42.2, of 128 37.6 against 38.6, of 256 38.5 against 37.7.)
  const int64_t pages = a.attn.batch * a.attn.cache.heads * a.attn.table_width;
  if (a.attn.cache.gpp * p.part_rows < 128)
    hipLaunchKernelGGL((weigh_kernel<16>), grid_of((pages + 15) / 16), dim3(256), 0, s, w);
  else
    hipLaunchKernelGGL((weigh_kernel<64>), grid_of((pages + 3) / 4), dim3(256), 0, s, w);
  return hipGetLastError();
}

}  // namespace nvfp4
