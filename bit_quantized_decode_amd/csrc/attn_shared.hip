// Attention of one new token per sequence where all sequences share a long prefix (nvfp4_attn_shared).
//
// Softmax sums over the prefix and over a sequence's own tokens join as any two stretches of one row do:
// with references r, r' and sums l, l' of terms 2^(s - r), the joined sums are those of the larger
// reference, the other's times 2^(r' - r).  So the prefix is one problem of its own: for each kv head, the
// queries of all sequences and of its group are the rows of a matrix, and its keys and values are read once for
// all of them (where that saves more than two launches cost, see apart()).  One launch leaves the prefix's partial sums, attn_kernel those of the own tokens, and a third
// joins them row by row.
//
// Bound by the vector units, which dequantise and exponentiate: 32 users of 40 heads under 32,768 NVFP4 tokens
// 55 us, of which 45 for the prefix (21.6 Gflop; 48 MB), 9 for up to 512 tokens of each user and 5 for the join; 200 under 8192
// bf16 tokens 79 us, 64 for the prefix (33.8 Gflop), 17 and 7.  Few rows are bound by the bytes: 7 users of 256-wide heads
// under 50,001 E4M3 tokens 41 us, 24 for the prefix (105 MB, 4.4 TB/s).
// (Two tiles in flight a wavefront instead of one gained nothing: 54.4 us against 55.1, 64-wide E4M3 heads 42.5 against 40.8.)
//
// The tiles and operands are those of attn_kernel.h.  Here a wavefront holds RT tiles of sixteen rows: one
// 32-token tile of the cache is read, and dequantised, once for 16 RT rows.  The wavefronts of a
// workgroup take the tiles of its share in turn and join through LDS at its end.
//
// (RT = 4 on one wavefront a SIMD: 32 users under 32,768 NVFP4 tokens 85 us against 66 with two of RT = 2, since then nothing
// runs while a wavefront waits.  Eight wavefronts that bring a tile's operands into LDS for 128 rows: long prefixes
// of 1000 bf16 rows run at 1.06 PFLOP/s of matrix instructions against 0.74, but the larger blocks' partial sums and the joins
// cost 10 us more: 77 us against 79 for 8192 tokens, 67 against 51 for the 32 users.)
#include <algorithm>

#include "attn_kernel.h"

namespace nvfp4 {
namespace {

// The shared prefix's partial sums.  Its units are (kv head, block of rows), a kv head's rows those of
// all sequences, (sequence, query head of the group) in order.  Each unit's tiles are cut evenly over `each` workgroups
// if that occupies nearly all CUs; else the line of all units' tiles is cut evenly over `grid` workgroups, of which some
// then hold the end of one unit and the beginning of another.  Less is cut where there is little to do.
// (Units of their own: 32 users of 40 heads under 32,768 NVFP4 tokens, 40 units, 58 us against 64.  That leave
// CUs idle: 70 users of 64 heads under 10,000, 144 units of one workgroup, 81 us against 65 along the line.)
struct Prefix {
  const int32_t* len;
  const int32_t* table;
  float* part;         // [piece][block_rows][DP + 4]: reference, sum, two unused, the padded head's sums
  int32_t most;        // tokens that the table holds
  int32_t units, row_blocks, block_rows, grid, each;
  int32_t share;       // tiles of a workgroup's share, at least: one a wavefront
};
__device__ __forceinline__ int prefix_len(const Prefix& p) {
  const int len = *p.len;
  return len < 0 ? 0 : len > p.most ? p.most : len;
}
// Workgroup w's share [begin, end) of the line, and the number of its first piece; that of the piece after
// a unit's end is one more.
struct Share {
  int begin, end, piece;
};
__device__ __forceinline__ Cut prefix_cut(const Prefix& p, int tiles) {
  if (p.each > 0) return cut_of(tiles, min(p.each, (tiles + p.share - 1) / p.share));
  const int line = p.units * tiles;
  return cut_of(line, min(p.grid, (line + p.share - 1) / p.share));
}
__device__ __forceinline__ int prefix_workgroups(const Prefix& p, const Cut& c) { return p.each > 0 ? p.units * c.n : c.n; }
__device__ __forceinline__ Share prefix_share(const Prefix& p, const Cut& c, int tiles, int w) {
  if (p.each > 0) {
    const int unit = (int)((unsigned)w / (unsigned)c.n), i = w - unit * c.n;
    return Share{unit * tiles + run_start(c, i), unit * tiles + run_start(c, i + 1), w};
  }
  // (Along the line each piece has one more workgroup or one more unit behind it.)
  const int begin = run_start(c, w);
  return Share{begin, run_start(c, w + 1), (int)((unsigned)begin / (unsigned)tiles) + w};
}
// A unit's pieces.
struct Pieces {
  int first, n;
};
__device__ __forceinline__ Pieces prefix_pieces(const Prefix& p, const Cut& c, int tiles, int unit) {
  if (p.each > 0) return Pieces{unit * c.n, c.n};
  const int w0 = run_of(c, unit * tiles);
  return Pieces{unit + w0, run_of(c, unit * tiles + tiles - 1) + 1 - w0};
}

struct PrefixParams {
  KvCache cache;
  const uint16_t* q;
  int64_t ldq;
  Prefix prefix;
  int32_t rows;        // of a kv head: batch * group
  int32_t group;
  float score_factor;
  int score_exp;
};

// Values d0 .. d0 + E - 1 of the queries of a kv head's row; rows and values that are not there: zeros, from
// addresses inside.
template <int E>
__device__ __forceinline__ void load_queries(const PrefixParams& a, int head, int row, int d0, uint32_t (&qv)[E / 2]) {
  const int d_here = a.cache.head_dim - d0;
  const bool in = row < a.rows && d_here > 0;
  const int b = in ? row / a.group : 0, qh = head * a.group + (in ? row - b * a.group : 0);
  const uint16_t* qp = a.q + (int64_t)b * a.ldq + qh * a.cache.head_dim + (in ? d0 : 0);
  const int last = in ? d_here - 8 : 0;
#pragma unroll
  for (int i = 0; i < E / 8; ++i) {
    const u32x4 x = load16(qp + min(8 * i, last));
#pragma unroll
    for (int j = 0; j < 4; ++j) qv[4 * i + j] = in && 8 * i <= last ? x[j] : 0u;
  }
}

// Wavefronts a SIMD.  (Two row tiles of heads beyond 128 have registers, and room for their sums in LDS, for one.)
constexpr int prefix_waves(int fmt, int db, int rt) { return rt == 1 ? waves_per_simd(fmt, db) : db <= 2 ? 2 : 1; }

// Neighbouring shares on one XCD, whose L2 then serves a kv head's other blocks of rows.
__device__ __forceinline__ int xcd_order(int wg, int n) {
  const int xcd = wg & 7;
  return xcd * (n >> 3) + min(xcd, n & 7) + (wg >> 3);
}

template <int FMT, int DB, int RT>
__global__ __launch_bounds__(256 * prefix_waves(FMT, DB, RT), (prefix_waves(FMT, DB, RT))) void prefix_kernel(const PrefixParams a) {
  using L = KvLayout<FMT, DB>;
  // Two row tiles: other blocks of rows read the same.  (200 users under 8192 bf16 tokens 80 us against 91.)
  constexpr int kPolicy = RT == 1 ? kStreamed : kCached;
  constexpr int kWaves = 4 * prefix_waves(FMT, DB, RT), kThreads = 64 * kWaves, kBlock = kRows * RT;
  constexpr int kDp = 64 * DB, kE = L::kE, kW = L::kW, kSteps = kE / 8, kQuads = kE / 4;
  struct Sums {
    float ml[kWaves][kBlock][2];
    float o[kWaves][kBlock][kDp + 4] __attribute__((aligned(16)));
  };
  __shared__ Sums lds;

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int qn = lane & 15, h = lane >> 4, d0 = kE * h;
  const int len = prefix_len(a.prefix), tiles = (len + kTile - 1) / kTile;
  if (tiles == 0) return;
  const Cut shares = prefix_cut(a.prefix, tiles);
  const int workgroups = prefix_workgroups(a.prefix, shares);
  if ((int)blockIdx.x >= workgroups) return;
  Share share = prefix_share(a.prefix, shares, tiles, xcd_order(blockIdx.x, workgroups));

  for (int s = share.begin; s < share.end; ++share.piece) {
    const int unit = (int)((unsigned)s / (unsigned)tiles), t0 = s - unit * tiles, t1 = min(tiles, t0 + share.end - s);
    const int head = unit / a.prefix.row_blocks, row0 = (unit - head * a.prefix.row_blocks) * kBlock;
    const int count = max((t1 - t0 - wave + kWaves - 1) / kWaves, 0);

    uint32_t qv[RT][kE / 2];
    float score_scale[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      load_queries<kE>(a, head, row0 + kRows * rt + qn, d0, qv[rt]);
      score_scale[rt] = query_scale<FMT>(qv[rt], a.score_factor, a.score_exp);
    }

    // Page lookups, as in attn_kernel, of this wavefront's tiles.
    int looked_up = -1;
    const auto look_up = [&](int it, int (&group)[2]) {
      if ((it & 31) == 0) {
        const int tok = (t0 + wave + kWaves * (it + (lane >> 1))) * kTile + (lane & 1) * kKvGroup;
        looked_up = -1;
        if (it + (lane >> 1) < count && tok < len) {
          const int tg = tok / kKvGroup, pg = tg / a.cache.gpp;
          const int page = a.prefix.table[pg];
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

    f32x4 o[RT][kW];
    float ref[RT], sum[RT], shift[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
      for (int i = 0; i < kW; ++i) o[rt][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      ref[rt] = kNegInf;
      sum[rt] = shift[rt] = 0.0f;
    }
    Tile<FMT, DB> t;
    int group[2];
    look_up(0, group);
    to_load(group);
    load_k<FMT, DB, kPolicy>(from, lane, t);
    __builtin_amdgcn_sched_barrier(0);
    load_v<FMT, DB, kPolicy>(from, lane, t);
    __builtin_amdgcn_sched_barrier(0);

    for (int it = 0; it < count; ++it) {
      const int tok0 = (t0 + wave + kWaves * it) * kTile;
      const bool has0 = group[0] >= 0, has1 = group[1] >= 0;
      const bool whole = has0 && has1 && tok0 + kTile <= len;
      if (it + 1 < count) look_up(it + 1, group);
      else group[0] = group[1] = -1;
      to_load(group);
      uint32_t okbits = 0xffu;
      if (!whole) {
        okbits = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int tok = tok0 + (i / 4) * kKvGroup + 4 * h + i % 4;
          okbits |= ((i / 4 ? has1 : has0) && tok < len) ? 1u << i : 0u;
        }
      }

      float x[RT][8];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        f32x4 acc[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) acc[rt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          uint32_t op[4];
          k_operand<FMT, DB>(t, half, k, op);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) acc[rt] = mma<FMT>(op, &qv[rt][4 * k], acc[rt]);
        }
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
          for (int i = 0; i < 4; ++i) x[rt][4 * half + i] = rounded_product(acc[rt][i], score_scale[rt]);
      }
      load_k<FMT, DB, kPolicy>(from, lane, t);

      if (!whole) {
        asm volatile("" : "+v"(okbits));   // (here, or the compiler tests the bits of whole tiles too)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
          for (int i = 0; i < 8; ++i) x[rt][i] = (okbits >> i) & 1u ? x[rt][i] : kNegInf;
      }
      // One branch for all row tiles: between it and the next step everything is one stretch of independent chains.
      float top[RT];
      bool move = false;
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        top[rt] = x[rt][0];
#pragma unroll
        for (int i = 1; i < 8; ++i) top[rt] = fmaxf(top[rt], x[rt][i]);
        move |= top[rt] - ref[rt] > Softmax<FMT>::kOffset + Softmax<FMT>::kSlack;
      }
      if (__any(move)) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          const float alpha = move_reference<FMT>(top[rt], ref[rt]);
          shift[rt] = ref[rt] == kNegInf ? 0.0f : ref[rt];
          sum[rt] *= alpha;
#pragma unroll
          for (int i = 0; i < kW; ++i) o[rt][i] *= alpha;
        }
      }
      uint32_t hi[RT][4], lo[RT][4];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        float p[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          p[i] = __builtin_amdgcn_exp2f(x[rt][i] - shift[rt]);
          sum[rt] += p[i];
        }
        split_terms<FMT>(p, hi[rt], lo[rt]);
      }

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
      load_v<FMT, DB, kPolicy>(from, lane, t);
#pragma unroll
      for (int j = 0; j < kW; ++j)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          o[rt][j] = mma<FMT>(op[j], hi[rt], o[rt][j]);
          if constexpr (FMT != kKvNvfp4) o[rt][j] = mma<FMT>(op[j], lo[rt], o[rt][j]);
        }
    }

    // The wavefronts' sums, joined by all threads into the piece.
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int r = kRows * rt + qn;
      sum[rt] += lane_xor(sum[rt], 16);
      sum[rt] += lane_xor(sum[rt], 32);
      if (h == 0) {
        lds.ml[wave][r][0] = ref[rt];
        lds.ml[wave][r][1] = sum[rt];
      }
      // o[rt][j][i] is d = W (4h + i) + j of row q.
#pragma unroll
      for (int u = 0; u < kQuads; ++u) {
        const int i = 4 * u / kW, j = 4 * u % kW;
        *reinterpret_cast<f32x4*>(&lds.o[wave][r][d0 + 4 * u]) = f32x4{o[rt][j][i], o[rt][j + 1][i], o[rt][j + 2][i], o[rt][j + 3][i]};
      }
    }
    __syncthreads();
    float* piece = a.prefix.part + (int64_t)share.piece * kBlock * (kDp + 4);
    const int rows = min(a.rows - row0, kBlock);
    for (int e = tid; e < rows * (kDp / 4); e += kThreads) {
      const int r = e / (kDp / 4), d = 4 * (e - r * (kDp / 4));
      float top = lds.ml[0][r][0], l = 0.0f;
#pragma unroll
      for (int i = 1; i < kWaves; ++i) top = fmaxf(top, lds.ml[i][r][0]);
      f32x4 acc{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < kWaves; ++i) {
        const float m = lds.ml[i][r][0];
        const float f = m == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(m - top);
        l += lds.ml[i][r][1] * f;
        acc += *reinterpret_cast<const f32x4*>(&lds.o[i][r][d]) * f;
      }
      if (d == 0) *reinterpret_cast<f32x4*>(piece + r * (kDp + 4)) = f32x4{top, l, 0.0f, 0.0f};
      *reinterpret_cast<f32x4*>(piece + r * (kDp + 4) + 4 + d) = acc;
    }
    __syncthreads();
    s += t1 - t0;
  }
}

struct JoinParams {
  Prefix prefix;
  const float* raw;        // of the own tokens
  const int32_t* lens;
  uint16_t* out;
  float* lse;
  int64_t ldo;
  int32_t batch, q_heads, group, head_dim;
  float v_scale;
};

// Each row by THREADS threads: its quads of values times as many runs of its pieces.  A run's pieces are read kPieces at a
// time and added in order, the runs after one another.  (A workgroup reads 64 pieces or so at once: 7 users of 256-wide heads under
// 50,001 E4M3 tokens 40.4 us against 42.6 with sixteen of them, 41.2 with 32.)
template <int DP, int THREADS>
__global__ __launch_bounds__(256) void join_kernel(const JoinParams a) {
  constexpr int kQuads = DP / 4, kRuns = THREADS / kQuads, kPieces = THREADS == 256 ? DP / 16 : 4, kRowsHere = 256 / THREADS;
  __shared__ float s_ml[kRowsHere][kRuns][2];
  __shared__ f32x4 s_o[kRowsHere][kRuns][kQuads];
  const int t = threadIdx.x % THREADS, at = threadIdx.x / THREADS, run = t / kQuads, d = 4 * (t - run * kQuads);
  const int64_t row = workgroup() * kRowsHere + at;
  const bool live = row < (int64_t)a.batch * a.q_heads && run < kRuns;
  const int b = live ? (int)(row / a.q_heads) : 0, qh = live ? (int)(row - (int64_t)b * a.q_heads) : 0;
  const int tiles = (prefix_len(a.prefix) + kTile - 1) / kTile;
  float top = kNegInf, l = 0.0f;
  f32x4 acc{0.0f, 0.0f, 0.0f, 0.0f};
  if (live && tiles > 0 && a.lens[b] >= 0) {       // below 0: a free place of the batch
    const int head = qh / a.group, r = b * a.group + qh - head * a.group;
    const int block = r / a.prefix.block_rows, unit = head * a.prefix.row_blocks + block;
    const Cut c = prefix_cut(a.prefix, tiles);
    const Pieces all = prefix_pieces(a.prefix, c, tiles, unit);
    const int n = all.n;
    const int i1 = n * (run + 1) / kRuns;
    const float* from = a.prefix.part + ((int64_t)all.first * a.prefix.block_rows + (r - block * a.prefix.block_rows)) * (DP + 4);
    const int64_t stride = (int64_t)a.prefix.block_rows * (DP + 4);
    for (int i = n * run / kRuns; i < i1; i += kPieces) {
      f32x4 ml[kPieces], v[kPieces];
#pragma unroll
      for (int j = 0; j < kPieces; ++j) {
        const float* p = from + min(i + j, i1 - 1) * stride;
        ml[j] = *reinterpret_cast<const f32x4*>(p);
        v[j] = *reinterpret_cast<const f32x4*>(p + 4 + d);
      }
#pragma unroll
      for (int j = 0; j < kPieces; ++j)
        if (i + j < i1) add_part(top, l, acc, ml[j][0], ml[j][1], v[j]);
    }
  }
  if (live && run == 0) {
    const float* own = a.raw + row * (DP + 4);
    add_part(top, l, acc, own[0], own[1], *reinterpret_cast<const f32x4*>(own + 4 + d));
  }
  if (kRuns > 1) {
    if (live) {
      if (d == 0) {
        s_ml[at][run][0] = top;
        s_ml[at][run][1] = l;
      }
      s_o[at][run][d / 4] = acc;
    }
    __syncthreads();
    if (live && run == 0) {
#pragma unroll
      for (int i = 1; i < kRuns; ++i) add_part(top, l, acc, s_ml[at][i][0], s_ml[at][i][1], s_o[at][i][d / 4]);
    }
  }
  if (!live || run > 0) return;
  const bool some = l > 0.0f || l != l;  // NaN stays NaN
  const float f = some ? a.v_scale / l : 0.0f;
  if (d < a.head_dim) {
    uint16_t* to = a.out + (int64_t)b * a.ldo + (int64_t)qh * a.head_dim + d;
    *reinterpret_cast<uint2*>(to) = make_uint2(pack_bf16x2(acc[0] * f, acc[1] * f), pack_bf16x2(acc[2] * f, acc[3] * f));
  }
  if (d == 0 && a.lse) a.lse[row] = some ? (top + __builtin_amdgcn_logf(l)) * kLn2 : kNegInf;
}

template <int DP>
void join_launch(const JoinParams& p, hipStream_t s) {
  // A wavefront a row where its pieces are few, a workgroup where there are more than it reads at once.  (200 users of 40 heads
  // under 8192 bf16 tokens, a piece or two a row: 83 us against 92, 64-wide 56 against 63; 16 users of 8 heads under 32,768, 32 pieces: 45 us
  // against 40; 7 users of 256-wide heads under 50,001 E4M3 tokens, 64 pieces: 58 against 40.)
  const int64_t rows = (int64_t)p.batch * p.q_heads, pieces = p.prefix.grid / p.prefix.units + 1;
  if (pieces <= 8 * (256 / DP)) hipLaunchKernelGGL((join_kernel<DP, 64>), grid_of((rows + 3) / 4), dim3(256), 0, s, p);
  else hipLaunchKernelGGL((join_kernel<DP, 256>), grid_of(rows), dim3(256), 0, s, p);
}

int head_rows_of(const AttnSharedLaunch& a) { return (int)(a.attn.batch * (a.attn.q_heads / a.attn.cache.heads)); }

int padded_of(const AttnSharedLaunch& a) { return (a.attn.cache.head_dim + 63) / 64; }

// Row tiles of a workgroup: one if that takes all rows, else two.  (Eight rows under 32,768 NVFP4 tokens 22.1 us against 24.4 with
// an empty second tile.)
int block_tiles_of(const AttnSharedLaunch& a) { return head_rows_of(a) <= kRows ? 1 : 2; }

int64_t prefix_units_of(const AttnSharedLaunch& a) {
  const int block = kRows * block_tiles_of(a);
  return (int64_t)a.attn.cache.heads * ((head_rows_of(a) + block - 1) / block);
}

int64_t prefix_tiles_of(const AttnSharedLaunch& a) { return (a.prefix_width * a.attn.cache.page_size + kTile - 1) / kTile; }

int prefix_share_of(const AttnSharedLaunch& a) {
  return 4 * prefix_waves(a.attn.format, padded_of(a), block_tiles_of(a));
}

// Workgroups a unit (0: the line is cut), see Prefix.
int prefix_each_of(const AttnSharedLaunch& a) {
  const int64_t units = prefix_units_of(a), each = units <= kCus ? kCus / units : 0;
  return 8 * each * units >= 7 * kCus ? (int)each : 0;
}

// Workgroups of the launch: as many as the longest prefix has work for.
int prefix_grid_of(const AttnSharedLaunch& a) {
  const int64_t units = prefix_units_of(a), tiles = prefix_tiles_of(a), each = prefix_each_of(a);
  const int64_t share = prefix_share_of(a);
  const auto shares = [&](int64_t n) { return (n + share - 1) / share; };
  const int64_t n = each > 0 ? units * std::min(each, shares(tiles)) : shares(units * tiles);
  return (int)std::min<int64_t>(n, kCus);
}

AttnLaunch behind_of(const AttnSharedLaunch& a) {
  AttnLaunch l = a.attn;
  l.table_width += a.prefix_width;
  return l;
}
// Whether each sequence reads the prefix by itself (kBehind), in one launch instead of three: where a prefix that fills its table
// is so few bytes, most of which come from caches, or nothing would be shared.  The host knows the table's size and not the
// prefix's, so that a short prefix in a large table takes three launches.
// (One against three, 40 heads.  NVFP4, 32 users: under 500 tokens 9.7 us against 19.1, 2000 (66 MB) 17.3 against 22.0, 3000 (98 MB)
// 21.8 against 23.0, 4000 (131 MB) 25.9 against 23.8.  The limit is where these cross.  The wider formats cross later: E4M3, 32 users,
// 2000 tokens (131 MB) 17.2 against 21.2, 3000 21.6 against 22.0, 4000 25.5 against 23.5; bf16, 16 users, 2000 (131 MB) 18.1 against
// 20.1, 4000 (262 MB) 21.5 against 22.5, 6000 28.8 against 23.6, 32 users 1000 (131 MB) 12.0 against 19.4, 2000 (262 MB) 15.9
// against 21.3.  One user of 16 heads under 30,000 E4M3 tokens 17.4 against 22.0.)
constexpr int64_t kApartBytes = int64_t(96) << 20;
bool apart(const AttnSharedLaunch& a) {
  const int64_t row_tiles = row_tiles_of(a.attn), block = kRows * block_tiles_of(a);
  const int64_t bytes = a.attn.batch * row_tiles * a.prefix_width * a.attn.cache.gpp * a.attn.cache.heads *
                        (int64_t)kv_code_bytes(a.attn.format, padded_of(a));
  const bool alone = a.attn.batch * row_tiles <= (head_rows_of(a) + block - 1) / block;
  return (alone || bytes <= kApartBytes) && attn_fits(behind_of(a)) &&
         behind_of(a).table_width * a.attn.cache.page_size <= int64_t(1) << 30;
}

size_t rounded(size_t bytes) { return (bytes + 255) & ~(size_t)255; }

size_t row_bytes(const AttnSharedLaunch& a) { return (64 * padded_of(a) + 4) * sizeof(float); }

// The workspace: attn_kernel's, the own tokens' sums, the prefix's pieces.
size_t raw_at(const AttnSharedLaunch& a) { return rounded(attn_workspace_bytes(a.attn)); }
size_t pieces_at(const AttnSharedLaunch& a) { return raw_at(a) + rounded((size_t)(a.attn.batch * a.attn.q_heads) * row_bytes(a)); }

template <int FMT, int DB>
void prefix_launch(const AttnSharedLaunch& a, const PrefixParams& p, hipStream_t s) {
  const dim3 grid((unsigned)p.prefix.grid);
  if (p.prefix.block_rows == kRows) hipLaunchKernelGGL((prefix_kernel<FMT, DB, 1>), grid, dim3(256 * prefix_waves(FMT, DB, 1)), 0, s, p);
  else hipLaunchKernelGGL((prefix_kernel<FMT, DB, 2>), grid, dim3(256 * prefix_waves(FMT, DB, 2)), 0, s, p);
}

template <int FMT>
void prefix_launch_db(const AttnSharedLaunch& a, const PrefixParams& p, hipStream_t s) {
  switch (padded_of(a)) {
    case 1: prefix_launch<FMT, 1>(a, p, s); break;
    case 2: prefix_launch<FMT, 2>(a, p, s); break;
    case 3: prefix_launch<FMT, 3>(a, p, s); break;
    default: prefix_launch<FMT, 4>(a, p, s); break;
  }
}

}  // namespace

bool attn_shared_fits(const AttnSharedLaunch& a) {
  if (a.attn.batch * a.attn.q_heads > (int64_t(1) << 30)) return false;
  return prefix_units_of(a) * (prefix_tiles_of(a) + 1) < (int64_t(1) << 31);
}

size_t attn_shared_workspace_bytes(const AttnSharedLaunch& a) {
  if (apart(a)) return attn_workspace_bytes(behind_of(a));
  return pieces_at(a) + (size_t)(prefix_units_of(a) + prefix_grid_of(a)) * (kRows * block_tiles_of(a)) * row_bytes(a);
}

hipError_t launch_attn_shared(const AttnSharedLaunch& a, hipStream_t s) {
  if (apart(a)) {
    ModeParams<kBehind> p;
    const AttnLaunch l = behind_of(a);
    fill_params(l, p);
    p.prefix_table = a.prefix_table;
    p.prefix_len = a.prefix_len;
    p.prefix_most = (int32_t)(a.prefix_width * a.attn.cache.page_size);
    p.own_most = (int32_t)(a.attn.table_width * a.attn.cache.page_size);
    p.own_width = a.attn.table_width;
    return attn_launch(l, p, s);
  }
  PrefixParams p;
  p.cache = a.attn.cache;
  p.q = a.attn.q;
  p.ldq = a.attn.ldq;
  p.rows = head_rows_of(a);
  p.group = a.attn.q_heads / a.attn.cache.heads;
  p.score_factor = score_factor_of(a.attn, p.score_exp);
  p.prefix.len = a.prefix_len;
  p.prefix.table = a.prefix_table;
  p.prefix.part = reinterpret_cast<float*>(static_cast<uint8_t*>(a.attn.ws) + pieces_at(a));
  p.prefix.most = (int32_t)(a.prefix_width * a.attn.cache.page_size);
  p.prefix.units = (int32_t)prefix_units_of(a);
  p.prefix.row_blocks = p.prefix.units / a.attn.cache.heads;
  p.prefix.block_rows = kRows * block_tiles_of(a);
  p.prefix.grid = prefix_grid_of(a);
  p.prefix.each = prefix_each_of(a);
  p.prefix.share = prefix_share_of(a);
  switch (a.attn.format) {
    case kKvBf16: prefix_launch_db<kKvBf16>(a, p, s); break;
    case kKvE4m3: prefix_launch_db<kKvE4m3>(a, p, s); break;
    default: prefix_launch_db<kKvNvfp4>(a, p, s); break;
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  ModeParams<kRaw> own;
  fill_params(a.attn, own);
  own.raw = reinterpret_cast<float*>(static_cast<uint8_t*>(a.attn.ws) + raw_at(a));
  e = attn_launch(a.attn, own, s);
  if (e != hipSuccess) return e;
  JoinParams j;
  j.prefix = p.prefix;
  j.raw = own.raw;
  j.lens = a.attn.lens;
  j.out = a.attn.out;
  j.lse = a.attn.lse;
  j.ldo = a.attn.ldo;
  j.batch = (int32_t)a.attn.batch;
  j.q_heads = a.attn.q_heads;
  j.group = p.group;
  j.head_dim = a.attn.cache.head_dim;
  j.v_scale = a.attn.cache.v_scale;
  switch (padded_of(a)) {
    case 1: join_launch<64>(j, s); break;
    case 2: join_launch<128>(j, s); break;
    case 3: join_launch<192>(j, s); break;
    default: join_launch<256>(j, s); break;
  }
  return hipGetLastError();
}

}  // namespace nvfp4
