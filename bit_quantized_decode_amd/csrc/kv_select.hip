// Which pages attention reads (nvfp4_kv_select) and which a cache keeps (nvfp4_kv_evict): both rank the pages of
// a sequence by 64-bit keys and take the best ones, ties to the lowest place, in ascending order.
//
// Scores.  For a query q and a page whose keys lie between lo and hi channel by channel,
//   sum_d max(q_d lo_d, q_d hi_d)  =  sum_d q_d (q_d < 0 ? lo_d : hi_d)
// is at least q.k of every key in it.  The products of bf16 numbers are exact in fp64 and their sum is
// formed in one order for all pages, whatever the launch: pages of equal bounds tie.
//
// Keys.  An fp64 number's bits, all flipped if it is negative and the sign bit alone if not, order as an
// unsigned integer; a NaN is taken above everything, and key 0 stands for a page that is not there.
//
// Choosing.  A workgroup finds the K-th largest key eight bits at a time: a histogram of the next eight
// bits of the keys that still agree with it, from the first bit in which any two differ; it stops as soon as the
// keys that agree are all taken or all of one kind.  Each thread holds a run of consecutive keys in registers; more
// keys than that stay in memory and are read in each step.
//
// What bounds them is latency where little is to be done: one user's choice of 64 pages out of 2048 for each of 8 kv
// heads (8.4 MB of bounds) takes 15 us, of which the launch 3, the scores 4, the way to the last workgroup of a pair 4 and
// choosing 4; 256 pages of 32 users are evicted in 8 us, 8192 of one in 35 (keys 9, choosing 11, places and outputs 11).
// So are 32 users of up to 512 pages and 8 kv heads of five rows, 20.5 us for 35 MB of bounds: the vector units issue in 24 % of the
// cycles, and wavefronts wait in 51 %.  Where scores are many, their rows count: 150 users of 500 pages (307 MB, most of it from the
// caches) take 47 us for one row a kv head (6.5 TB/s), 77 for five and 190 for sixteen, the vector units issuing in 50, 60 and 69 %
// of the cycles.
#include <algorithm>
#include <type_traits>

#include "attn_kernel.h"

namespace nvfp4 {
namespace {

typedef unsigned long long u64;

__device__ __forceinline__ u64 key_of(double v) {
  const u64 u = (u64)__double_as_longlong(v + 0.0);   // -0 becomes 0
  if (v != v) return ~0ull;
  return u >> 63 ? ~u : u | 1ull << 63;
}

// Keys in memory are written through to it and read from it: other workgroups may have written them.
__device__ __forceinline__ u64 load_key(const u64* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void store_key(u64* p, u64 k) {
  __hip_atomic_store(p, k, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// A thread's share of n keys: those from `begin` to `end`, in registers if PER takes them (each(): (place, key) of
// its keys in order).
template <int THREADS, int PER>
struct Keys {
  u64 k[PER];
  const u64* memory;   // where the keys are if they are not in registers
  int begin, end;
  __device__ __forceinline__ void share(int n) {
    const int per = (n + THREADS - 1) / THREADS;
    begin = min((int)threadIdx.x * per, n);
    end = min(begin + per, n);
  }
  __device__ __forceinline__ bool held(int n) const { return n <= THREADS * PER; }
  template <class F>
  __device__ __forceinline__ void each(int n, F f) const {
    if (held(n)) {
#pragma unroll
      for (int j = 0; j < PER; ++j)
        if (begin + j < end) f(begin + j, k[j]);
    } else {
      for (int i = begin; i < end; ++i) f(i, load_key(memory + i));
    }
  }
};

constexpr int kDigit = 8, kBins = 1 << kDigit;

template <int THREADS>
struct SelectLds {
  int hist[2][kBins];
  int wave_sum[THREADS / 64];
  uint32_t bits[THREADS / 64][4];
  int digit, above;
};

// Exclusive sum of v over the workgroup's threads, in order; total: that of all.
template <int THREADS>
__device__ __forceinline__ int block_scan(int v, int* wave_sum, int& total) {
  const int wave = threadIdx.x >> 6, upto = lane_scan(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 63) wave_sum[wave] = upto;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int i = 0; i < THREADS / 64; ++i) {
    const int s = wave_sum[i];
    before += i < wave ? s : 0;
    total += s;
  }
  return before + upto - v;
}

template <bool AND, int CTRL, int ROWS>
__device__ __forceinline__ uint32_t join_bits(uint32_t v) {
  const uint32_t other = (uint32_t)__builtin_amdgcn_update_dpp(AND ? -1 : 0, (int)v, CTRL, ROWS, 0xf, false);
  return AND ? v & other : v | other;
}
template <bool AND>
__device__ __forceinline__ uint32_t lanes_bits(uint32_t v) {  // of all lanes, in the last
  v = join_bits<AND, 0x111, 0xf>(v);
  v = join_bits<AND, 0x112, 0xf>(v);
  v = join_bits<AND, 0x114, 0xf>(v);
  v = join_bits<AND, 0x118, 0xf>(v);
  v = join_bits<AND, 0x142, 0xa>(v);
  return join_bits<AND, 0x143, 0xc>(v);
}

// Of n keys those to take, in the bits of `mask`: all above `over`, and the first `ties` of those equal to it.
struct Chosen {
  u64 over, mask;
  int ties;
  bool all;            // those equal are no more than `ties`
};

// The `want` largest of n keys, 0 < want < the number of keys that are not 0 (those that are 0 are never
// among them).  Called by all threads.
template <int THREADS, int PER>
__device__ Chosen choose(const Keys<THREADS, PER>& keys, int n, int want, SelectLds<THREADS>& s) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  u64 both = ~0ull, any = 0;
  keys.each(n, [&](int, u64 k) {
    both &= k != 0 ? k : ~0ull;
    any |= k;
  });
  const uint32_t bits[4] = {lanes_bits<true>((uint32_t)both), lanes_bits<true>((uint32_t)(both >> 32)),
                            lanes_bits<false>((uint32_t)any), lanes_bits<false>((uint32_t)(any >> 32))};
  __syncthreads();
  if (lane == 63) {
#pragma unroll
    for (int i = 0; i < 4; ++i) s.bits[wave][i] = bits[i];
  }
  for (int i = tid; i < kBins; i += THREADS) s.hist[0][i] = 0;
  __syncthreads();
  both = ~0ull, any = 0;
#pragma unroll
  for (int i = 0; i < THREADS / 64; ++i) {
    both &= (u64)s.bits[i][1] << 32 | s.bits[i][0];
    any |= (u64)s.bits[i][3] << 32 | s.bits[i][2];
  }
  // Bits above `top` are the same in all keys.
  int top = both == any ? 0 : 64 - __builtin_clzll(both ^ any);
  Chosen c;
  c.mask = top >= 64 ? 0 : ~0ull << top;
  c.over = any & c.mask;
  c.ties = want;
  c.all = false;
  for (int step = 0; top > 0; step ^= 1) {
    const int bits = top < kDigit ? top : kDigit, shift = top - bits;
    int* hist = s.hist[step];
    keys.each(n, [&](int, u64 k) {
      if (k != 0 && (k & c.mask) == c.over) atomicAdd(&hist[(int)(k >> shift) & ((1 << bits) - 1)], 1);
    });
    __syncthreads();
    // The digit that holds the ties-th largest: one wavefront, four digits a lane, from the largest down.
    if (wave == 0) {
      constexpr int kMine = kBins / 64;
      int h[kMine], mine = 0;
#pragma unroll
      for (int j = 0; j < kMine; ++j) {
        h[j] = hist[kBins - 1 - kMine * lane - j];
        mine += h[j];
      }
      int above = lane_scan(mine) - mine;
#pragma unroll
      for (int j = 0; j < kMine; ++j) {
        if (above < c.ties && above + h[j] >= c.ties) {
          s.digit = kBins - 1 - kMine * lane - j;
          s.above = above;
        }
        above += h[j];
      }
    }
    for (int i = tid; i < kBins; i += THREADS) s.hist[step ^ 1][i] = 0;
    __syncthreads();
    const int digit = s.digit, left = hist[digit];
    c.over |= (u64)digit << shift;
    c.mask |= ((1ull << bits) - 1) << shift;
    c.ties -= s.above;
    top = shift;
    c.all = left == c.ties;         // all that agree are taken
    if (c.all) break;
  }
  return c;
}

// Calls emit(place, rank) for each of the thread's keys that `taken(place, key)` says, rank counting them in order over all
// threads; the count.
template <int THREADS, int PER, class TAKEN, class EMIT>
__device__ __forceinline__ int compact(const Keys<THREADS, PER>& keys, int n, int* wave_sum, TAKEN taken, EMIT emit) {
  int mine = 0, total;
  keys.each(n, [&](int i, u64 k) { mine += taken(i, k) ? 1 : 0; });
  int rank = block_scan<THREADS>(mine, wave_sum, total);
  keys.each(n, [&](int i, u64 k) {
    if (taken(i, k)) emit(i, rank++);
  });
  return total;
}

// Ties beyond those that are taken: the place where the first one left out lies (n: none is).
template <int THREADS, int PER>
__device__ __forceinline__ int ties_end(const Keys<THREADS, PER>& keys, int n, const Chosen& c, int* wave_sum, int* out) {
  if (c.all) return n;
  if (threadIdx.x == 0) *out = n;
  __syncthreads();
  compact(keys, n, wave_sum, [&](int, u64 k) { return k != 0 && (k & c.mask) == c.over; },
          [&](int i, int rank) { if (rank == c.ties) *out = i; });
  __syncthreads();
  return *out;
}

__device__ __forceinline__ bool is_chosen(u64 k, int i, const Chosen& c, int end) {
  const u64 m = k & c.mask;
  return k != 0 && (m > c.over || (m == c.over && i < end));
}

// ---- selection for attention --------------------------------------------------

constexpr int kThreads = 256;
constexpr int kCounters = kSelectCounterBytes / sizeof(unsigned);  // (sequence, kv head)s whose scores may be cut over workgroups

constexpr int kSelectFew = 4, kSelectMany = 16;  // keys a thread holds: of tables of up to 1024 and 4096 pages

struct SelectParams {
  KvSelectLaunch a;
  unsigned* counters;
  u64* keys;                           // [batch][heads][table_width]
  int chunk, shares;                   // pages of a workgroup's share; shares of a table
};

// v of another lane of the sixteen.
template <int CTRL>
__device__ __forceinline__ double partner(double v) {
  const u64 u = (u64)__double_as_longlong(v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, 0xf, 0xf, true);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, 0xf, 0xf, true);
  return __longlong_as_double((long long)((u64)hi << 32 | lo));
}
// Sums over sixteen lanes of N values: lane j is left with value j % N's.  Each exchange halves what a lane keeps, the last
// ones (eight and four lanes round) add what is left.
template <int N>
__device__ __forceinline__ double sums16(const double (&v)[N], int j) {
  static_assert(N == 2 || N == 4, "pages at once");
  double a;
  if constexpr (N == 4) {
    const bool two = j & 2, one = j & 1;
    const double x = (two ? v[2] : v[0]) + partner<0x4e>(two ? v[0] : v[2]);
    const double y = (two ? v[3] : v[1]) + partner<0x4e>(two ? v[1] : v[3]);
    a = (one ? y : x) + partner<0xb1>(one ? x : y);
  } else {
    const bool one = j & 1;
    a = (one ? v[1] : v[0]) + partner<0xb1>(one ? v[0] : v[1]);
    a += partner<0x4e>(a);
  }
  a += partner<0x128>(a);
  return a + partner<0x124>(a);
}

// CUT: a table's pages are scored by several workgroups, the last of which to arrive selects.
template <int DB, bool CUT, int PER>
__global__ __launch_bounds__(kThreads) void select_kernel(const SelectParams p) {
  constexpr int kUnits = 2 * DB;       // pairs of channels that a lane holds of a page's bounds
  constexpr int kAhead = DB <= 2 ? 4 : 2;  // pages of a sixteen of lanes whose bounds are read at once
  // Heads of up to 128: a query's values in LDS twice, see below.
  constexpr bool kSplit = DB <= 2;
  constexpr int kParts = kSplit ? 2 : 1, kStage = 16 / kParts;  // (query rows in LDS at a time)
  const KvSelectLaunch& a = p.a;
  __shared__ double s_q[kStage][kUnits][16][2 * kParts];
  __shared__ union {
    u64 keys[CUT ? 1 : kThreads * PER];
    int list[kThreads * PER];
  } s;
  u64* const s_keys = s.keys;
  __shared__ SelectLds<kThreads> s_sel;
  __shared__ int s_end;
  const int tid = threadIdx.x, j = tid & 15;
  // (A table's shares apart in the launch, so that those of a long one are on CUs of their own: 32 ragged users 30 us against 33.)
  const unsigned pairs = gridDim.x / (unsigned)p.shares, share = blockIdx.x / pairs, pair = blockIdx.x - share * pairs;
  const int b = (int)(pair / (unsigned)a.heads), head = (int)(pair - (unsigned)b * (unsigned)a.heads);

  const int64_t most = a.table_width * a.page_size;
  const int64_t len = min((int64_t)max(a.lens[b], 0), most);
  const int n = (int)((len + a.page_size - 1) / a.page_size), budget = (int)a.budget;
  const int first = (int)share * p.chunk;
  const bool scored = n > budget && budget > 1;  // there is a choice
  if (first > 0 && (!scored || first >= n - 1)) return;
  const int32_t* table = a.table + (int64_t)b * a.table_width;
  const auto there = [&](int page) { return page >= 0 && page < a.pages; };
  Keys<kThreads, PER> keys;
  keys.memory = p.keys + (int64_t)pair * a.table_width;
  const int others = max(n - 1, 0);     // the last page is always taken
  keys.share(others);
  const bool in_lds = !CUT && keys.held(others);

  if (scored) {
    const int end = min(first + p.chunk, others);
    u64* memory = p.keys + (int64_t)pair * a.table_width;
    for (int g0 = 0; g0 < a.group; g0 += kStage) {
      const int rows = min(a.group - g0, kStage);
      __syncthreads();
      for (int e = tid; e < rows * kUnits * 32; e += kThreads) {
        const int r = e / (kUnits * 32), x = e - r * (kUnits * 32);   // of a row: [unit][lane][channel]
        const int d = (x >> 1 & 15) * (4 * DB) + 2 * (x >> 5) + (x & 1);
        const uint16_t v = d < a.head_dim ? a.q[(int64_t)b * a.ldq + (int64_t)(head * a.group + g0 + r) * a.head_dim + d] : 0;
        const double q = (double)bf16_lo(v);
        double* to = &s_q[r][0][0][0] + kParts * x;
        if constexpr (kSplit) {
          to[0] = q < 0.0 ? 0.0 : q;
          to[1] = q < 0.0 ? q : 0.0;
        } else {
          to[0] = q;
        }
      }
      __syncthreads();
      // Each sixteen lanes take a page: kAhead of them in flight.
      constexpr int kAtOnce = kThreads / 16;
      for (int i0 = first + (tid >> 4); i0 < end; i0 += kAhead * kAtOnce) {
        int page[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const int i = i0 + k * kAtOnce;
          page[k] = i < end ? table[i] : -1;
        }
        uint2 l[kAhead][DB], h[kAhead][DB];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const uint16_t* lo = a.bounds + ((int64_t)(there(page[k]) ? page[k] : 0) * a.heads + head) * 2 * a.head_dim;
#pragma unroll
          for (int u = 0; u < DB; ++u) {
            const int d = 4 * DB * j + 4 * u;
            l[k][u] = h[k][u] = make_uint2(0, 0);
            if (there(page[k]) && d < a.head_dim) {
              l[k][u] = *reinterpret_cast<const uint2*>(lo + d);
              h[k][u] = *reinterpret_cast<const uint2*>(lo + a.head_dim + d);
            }
          }
        }
        double low[kAhead][2 * kUnits], high[kAhead][2 * kUnits];
        u16x2 largest{0, 0};            // magnitudes: finite below 0x7f80
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
#pragma unroll
          for (int u = 0; u < DB; ++u) {
            const uint32_t w[4] = {l[k][u].x, l[k][u].y, h[k][u].x, h[k][u].y};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              double* to = i < 2 ? &low[k][4 * u + 2 * i] : &high[k][4 * u + 2 * i - 4];
              to[0] = bf16_lo(w[i]);
              to[1] = bf16_hi(w[i]);
              if constexpr (kSplit) largest = __builtin_elementwise_max(largest, __builtin_bit_cast(u16x2, w[i] & 0x7fff7fffu));
            }
          }
        // For finite bounds both products are formed, of q's part below 0 with lo and of the rest with hi, one of which is 0: a
        // select costs two instructions, a product one.  (32 users of 1000 pages of five rows 40 us against 46, of 500 pages
        // of eight rows 31 against 36; one row, for which four pages' registers at once are too many, 19 against 17.  256-wide
        // heads, whose parts LDS takes longer to read than selects take: 40 against 35.)
        double best = -__builtin_inf();
        bool nan = false;
        const auto score = [&](auto both) {
          for (int r = 0; r < rows; ++r) {
            double sum[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) sum[k] = 0.0;
#pragma unroll
            for (int u = 0; u < kUnits; ++u)
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const double up = s_q[r][u][j][kParts * c], down = s_q[r][u][j][kParts * c + kParts - 1];
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                  const double lo = low[k][2 * u + c], hi = high[k][2 * u + c];
                  if constexpr (decltype(both)::value) {
                    sum[k] = __builtin_fma(up, hi, sum[k]);
                    sum[k] = __builtin_fma(down, lo, sum[k]);
                  } else {
                    sum[k] = down < 0.0 ? __builtin_fma(down, lo, sum[k]) : __builtin_fma(up, hi, sum[k]);
                  }
                }
              }
            const double all = sums16(sum, j);
            nan |= all != all;
            best = fmax(best, all);
          }
        };
        const bool finite = !__any(largest[0] >= 0x7f80 || largest[1] >= 0x7f80);
        if (kSplit && finite) score(std::bool_constant<kSplit>());
        else score(std::false_type());
        const int k = j % kAhead, i = i0 + k * kAtOnce;
        if (j < kAhead && i < end) {
          int mine = page[0];
#pragma unroll
          for (int m = 1; m < kAhead; ++m) mine = k == m ? page[m] : mine;
          const u64 key = !there(mine) ? 0 : nan ? ~0ull : key_of(best);
          if (in_lds) s_keys[i] = g0 > 0 ? max(s_keys[i], key) : key;
          else store_key(memory + i, g0 > 0 ? max(load_key(memory + i), key) : key);
        }
      }
    }
    const unsigned shares = (unsigned)((others + p.chunk - 1) / p.chunk);
    if (CUT && shares > 1) {
      if (!arrive_last(p.counters + pair, shares)) return;
    } else {
      __builtin_amdgcn_s_waitcnt(0);    // keys in memory have arrived there
      __syncthreads();
    }
    if (keys.held(others)) {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int at = keys.begin + i;
        keys.k[i] = at >= keys.end ? 0 : in_lds ? s_keys[at] : load_key(memory + at);
      }
    }
  }

  // The best `budget - 1` of the pages before the last that are there, and the last.
  int32_t* out = a.pages_out + (int64_t)pair * a.budget;
  int taken = 0;
  if (others > 0 && budget > 1) {
    // (Places first, then all their pages at once: a table's entry is a trip to memory.)
    const bool listed = keys.held(others);
    const auto emit = [&](int i, int place) {
      if (listed) s.list[place] = i;
      else out[place] = table[i];
    };
    int mine = 0, total = 0;
    if (scored) {
      keys.each(others, [&](int, u64 k) { mine += k != 0 ? 1 : 0; });
      block_scan<kThreads>(mine, s_sel.wave_sum, total);
    }
    if (total > budget - 1) {
      const Chosen c = choose(keys, others, budget - 1, s_sel);
      const int end = ties_end(keys, others, c, s_sel.wave_sum, &s_end);
      taken = compact(keys, others, s_sel.wave_sum, [&](int i, u64 k) { return is_chosen(k, i, c, end); }, emit);
    } else {                            // all that are there
      for (int i = keys.begin; i < keys.end; ++i) taken += there(table[i]) ? 1 : 0;
      int place = block_scan<kThreads>(taken, s_sel.wave_sum, taken);
      for (int i = keys.begin; i < keys.end; ++i)
        if (there(table[i])) emit(i, place++);
    }
    __syncthreads();
    if (listed)
      for (int i = tid; i < taken; i += kThreads) out[i] = table[s.list[i]];
  }
  if (tid == 0 && n > 0) out[taken] = there(table[n - 1]) ? table[n - 1] : -1;
  if (n > 0) ++taken;
  if (tid == 0 && head == 0)
    a.lens_out[b] = n > 0 ? (int)((taken - 1) * (int64_t)a.page_size + (len - 1) % a.page_size + 1) : 0;
  for (int i = taken + tid; i < budget; i += kThreads) out[i] = -1;
}

// ---- eviction -------------------------------------------------------------------

struct EvictParams {
  KvEvictLaunch a;
  u64* keys;                           // [batch][table_width], if registers do not hold them
};

constexpr int kEvictFew = 256, kEvictMany = 1024;  // threads
constexpr int kPerFew = 4, kPerMany = 8;           // keys that each holds
constexpr int kHeadsAtOnce = 8, kPagesAtOnce = 4;  // loads in flight of a thread

// One workgroup a sequence.
template <int THREADS, int PER>
__global__ __launch_bounds__(THREADS) void evict_kernel(const EvictParams p) {
  const KvEvictLaunch& a = p.a;
  __shared__ union {
    u64 keys[THREADS * PER];
    int list[THREADS * PER];      // places of the pages that stay, in order, and behind them of those dropped
  } s;
  __shared__ int s_table[THREADS * PER];
  __shared__ SelectLds<THREADS> s_sel;
  __shared__ int s_end;
  const int tid = threadIdx.x, b = blockIdx.x;
  const int64_t most = a.table_width * a.page_size;
  const int64_t len = min((int64_t)max(a.lens[b], 0), most);
  const int n = (int)((len + a.page_size - 1) / a.page_size), budget = (int)a.budget;
  const int32_t* table = a.table + (int64_t)b * a.table_width;
  const float* weights = a.weights + (int64_t)b * a.heads * a.table_width;
  u64* memory = p.keys ? p.keys + (int64_t)b * a.table_width : nullptr;
  Keys<THREADS, PER> keys;
  keys.memory = memory;
  keys.share(n);
  const bool held = keys.held(n);

  // Pages from `late` on are the newest ones, kept whatever they weigh: key 1 if they are there.  The others' keys are
  // their weights', the first `sink` places above all.  Key 0: not there.
  const int late = a.recent < n ? n - (int)a.recent : 0;
  const auto weigh = [&](int base, auto at_once) {
    constexpr int kPages = decltype(at_once)::value;
    int page[kPages];
    double sum[kPages];
#pragma unroll
    for (int m = 0; m < kPages; ++m) {
      const int i = base + m * THREADS + tid;
      page[m] = i < n ? table[i] : -1;
      sum[m] = 0.0;
    }
    for (int h0 = 0; h0 < a.heads; h0 += kHeadsAtOnce) {
      float w[kPages][kHeadsAtOnce];
#pragma unroll
      for (int m = 0; m < kPages; ++m) {
        const int i = base + m * THREADS + tid;
#pragma unroll
        for (int h = 0; h < kHeadsAtOnce; ++h)
          w[m][h] = h0 + h < a.heads && i < late ? weights[(int64_t)(h0 + h) * a.table_width + i] : 0.0f;
      }
#pragma unroll
      for (int m = 0; m < kPages; ++m)
#pragma unroll
        for (int h = 0; h < kHeadsAtOnce; ++h) sum[m] += (double)w[m][h];
    }
#pragma unroll
    for (int m = 0; m < kPages; ++m) {
      const int i = base + m * THREADS + tid;
      if (i >= n) continue;
      u64 k = page[m] >= 0 || i == n - 1 ? 1 : 0;
      if (i < late && k != 0) k = i < a.sink ? ~0ull : max(key_of(sum[m]), (u64)2);
      if (held) {
        s.keys[i] = k;
        s_table[i] = page[m];
      } else {
        store_key(memory + i, k);
      }
    }
  };
  int base = 0;
  for (; n - base > THREADS; base += kPagesAtOnce * THREADS) weigh(base, std::integral_constant<int, kPagesAtOnce>());
  if (base < n) weigh(base, std::integral_constant<int, 1>());
  __builtin_amdgcn_s_waitcnt(0);        // keys in memory have arrived there
  __syncthreads();
  if (held) {
#pragma unroll
    for (int i = 0; i < PER; ++i) keys.k[i] = keys.begin + i < keys.end ? s.keys[keys.begin + i] : 0;
  }
  // How many there are of each kind.  Of the newest, the oldest that the budget has no room for are left out: those of
  // rank below `skip`.
  int mine = 0, newest, others;
  keys.each(n, [&](int i, u64 k) { mine += k != 0 && i < late ? 1 : 0; });
  block_scan<THREADS>(mine, s_sel.wave_sum, others);
  mine = 0;
  keys.each(n, [&](int i, u64 k) { mine += k != 0 && i >= late ? 1 : 0; });
  const int rank0 = block_scan<THREADS>(mine, s_sel.wave_sum, newest);
  const int skip = max(newest - budget, 0), want = min(budget - (newest - skip), others);
  // The chosen ones of the others: their keys alone are looked at.
  Chosen c{0, 0, 0, true};
  int end = n;
  if (want > 0 && want < others) {
    Keys<THREADS, PER> old = keys;
    old.share(n);
    old.end = min(old.end, late);
    c = choose(old, n, want, s_sel);
    end = ties_end(old, n, c, s_sel.wave_sum, &s_end);
  }
  int late_rank = rank0;
  const auto kept = [&](int i, u64 k, int rank) {
    if (k == 0) return false;
    if (i >= late) return rank >= skip;
    return want > 0 && (want >= others || is_chosen(k, i, c, end));
  };
  // Kept pages, dropped ones and their places in one go over the keys.
  int stay = 0, gone = 0, stay_all, gone_all;
  keys.each(n, [&](int i, u64 k) {
    const bool keep = kept(i, k, late_rank);
    late_rank += k != 0 && i >= late ? 1 : 0;
    stay += keep ? 1 : 0;
    gone += !keep && k != 0 ? 1 : 0;
  });
  int stay_at = block_scan<THREADS>(stay, s_sel.wave_sum, stay_all);
  int gone_at = block_scan<THREADS>(gone, s_sel.wave_sum, gone_all);
  late_rank = rank0;
  int32_t* out = a.table_out + (int64_t)b * a.budget;
  int32_t* freed = a.freed ? a.freed + (int64_t)b * a.table_width : nullptr;
  // (Places first, then all pages and weights at once: each is a trip to memory.  The scans above come after the last read
  // of the keys in LDS.)
  const auto move = [&](int i, int to) {
    out[to] = held ? s_table[i] : table[i];
    if (!a.weights_out) return;
    float* dst = a.weights_out + (int64_t)b * a.heads * a.budget + to;
    for (int h0 = 0; h0 < a.heads; h0 += kHeadsAtOnce) {
      float w[kHeadsAtOnce];
#pragma unroll
      for (int h = 0; h < kHeadsAtOnce; ++h)
        if (h0 + h < a.heads) w[h] = weights[(int64_t)(h0 + h) * a.table_width + i];
#pragma unroll
      for (int h = 0; h < kHeadsAtOnce; ++h)
        if (h0 + h < a.heads) dst[(int64_t)(h0 + h) * a.budget] = w[h];
    }
  };
  keys.each(n, [&](int i, u64 k) {
    const bool keep = kept(i, k, late_rank);
    late_rank += k != 0 && i >= late ? 1 : 0;
    if (keep) {
      if (held) s.list[stay_at] = i;
      else move(i, stay_at);
      ++stay_at;
    } else if (k != 0) {
      if (held) s.list[stay_all + gone_at] = i;
      else if (freed) freed[gone_at] = table[i];
      ++gone_at;
    }
  });
  if (held) {
    __syncthreads();
    for (int r = tid; r < stay_all; r += THREADS) move(s.list[r], r);
    if (freed)
      for (int r = tid; r < gone_all; r += THREADS) freed[r] = s_table[s.list[stay_all + r]];
  }
  if (tid == 0) a.lens_out[b] = n > 0 ? (int)((stay_all - 1) * (int64_t)a.page_size + (len - 1) % a.page_size + 1) : 0;
  for (int i = stay_all + tid; i < budget; i += THREADS) {
    out[i] = -1;
    if (a.weights_out)
      for (int h = 0; h < a.heads; ++h) a.weights_out[((int64_t)b * a.heads + h) * a.budget + i] = 0.0f;
  }
  if (freed)
    for (int64_t i = gone_all + tid; i < a.table_width; i += THREADS) freed[i] = -1;
  // The workspace's front, where other calls have their counters, held the first sequence's keys alone: it is left zero.
  static_assert(kCounterBytes <= kEvictMany * kPerMany * sizeof(u64), "counters under one sequence's keys");
  if (!held && b == 0) {
    __syncthreads();
    for (int i = tid; i < (int)(kCounterBytes / sizeof(u64)); i += THREADS) store_key(memory + i, 0);
  }
}

// Pages of a workgroup's share: one workgroup a (sequence, kv head) where those fill the GPU or have no counter; else
// so that there are four a CU, but 64 pages at least.  (32 users of 8 kv heads: two a CU 45 us for 1000 pages against 42.6, 25.8 for 500
// against 25.3.  One user: shares of 32 pages and more 23.4 us for 2048 pages against 20.7, of 128 22.3; for 500 10.2 and 12.5 against
// 9.7.)
int64_t chunk_of(const KvSelectLaunch& a) {
  const int64_t pairs = a.batch * a.heads;
  if (pairs >= kCounters) return a.table_width;
  const int64_t parts = kCounters / pairs;
  const int64_t chunk = ((a.table_width + parts - 1) / parts + 15) / 16 * 16;
  return std::min(a.table_width, std::max<int64_t>(chunk, 64));
}

template <int DB, int PER>
void select_launch_per(const SelectParams& p, bool cut, dim3 grid, hipStream_t s) {
  if (cut) hipLaunchKernelGGL((select_kernel<DB, true, PER>), grid, dim3(kThreads), 0, s, p);
  else hipLaunchKernelGGL((select_kernel<DB, false, PER>), grid, dim3(kThreads), 0, s, p);
}
template <int DB>
void select_launch(const SelectParams& p, bool cut, dim3 grid, hipStream_t s) {
  // (One user of 1000 pages 14.1 us against 18.5, 32 users of 500 25.4 against 30.1, 150 of 500 77.6 against 84.7.)
  if (p.a.table_width <= kThreads * kSelectFew) select_launch_per<DB, kSelectFew>(p, cut, grid, s);
  else select_launch_per<DB, kSelectMany>(p, cut, grid, s);
}

}  // namespace

size_t kv_select_workspace_bytes(const KvSelectLaunch& a) {
  if (a.table_width <= a.budget) return 0;
  if (chunk_of(a) >= a.table_width && a.table_width <= kThreads * kSelectMany) return 0;
  return kCounterBytes + (size_t)(a.batch * a.heads) * a.table_width * sizeof(u64);
}

hipError_t launch_kv_select(const KvSelectLaunch& a, hipStream_t s) {
  SelectParams p;
  p.a = a;
  p.counters = static_cast<unsigned*>(a.ws);
  p.keys = a.ws ? reinterpret_cast<u64*>(static_cast<uint8_t*>(a.ws) + kCounterBytes) : nullptr;
  const int64_t chunk = std::max<int64_t>(a.table_width <= a.budget ? a.table_width : chunk_of(a), 1);
  p.chunk = (int)chunk;
  const bool cut = chunk < a.table_width;
  p.shares = (int)std::max<int64_t>((a.table_width + chunk - 1) / chunk, 1);
  const dim3 grid((unsigned)(a.batch * a.heads * p.shares));
  switch ((a.head_dim + 63) / 64) {
    case 1: select_launch<1>(p, cut, grid, s); break;
    case 2: select_launch<2>(p, cut, grid, s); break;
    case 3: select_launch<3>(p, cut, grid, s); break;
    default: select_launch<4>(p, cut, grid, s); break;
  }
  return hipGetLastError();
}

size_t kv_evict_workspace_bytes(const KvEvictLaunch& a) {
  return a.table_width <= kEvictMany * kPerMany ? 0 : (size_t)a.batch * a.table_width * sizeof(u64);
}

hipError_t launch_kv_evict(const KvEvictLaunch& a, hipStream_t s) {
  EvictParams p;
  p.a = a;
  p.keys = static_cast<u64*>(a.ws);
  const dim3 grid((unsigned)a.batch);
  // Few threads where they hold the table's keys.  (32 users of 256 pages 8.4 us against 12.5, of 1000 15.0 against 15.7, of 2000 on
  // eight keys a thread 24.8 against 20.0; 300 users of 1000 18.0 against 30.1.)
  if (a.table_width <= kEvictFew * kPerFew) hipLaunchKernelGGL((evict_kernel<kEvictFew, kPerFew>), grid, dim3(kEvictFew), 0, s, p);
  else hipLaunchKernelGGL((evict_kernel<kEvictMany, kPerMany>), grid, dim3(kEvictMany), 0, s, p);
  return hipGetLastError();
}

}  // namespace nvfp4
