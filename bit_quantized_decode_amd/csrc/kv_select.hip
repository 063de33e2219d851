// Which pages attention reads (nvfp4_kv_select) and which a cache keeps (nvfp4_kv_evict): both rank the pages of
// a sequence by 64-bit keys and take the best ones, ties to the lowest place, in ascending order.
//
// Scores.  For a query q and a page whose keys lie between lo and hi channel by channel,
//   sum_d max(q_d lo_d, q_d hi_d)  =  sum_d q_d (q_d < 0 ? lo_d : hi_d)
// is at least q.k of every key in it.  The products of bf16 numbers are exact in fp64, and their sum is
// rounded to 2^-53, so that the order of two pages does not depend on how the sum is cut; ties are ties.
//
// Keys.  An fp64 number's bits, all flipped if it is negative and the sign bit alone if not, order as an
// unsigned integer; a NaN is taken above everything, and key 0 stands for a page that is not there.
//
// Selection.  A workgroup finds the K-th largest key eight bits at a time: a histogram of the next eight
// bits of the keys that still agree with it, from the first bit in which any two differ; it stops as soon as the
// keys that agree are all taken or all of one kind.
#include <algorithm>

#include "attn_launchers.h"
#include "device_common.h"

namespace nvfp4 {
namespace {

typedef unsigned long long u64;

__device__ __forceinline__ u64 key_of(double v) {
  const u64 u = (u64)__double_as_longlong(v + 0.0);   // -0 becomes 0
  if (v != v) return ~0ull;
  return u >> 63 ? ~u : u | 1ull << 63;
}

// Keys of one sequence (and kv head), in LDS where they fit, in memory beyond (written through to it and read from
// it: other workgroups may have written them).
constexpr int kKeysInLds = 4096;
struct Keys {
  u64* lds;            // nullptr: in memory
  u64* memory;
};
__device__ __forceinline__ u64 load_key(const u64* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void store_key(u64* p, u64 k) {
  __hip_atomic_store(p, k, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ u64 get_key(const Keys& k, int i) { return k.lds ? k.lds[i] : load_key(k.memory + i); }

template <int THREADS>
struct SelectLds {
  int hist[256];
  int wave_sum[THREADS / 64];
  u64 all_and[THREADS / 64], all_or[THREADS / 64];
  int digit, above;
};

// Exclusive sum of v over the workgroup's threads, in order; total: that of all.
template <int THREADS>
__device__ __forceinline__ int block_scan(int v, int* wave_sum, int& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int upto = v;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int other = __shfl_up(upto, off);
    upto += lane >= off ? other : 0;
  }
  __syncthreads();
  if (lane == 63) wave_sum[wave] = upto;
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

// Of n keys those to take, in the bits of `mask`: all above `over`, and the first `ties` of those equal to it.
struct Chosen {
  u64 over, mask;
  int ties;
  bool all;            // those equal are no more than `ties`
};

// The `want` largest of n keys, 0 < want <= the number of keys that are not 0 (those that are 0 are never
// among them).  Called by all threads, after the keys are visible to all.
template <int THREADS>
__device__ Chosen choose(const Keys& keys, int n, int want, SelectLds<THREADS>& s) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  u64 both = ~0ull, any = 0;
  for (int i = tid; i < n; i += THREADS) {
    const u64 k = get_key(keys, i);
    if (k != 0) {
      both &= k;
      any |= k;
    }
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) {
    both &= __shfl_xor(both, off);
    any |= __shfl_xor(any, off);
  }
  __syncthreads();
  if (lane == 0) {
    s.all_and[wave] = both;
    s.all_or[wave] = any;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < THREADS / 64; ++i) {
    both &= s.all_and[i];
    any |= s.all_or[i];
  }
  // Bits above `top` are the same in all keys.
  int top = both == any ? 0 : 64 - __builtin_clzll(both ^ any);
  Chosen c;
  c.mask = top >= 64 ? 0 : ~0ull << top;
  c.over = any & c.mask;
  c.ties = want;
  c.all = false;
  while (top > 0) {
    const int bits = top < 8 ? top : 8, shift = top - bits;
    __syncthreads();
    for (int i = tid; i < 256; i += THREADS) s.hist[i] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += THREADS) {
      const u64 k = get_key(keys, i);
      if (k != 0 && (k & c.mask) == c.over) atomicAdd(&s.hist[(int)(k >> shift) & ((1 << bits) - 1)], 1);
    }
    __syncthreads();
    // The digit that holds the ties-th largest: one wavefront, four digits a lane, from the largest down.
    if (wave == 0) {
      int h[4], mine = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        h[j] = s.hist[255 - 4 * lane - j];
        mine += h[j];
      }
      int upto = mine;
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const int other = __shfl_up(upto, off);
        upto += lane >= off ? other : 0;
      }
      int above = upto - mine;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (above < c.ties && above + h[j] >= c.ties) {
          s.digit = 255 - 4 * lane - j;
          s.above = above;
        }
        above += h[j];
      }
    }
    __syncthreads();
    const int digit = s.digit, left = s.hist[digit];
    c.over |= (u64)digit << shift;
    c.mask |= ((1ull << bits) - 1) << shift;
    c.ties -= s.above;
    top = shift;
    c.all = left == c.ties;         // all that agree are taken
    if (c.all) break;
  }
  __syncthreads();
  return c;
}

// Calls emit(i, place) for each i < n that `taken(i)` says, place counting them in order, over all threads; the count.
template <int THREADS, class TAKEN, class EMIT>
__device__ __forceinline__ int compact(int n, int* wave_sum, TAKEN taken, EMIT emit) {
  const int per = (n + THREADS - 1) / THREADS, i0 = min((int)threadIdx.x * per, n), i1 = min(i0 + per, n);
  int mine = 0;
  for (int i = i0; i < i1; ++i) mine += taken(i) ? 1 : 0;
  int total, place = block_scan<THREADS>(mine, wave_sum, total);
  for (int i = i0; i < i1; ++i)
    if (taken(i)) emit(i, place++);
  return total;
}

// Ties beyond those that are taken: the place where the first one left out lies (n: none is).
template <int THREADS>
__device__ __forceinline__ int ties_end(const Keys& keys, int n, const Chosen& c, int* wave_sum, int* out) {
  if (c.all) return n;
  if (threadIdx.x == 0) *out = n;
  __syncthreads();
  compact<THREADS>(n, wave_sum, [&](int i) { const u64 k = get_key(keys, i); return k != 0 && (k & c.mask) == c.over; },
                   [&](int i, int place) { if (place == c.ties) *out = i; });
  __syncthreads();
  return *out;
}

__device__ __forceinline__ bool is_chosen(u64 k, int i, const Chosen& c, int end) {
  const u64 m = k & c.mask;
  return k != 0 && (m > c.over || (m == c.over && i < end));
}

// ---- selection for attention --------------------------------------------------

constexpr int kThreads = 256;
constexpr int kStage = 16;             // query rows in LDS at a time
constexpr int kCounters = 1024;        // (sequence, kv head)s whose scores may be cut over several workgroups

struct SelectParams {
  KvSelectLaunch a;
  unsigned* counters;
  u64* keys;                           // [batch][heads][table_width]
  int chunk, shares;                   // pages of a workgroup's share; shares of a table
  bool cut;                            // over several workgroups
};

template <int DB>
__global__ __launch_bounds__(kThreads) void select_kernel(const SelectParams p) {
  constexpr int kUnits = 2 * DB;       // pairs of channels that a lane holds of a page's bounds
  const KvSelectLaunch& a = p.a;
  __shared__ double s_q[kStage][kUnits][16][2];
  __shared__ u64 s_keys[kKeysInLds];
  __shared__ SelectLds<kThreads> s_sel;
  __shared__ int s_end;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, j = lane & 15;
  const unsigned wg = blockIdx.x / (unsigned)p.shares;
  const int b = (int)(wg / (unsigned)a.heads), head = (int)(wg - (unsigned)b * (unsigned)a.heads);
  const int64_t pair = wg;

  const int64_t most = a.table_width * a.page_size;
  const int64_t len = min((int64_t)max(a.lens[b], 0), most);
  const int n = (int)((len + a.page_size - 1) / a.page_size), budget = (int)a.budget;
  const int first = (int)(blockIdx.x - wg * (unsigned)p.shares) * p.chunk;
  const bool scored = n > budget;       // there is a choice
  if (first > 0 && (!scored || first >= n - 1)) return;
  const int32_t* table = a.table + (int64_t)b * a.table_width;
  const auto there = [&](int i) { const int page = table[i]; return page >= 0 && page < a.pages; };
  Keys keys;
  keys.lds = !p.cut && n <= kKeysInLds ? s_keys : nullptr;
  keys.memory = p.keys + pair * a.table_width;

  if (scored) {
    const int end = min(first + p.chunk, n - 1);    // the last page is always taken
    for (int g0 = 0; g0 < a.group; g0 += kStage) {
      const int rows = min(a.group - g0, kStage);
      __syncthreads();
      for (int e = tid; e < rows * kUnits * 32; e += kThreads) {
        const int r = e / (kUnits * 32), x = e - r * (kUnits * 32);   // of a row: [unit][lane][2]
        const int d = (x >> 1 & 15) * (4 * DB) + 2 * (x >> 5) + (x & 1);
        const uint16_t v = d < a.head_dim ? a.q[(int64_t)b * a.ldq + (int64_t)(head * a.group + g0 + r) * a.head_dim + d] : 0;
        (&s_q[r][0][0][0])[x] = (double)bf16_lo(v);
      }
      __syncthreads();
      for (int i0 = first + 4 * wave; i0 < end; i0 += 4 * (kThreads / 64)) {
        const int i = i0 + (lane >> 4);
        const bool live = i < end && there(min(i, end - 1));
        const int page = live ? table[i] : 0;
        const uint16_t* lo = a.bounds + ((int64_t)page * a.heads + head) * 2 * a.head_dim;
        double low[2 * kUnits], high[2 * kUnits];
#pragma unroll
        for (int u = 0; u < DB; ++u) {
          const int d = 4 * DB * j + 4 * u;
          uint2 l = make_uint2(0, 0), h = l;
          if (live && d < a.head_dim) {
            l = *reinterpret_cast<const uint2*>(lo + d);
            h = *reinterpret_cast<const uint2*>(lo + a.head_dim + d);
          }
          low[4 * u] = bf16_lo(l.x), low[4 * u + 1] = bf16_hi(l.x), low[4 * u + 2] = bf16_lo(l.y), low[4 * u + 3] = bf16_hi(l.y);
          high[4 * u] = bf16_lo(h.x), high[4 * u + 1] = bf16_hi(h.x), high[4 * u + 2] = bf16_lo(h.y), high[4 * u + 3] = bf16_hi(h.y);
        }
        u64 best = 0;
        for (int r = 0; r < rows; ++r) {
          double sum = 0.0;
#pragma unroll
          for (int u = 0; u < kUnits; ++u) {
            const double q0 = s_q[r][u][j][0], q1 = s_q[r][u][j][1];
            sum += q0 * (q0 < 0.0 ? low[2 * u] : high[2 * u]);
            sum += q1 * (q1 < 0.0 ? low[2 * u + 1] : high[2 * u + 1]);
          }
#pragma unroll
          for (int off = 8; off >= 1; off >>= 1) sum += __shfl_xor(sum, off);
          best = max(best, key_of(sum));
        }
        if (j == 0 && i < end) {
          if (!live) best = 0;
          u64* to = keys.lds ? keys.lds + i : keys.memory + i;
          if (keys.lds) *to = g0 > 0 ? max(*to, best) : best;
          else store_key(to, g0 > 0 ? max(load_key(to), best) : best);
        }
      }
    }
    if (p.cut) {
      const unsigned shares = (unsigned)((n - 1 + p.chunk - 1) / p.chunk);
      if (shares > 1 && !arrive_last(p.counters + pair, shares)) return;
      if (n <= kKeysInLds) {            // this workgroup reads them several times
        if (shares == 1) {
          __builtin_amdgcn_s_waitcnt(0);
          __syncthreads();
        }
        for (int i = tid; i < n - 1; i += kThreads) s_keys[i] = load_key(keys.memory + i);
        keys.lds = s_keys;
      }
    }
    __builtin_amdgcn_s_waitcnt(0);      // keys in memory have arrived there
    __syncthreads();
  }

  // The best `budget - 1` of the pages before the last that are there, and the last.
  int32_t* out = a.pages_out + pair * a.budget;
  int taken = 0;
  if (n > 1 && budget > 1) {
    const auto emit = [&](int i, int place) { out[place] = table[i]; };
    int total = 0;
    if (scored) {
      int mine = 0;
      for (int i = tid; i < n - 1; i += kThreads) mine += get_key(keys, i) != 0 ? 1 : 0;
      block_scan<kThreads>(mine, s_sel.wave_sum, total);
    }
    if (scored && total > budget - 1) {
      const Chosen c = choose<kThreads>(keys, n - 1, budget - 1, s_sel);
      const int end = ties_end<kThreads>(keys, n - 1, c, s_sel.wave_sum, &s_end);
      taken = compact<kThreads>(n - 1, s_sel.wave_sum, [&](int i) { return is_chosen(get_key(keys, i), i, c, end); }, emit);
    } else {
      taken = compact<kThreads>(n - 1, s_sel.wave_sum, there, emit);
    }
  }
  if (tid == 0) {
    if (n > 0) out[taken++] = there(n - 1) ? table[n - 1] : -1;
    s_end = taken;
    if (head == 0) a.lens_out[b] = n > 0 ? (int)((taken - 1) * (int64_t)a.page_size + (len - 1) % a.page_size + 1) : 0;
  }
  __syncthreads();
  for (int i = s_end + tid; i < budget; i += kThreads) out[i] = -1;
}

// ---- eviction -------------------------------------------------------------------

constexpr int kEvictThreads = 1024;

struct EvictParams {
  KvEvictLaunch a;
  u64* keys;                           // [batch][table_width], if they do not fit LDS
};

__global__ __launch_bounds__(kEvictThreads) void evict_kernel(const EvictParams p) {
  const KvEvictLaunch& a = p.a;
  __shared__ u64 s_keys[kKeysInLds];
  __shared__ SelectLds<kEvictThreads> s_sel;
  __shared__ int s_end;
  const int tid = threadIdx.x, b = blockIdx.x;
  const int64_t most = a.table_width * a.page_size;
  const int64_t len = min((int64_t)max(a.lens[b], 0), most);
  const int n = (int)((len + a.page_size - 1) / a.page_size), budget = (int)a.budget;
  const int32_t* table = a.table + (int64_t)b * a.table_width;
  const float* weights = a.weights + (int64_t)b * a.heads * a.table_width;
  const auto there = [&](int i) { return table[i] >= 0 || i == n - 1; };
  Keys keys;
  keys.lds = n <= kKeysInLds ? s_keys : nullptr;
  keys.memory = p.keys ? p.keys + (int64_t)b * a.table_width : nullptr;

  // Pages from `late` on are the newest ones, kept whatever they weigh: those that are there, as far as the budget goes.
  int late = a.recent < n ? n - (int)a.recent : 0, newest = 0, mine = 0;
  for (int i = late + tid; i < n; i += kEvictThreads) mine += there(i) ? 1 : 0;
  block_scan<kEvictThreads>(mine, s_sel.wave_sum, newest);
  int skip = max(newest - budget, 0);   // of them, the oldest that the budget leaves out
  newest -= skip;
  // The others by weight, the first `sink` places above all weights.
  int others = 0;
  mine = 0;
  for (int i = tid; i < late; i += kEvictThreads) {
    u64 k = 0;
    if (table[i] >= 0) {
      double sum = 0.0;
      for (int h = 0; h < a.heads; ++h) sum += (double)weights[(int64_t)h * a.table_width + i];
      k = i < a.sink ? ~0ull : key_of(sum);
      ++mine;
    }
    if (keys.lds) keys.lds[i] = k;
    else store_key(keys.memory + i, k);
  }
  if (!keys.lds) __builtin_amdgcn_s_waitcnt(0);
  block_scan<kEvictThreads>(mine, s_sel.wave_sum, others);
  const int want = min(budget - newest, others);
  Chosen c{~0ull, ~0ull, 0, true};
  int end = 0;
  if (want > 0 && want < others) {
    c = choose<kEvictThreads>(keys, late, want, s_sel);
    end = ties_end<kEvictThreads>(keys, late, c, s_sel.wave_sum, &s_end);
  }
  // How many of the newest are left out is a matter of their order: those before place `from`.
  int from = late;
  if (skip > 0) {
    __syncthreads();
    if (tid == 0) s_end = n;
    __syncthreads();
    const int late0 = late;
    compact<kEvictThreads>(n - late0, s_sel.wave_sum, [&](int i) { return there(late0 + i); },
                           [&](int i, int place) { if (place == skip) s_end = late0 + i; });
    __syncthreads();
    from = s_end;
    __syncthreads();
  }
  const auto kept = [&](int i) {
    if (i >= late) return i >= from && there(i);
    if (want <= 0) return false;
    return want >= others ? table[i] >= 0 : is_chosen(get_key(keys, i), i, c, end);
  };
  int32_t* out = a.table_out + (int64_t)b * a.budget;
  const int taken = compact<kEvictThreads>(n, s_sel.wave_sum, kept, [&](int i, int place) {
    out[place] = table[i];
    if (a.weights_out)
      for (int h = 0; h < a.heads; ++h)
        a.weights_out[((int64_t)b * a.heads + h) * a.budget + place] = weights[(int64_t)h * a.table_width + i];
  });
  if (tid == 0) a.lens_out[b] = n > 0 ? (int)((taken - 1) * (int64_t)a.page_size + (len - 1) % a.page_size + 1) : 0;
  for (int i = taken + tid; i < budget; i += kEvictThreads) {
    out[i] = -1;
    if (a.weights_out)
      for (int h = 0; h < a.heads; ++h) a.weights_out[((int64_t)b * a.heads + h) * a.budget + i] = 0.0f;
  }
  if (a.freed) {
    int32_t* gone = a.freed + (int64_t)b * a.table_width;
    const int dropped = compact<kEvictThreads>(n, s_sel.wave_sum, [&](int i) { return table[i] >= 0 && !kept(i); },
                                               [&](int i, int place) { gone[place] = table[i]; });
    for (int64_t i = dropped + tid; i < a.table_width; i += kEvictThreads) gone[i] = -1;
  }
}

// Pages of a workgroup's share: one workgroup a (sequence, kv head) where those fill the GPU or have no counter; else
// so that there are four a CU, but 64 pages at least.
int64_t chunk_of(const KvSelectLaunch& a) {
  const int64_t pairs = a.batch * a.heads;
  if (pairs >= kCounters) return a.table_width;
  const int64_t parts = kCounters / pairs;
  const int64_t chunk = ((a.table_width + parts - 1) / parts + 15) / 16 * 16;
  return std::min(a.table_width, std::max<int64_t>(chunk, 64));
}

}  // namespace

size_t kv_select_workspace_bytes(const KvSelectLaunch& a) {
  if (a.table_width <= a.budget) return 0;
  if (chunk_of(a) >= a.table_width && a.table_width <= kKeysInLds) return 0;
  return kCounters * sizeof(unsigned) + (size_t)(a.batch * a.heads) * a.table_width * sizeof(u64);
}

hipError_t launch_kv_select(const KvSelectLaunch& a, hipStream_t s) {
  SelectParams p;
  p.a = a;
  p.counters = static_cast<unsigned*>(a.ws);
  p.keys = reinterpret_cast<u64*>(static_cast<uint8_t*>(a.ws) + kCounters * sizeof(unsigned));
  const int64_t chunk = std::max<int64_t>(a.table_width <= a.budget ? a.table_width : chunk_of(a), 1);
  p.chunk = (int)chunk;
  p.cut = chunk < a.table_width;
  p.shares = (int)std::max<int64_t>((a.table_width + chunk - 1) / chunk, 1);
  const dim3 grid((unsigned)(a.batch * a.heads * p.shares));
  switch ((a.head_dim + 63) / 64) {
    case 1: hipLaunchKernelGGL((select_kernel<1>), grid, dim3(kThreads), 0, s, p); break;
    case 2: hipLaunchKernelGGL((select_kernel<2>), grid, dim3(kThreads), 0, s, p); break;
    case 3: hipLaunchKernelGGL((select_kernel<3>), grid, dim3(kThreads), 0, s, p); break;
    default: hipLaunchKernelGGL((select_kernel<4>), grid, dim3(kThreads), 0, s, p); break;
  }
  return hipGetLastError();
}

size_t kv_evict_workspace_bytes(const KvEvictLaunch& a) {
  return a.table_width <= kKeysInLds ? 0 : (size_t)a.batch * a.table_width * sizeof(u64);
}

hipError_t launch_kv_evict(const KvEvictLaunch& a, hipStream_t s) {
  EvictParams p;
  p.a = a;
  p.keys = static_cast<u64*>(a.ws);
  hipLaunchKernelGGL(evict_kernel, dim3((unsigned)a.batch), dim3(kEvictThreads), 0, s, p);
  return hipGetLastError();
}

}  // namespace nvfp4
