/*
 * nvfp4_attn.h -- the attention side of a decode layer on AMD Instinct MI355X (gfx950):
 * rotary positions, a quantised paged key-value cache, and attention of one
 * new token per sequence over that cache.
 *
 * Part of libnvfp4.so; the conventions of nvfp4.h hold for every call here:
 * device pointers unless marked (host), the caller owns all memory, `stream` is
 * a hipStream_t, arguments are validated on the host before anything is
 * enqueued, statuses and nvfp4_last_error() as there, results bit-identical
 * from call to call.  These calls stand between the layer's QKV product and its
 * O product: nvfp4_kv_append() takes the QKV rows as nvfp4_gemv / nvfp4_gemm
 * write them, nvfp4_attn_decode() writes the rows that the O product reads.
 *
 * Activations are fp32 or bf16 rows, one per token, of `heads` heads of
 * head_dim elements; consecutive tokens are a leading dimension (in elements, a
 * multiple of 8) apart, so a row may be part of a wider one (the q, k and v of
 * a fused QKV row).  head_dim is a multiple of 16, at most 256.  Row data is
 * 16-byte aligned, positions, lengths and page tables 4-byte, slots and
 * frequency tables 8-byte.
 */
#ifndef NVFP4_ATTN_H_
#define NVFP4_ATTN_H_

#include "nvfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- rotary positions -----------------------------------------------------
 * Pair i of a head (i < rot_dim / 2) is turned by pos * f_i turns:
 *   (a, b) -> magnitude * (a cos t - b sin t, a sin t + b cos t),  t = 2 pi pos f_i.
 * NVFP4_ROPE_HALF pairs elements (i, i + rot_dim/2), NVFP4_ROPE_INTERLEAVED pairs
 * (2i, 2i + 1).  Elements from rot_dim on are copied unchanged.  rot_dim is a
 * multiple of 16, 0 <= rot_dim <= head_dim.
 *
 * The table holds f_i as a 64-bit fixed-point fraction of a turn (f_i * 2^64,
 * modulo one turn), so that pos * f_i is reduced modulo one turn exactly for every
 * 32-bit position: far positions lose nothing.  nvfp4_rope_freqs() fills one;
 * any other scaling is a table of the caller's own.
 */
typedef enum nvfp4_rope_layout {
  NVFP4_ROPE_HALF = 0,
  NVFP4_ROPE_INTERLEAVED = 1
} nvfp4_rope_layout;

typedef enum nvfp4_rope_scaling {
  NVFP4_ROPE_NONE = 0,      /* f_i = base^(-2i / rot_dim) / (2 pi) */
  NVFP4_ROPE_LINEAR = 1,    /* f_i / factor */
  NVFP4_ROPE_YARN = 2       /* the Ignis README's long contexts: f_i kept for pairs that turn more than
                               beta_fast times over original_max positions, f_i / factor for those under
                               beta_slow turns, a linear ramp over the pair index between (its ends
                               rounded outwards to whole pairs, within [0, rot_dim - 1]);
                               magnitude = 0.1 ln(factor) + 1 */
} nvfp4_rope_scaling;

typedef struct nvfp4_rope_config {
  int64_t rot_dim;          /* multiple of 16, 0..256 */
  double base;              /* > 1 */
  int scaling;              /* nvfp4_rope_scaling */
  double factor;            /* >= 1 (linear, YaRN) */
  double original_max;      /* > 0 (YaRN) */
  double beta_fast;         /* YaRN: > beta_slow */
  double beta_slow;         /* YaRN: > 0 */
} nvfp4_rope_config;

/* (host) Fills freqs (host memory, rot_dim / 2 entries; copy it to the device
 * once) and *magnitude (1 unless YaRN). */
int nvfp4_rope_freqs(const nvfp4_rope_config* config /* host */, uint64_t* freqs /* host */,
                     float* magnitude /* host */);

/* Turns every head of `tokens` rows; one rounding, to y_dtype.  y == x turns in
 * place (same dtype and leading dimension; any other overlap of x and y is not
 * allowed).  inverse != 0 turns by -t: the inverse at magnitude 1, and at any
 * magnitude the gradient (dx from dy).  tokens == 0 or heads == 0 is a no-op. */
typedef struct nvfp4_rope_args {
  int64_t tokens, heads, head_dim, rot_dim;
  int layout;               /* nvfp4_rope_layout */
  int inverse;
  float magnitude;
  const int32_t* positions; /* [tokens], any 32-bit value */
  const uint64_t* freqs;    /* [rot_dim / 2] */
  const void* x;            /* [tokens][ldx], heads * head_dim used */
  int x_dtype;
  int64_t ldx;
  void* y;                  /* [tokens][ldy] */
  int y_dtype;
  int64_t ldy;
} nvfp4_rope_args;

int nvfp4_rope(const nvfp4_rope_args* args /* host */, void* stream);

/* ---- the paged key-value cache -----------------------------------------------
 * A pool of `pages` pages, each holding the keys and values of page_size tokens
 * (a multiple of 16) for all kv_heads heads.  A token's place is its slot,
 * page * page_size + offset.  The bytes' order inside the pool is private to the
 * library (a gfx950 tile layout); nvfp4_kv_append() writes it, nvfp4_kv_read()
 * and nvfp4_attn_decode() read it.  The pool needs no initial contents.
 *
 * Formats, for the head_dim values v of one token and head (k and v alike):
 *   NVFP4_KV_BF16   bf16, rounded to nearest even (2 bytes a value);
 *   NVFP4_KV_E4M3   codes e4m3(v / X) with X the smallest power of two for which
 *                   the largest |v| / X is at most 448, its exponent at least
 *                   -110 (-110 for a zero row) (1 byte a value + 1 a row); codes that
 *                   would stand for 2^128 saturate at the largest finite, 1.875 *
 *                   2^127.  A row with an infinity or NaN reads back as NaN throughout;
 *   NVFP4_KV_NVFP4  nvfp4_quantize()'s rule with the tensor scale given (k_scale,
 *                   v_scale): per 16 values a scale E4M3FN nearest to
 *                   amax / (6 s_t), codes E2M1 nearest to |v| / (e4m3(scale) s_t)
 *                   (0.5625 bytes a value).  A block with an infinity or NaN
 *                   reads back as NaN.
 * All roundings are to nearest, ties to even, saturating at 448 and 6; every
 * quotient and product is a single-precision operation.
 */
typedef enum nvfp4_kv_format {
  NVFP4_KV_BF16 = 0,
  NVFP4_KV_E4M3 = 1,
  NVFP4_KV_NVFP4 = 2
} nvfp4_kv_format;

typedef struct nvfp4_kv_cache {
  void* pool;               /* nvfp4_kv_cache_bytes() bytes, 16-byte aligned */
  int64_t pages;            /* >= 1; pages * page_size * kv_heads <= 2^34 */
  int64_t page_size;        /* multiple of 16, <= 65536 */
  int64_t kv_heads;         /* 1..1024 */
  int64_t head_dim;         /* multiple of 16, 16..256 */
  int format;               /* nvfp4_kv_format */
  float k_scale, v_scale;   /* tensor scales, 2^-64 .. 2^64; 1 unless NVFP4_KV_NVFP4 */
} nvfp4_kv_cache;

/* (host) *bytes = size of the pool (cache->pool is not looked at). */
int nvfp4_kv_cache_bytes(const nvfp4_kv_cache* cache /* host */, size_t* bytes /* host */);

/* Writes the keys and values of `tokens` tokens into their slots.  With freqs
 * given (not NULL), k is turned first (in fp32, with no rounding before the
 * format's own), and with q given too, q is turned into q_out (bf16): one launch
 * for all that stands between the QKV product and the attention.  A token whose
 * slot is outside [0, pages * page_size) is skipped: nothing of it is read,
 * neither the cache nor its row of q_out is written (rows that only pad a
 * batch: slot -1).  Other slots must be distinct: of two tokens with one slot,
 * either's bytes may end up there, mixed.  tokens == 0 is a no-op. */
typedef struct nvfp4_kv_append_args {
  const nvfp4_kv_cache* cache;  /* host */
  int64_t tokens;
  const int64_t* slots;     /* [tokens] */
  const void* k;            /* [tokens][ldk], kv_heads * head_dim used */
  const void* v;            /* [tokens][ldv] */
  int dtype;                /* of k, v and q: NVFP4_F32 or NVFP4_BF16 */
  int64_t ldk, ldv;
  /* optional rotary positions (freqs NULL: none) */
  const uint64_t* freqs;    /* [rot_dim / 2] */
  const int32_t* positions; /* [tokens] */
  int64_t rot_dim;
  int layout;
  float magnitude;
  /* optional queries (q NULL: none); need freqs */
  int64_t q_heads;
  const void* q;            /* [tokens][ldq], q_heads * head_dim used */
  int64_t ldq;
  uint16_t* q_out;          /* bf16 [tokens][ldqo]; may be q itself if q is bf16 and ldqo == ldq */
  int64_t ldqo;
} nvfp4_kv_append_args;

int nvfp4_kv_append(const nvfp4_kv_append_args* args /* host */, void* stream);

/* Reads back the values that the cache holds for `tokens` slots:
 * k_out [tokens][ldk], v_out [tokens][ldv] of kv_heads * head_dim, out_dtype
 * (one rounding).  Either may be NULL.  Rows of slots outside the pool are left
 * as they were.  The same slot may be read more than once. */
int nvfp4_kv_read(const nvfp4_kv_cache* cache /* host */, const int64_t* slots, int64_t tokens, void* k_out,
                  int64_t ldk, void* v_out, int64_t ldv, int out_dtype, void* stream);

/* ---- attention of one new token per sequence over the cache -------------------
 * For sequence b of length n_b = seq_lens[b] (clamped to [0, table_width *
 * page_size]; it counts the new token, already appended) and query head h, with
 * kv head h / (q_heads / kv_heads):
 *   s_j = scale * q . k_j   over max(0, n_b - window) <= j < n_b (window 0: all),
 *   o   = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),   m = max_j s_j,
 *   lse = m + ln sum_j exp(s_j - m).
 * Token j of sequence b lies in page page_table[b * table_width + j / page_size].
 * A page id outside [0, pages) holds nothing: its tokens are left out of the sums
 * (an evicted page: -1).  A row left with no token, or only with scores of -inf,
 * gives zeros and lse = -inf.  Table entries past a sequence's last page are not
 * looked at, cache slots past its length have no effect whatever they hold.
 * Infinities and NaN that a row attends to act as in the formulas: a query's or
 * key's make the scores that they enter infinite or NaN (a product with zero), and
 * so do scores past fp32's range; a token of score -inf weighs nothing, one of
 * score +inf or NaN makes its query head's row and lse NaN.  A value's make the
 * outputs that they enter infinite or NaN, even where the token weighs nothing.
 * Several rows may share pages: a few new tokens of one sequence are rows with
 * the same table and lengths n, n + 1, ...  Each row, and each sixteen query heads
 * of one kv head, reads its cache by itself.
 *
 * Scores, maxima, sums and outputs are held in fp32.  The exp() terms enter the
 * matrix cores rounded to within 2^-17 of each (bf16 and E4M3 caches: the sum of
 * two bf16 numbers) or 2^-11 (NVFP4: one f16 number, an eighth of the rounding
 * of o to bf16; a term below 2^-25 of the row's largest to within 2^-36 of that);
 * their sum takes them whole.  No term of a bf16 or E4M3 cache is above 1: sums
 * over n tokens stay finite for values up to 2^127 / n.  Its terms keep those
 * 2^-17 down to 2^-100 of the row's largest.
 * o is bf16, rounded once; out overlaps no input.  The work is split evenly over the GPU along all
 * sequences' lengths, whatever their mix, and joined in a fixed order.
 *
 * One call takes up to 2^31 tiles of 32 tokens, counted over all sequences, kv
 * heads and sixteens of a kv head's query heads, each at the longest length that
 * the table (or the window) allows, plus a few for each; more is refused.
 *
 * The workspace's first NVFP4_ATTN_COUNTER_BYTES must be zero before its first
 * use; every call leaves them zero.  Calls that share one must not overlap.
 * One workspace may serve the attentions and selections of nvfp4_attn_long.h too,
 * its first NVFP4_SELECT_COUNTER_BYTES zero before its first use; those of nvfp4.h
 * are laid out otherwise and apart from it.
 * batch == 0 is a no-op.
 */
#define NVFP4_ATTN_COUNTER_BYTES 1024

typedef struct nvfp4_attn_args {
  const nvfp4_kv_cache* cache;  /* host */
  int64_t batch;            /* 0..65536 */
  int64_t q_heads;          /* multiple of kv_heads */
  const uint16_t* q;        /* bf16 [batch][ldq] */
  int64_t ldq;
  const int32_t* page_table;/* [batch][table_width] */
  int64_t table_width;      /* >= 0; table_width * page_size <= 2^30 */
  const int32_t* seq_lens;  /* [batch] */
  float scale;              /* > 0, at most 2^127 */
  int64_t window;           /* >= 0; 0: none */
  uint16_t* out;            /* bf16 [batch][ldo] */
  int64_t ldo;
  float* lse;               /* optional, fp32 [batch][q_heads] */
  void* workspace;
  size_t workspace_bytes;
} nvfp4_attn_args;

/* (host) Depends on batch, q_heads, table_width, window and the cache's shape and format only. */
int nvfp4_attn_decode_workspace_bytes(const nvfp4_attn_args* args /* host */, size_t* bytes /* host */);
int nvfp4_attn_decode(const nvfp4_attn_args* args /* host */, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* NVFP4_ATTN_H_ */
