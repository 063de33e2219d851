/*
 * nvfp4_attn_long.h -- reading less of a long key-value cache on AMD Instinct MI355X (gfx950):
 * attention of a batch over a prefix that all its sequences share, attention over the pages that a
 * cheap score selects, and eviction of pages by the attention weight that they have had.
 *
 * Part of libnvfp4.so, beside nvfp4_attn.h: the same cache, page tables, conventions and results as
 * nvfp4_attn_decode(), whose documentation of formulas, precision, infinities, limits and
 * workspaces holds for every attention here but for what is said below.
 */
#ifndef NVFP4_ATTN_LONG_H_
#define NVFP4_ATTN_LONG_H_

#include "nvfp4_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- a prefix that all sequences share ------------------------------------------
 * Sequence b attends to the prefix's tokens, then to its own:
 *   s_j = scale * q . k_j   over the first n = *prefix_len tokens of prefix_table (clamped to
 *                           [0, prefix_width * page_size]) and the first seq_lens[b] of its own table,
 * with o and lse as nvfp4_attn_decode() defines them over both.  attn.page_table and attn.seq_lens count
 * the own tokens alone: the first of them starts a page.  The prefix is read once for all sequences
 * (by each, in one launch, where its table holds little).
 * A sequence whose length is below 0 is a free place of the batch: it attends to nothing, not to the
 * prefix either, and its row is zeros with lse = -inf.  attn.window must be 0.  Prefix pages outside
 * [0, pages) hold nothing.  The prefix's pages may be anyone's, a sequence's own among them.
 *
 * In one call batch * q_heads is at most 2^30, and the prefix's tiles of 32 tokens, counted for every kv head
 * and 16 or 32 rows of batch * q_heads / kv_heads, fewer than 2^31 at the longest prefix that its table allows.
 */
typedef struct nvfp4_attn_shared_args {
  nvfp4_attn_args attn;
  const int32_t* prefix_table;  /* [prefix_width] */
  int64_t prefix_width;         /* >= 0; prefix_width * page_size <= 2^30 */
  const int32_t* prefix_len;    /* one number */
} nvfp4_attn_shared_args;

/* (host) Depends on attn's shapes as nvfp4_attn_decode_workspace_bytes() does, and on prefix_width. */
int nvfp4_attn_shared_workspace_bytes(const nvfp4_attn_shared_args* args /* host */, size_t* bytes /* host */);
int nvfp4_attn_shared(const nvfp4_attn_shared_args* args /* host */, void* stream);

/* ---- attention over selected pages ---------------------------------------------------
 * nvfp4_kv_bounds(): bounds[page][kv head][0][d] and [1][d], the smallest and the largest value of channel d
 * among the keys of the page's page_size tokens, for the n pages listed (those outside [0, pages) are skipped; a
 * page may be listed twice).  In bf16, exact: the cache's values, divided by k_scale.  A channel with a NaN has NaN
 * in both.  A page's bounds mean something once all its places are written; kv_select() needs
 * them of every page of a sequence but its last, so that they are formed when a page is full.
 */
int nvfp4_kv_bounds(const nvfp4_kv_cache* cache /* host */, const int32_t* pages, int64_t n /* 0..2^24; n * kv_heads at most 2^32 */,
                    uint16_t* bounds /* bf16 [cache->pages][kv_heads][2][head_dim], 16-byte aligned */, void* stream);

/* nvfp4_kv_select(): of the N = ceil(n_b / page_size) pages of sequence b (n_b = seq_lens[b], clamped to
 * [0, table_width * page_size]) the last one and, of the others, the budget - 1 with the highest scores
 *   score(i) = max over the kv head's query heads of sum_d max(q_d lo_d, q_d hi_d),
 * an upper bound of q . k over the page; all of them if they are no more.  Scores are formed in fp64 and ties go to the
 * earlier page; a NaN ranks above everything.  Pages outside [0, pages) are not there: never selected,
 * but for the last one, which is given as -1.
 * pages_out[b][kv head] lists the selected pages' ids in the sequence's order, then -1; lens_out[b] is the
 * length that goes with them, the same for every kv head: all selected pages are full but the last.  So
 * nvfp4_attn_decode_heads() over pages_out and lens_out is attention over the selected pages. */
typedef struct nvfp4_kv_select_args {
  const nvfp4_kv_cache* cache;  /* host; its pool is not looked at */
  int64_t batch;            /* 0..65536; batch * kv_heads at most 2^23 */
  int64_t q_heads;          /* multiple of kv_heads */
  const uint16_t* q;        /* bf16 [batch][ldq], 16-byte aligned */
  int64_t ldq;
  const uint16_t* bounds;   /* bf16 [cache->pages][kv_heads][2][head_dim], 16-byte aligned */
  const int32_t* page_table;/* [batch][table_width] */
  int64_t table_width;      /* >= 0; table_width * page_size <= 2^30 */
  const int32_t* seq_lens;  /* [batch] */
  int64_t budget;           /* >= 1; budget * page_size <= 2^30 */
  int32_t* pages_out;       /* [batch][kv_heads][budget] */
  int32_t* lens_out;        /* [batch] */
  void* workspace;          /* 16-byte aligned; its first NVFP4_SELECT_COUNTER_BYTES zero before its first use, and left zero by
                             * every call and by every attention: one workspace may serve both */
  size_t workspace_bytes;
} nvfp4_kv_select_args;
#define NVFP4_SELECT_COUNTER_BYTES 4096

/* (host) Depends on batch, table_width, budget and the cache's kv_heads. */
int nvfp4_kv_select_workspace_bytes(const nvfp4_kv_select_args* args /* host */, size_t* bytes /* host */);
int nvfp4_kv_select(const nvfp4_kv_select_args* args /* host */, void* stream);

/* nvfp4_attn_decode() with a page table for each kv head: page_table is [batch][kv_heads][table_width].
 * Workspace: nvfp4_attn_decode_workspace_bytes(). */
int nvfp4_attn_decode_heads(const nvfp4_attn_args* args /* host */, void* stream);

/* ---- the weight that pages have had, and eviction by it --------------------------------
 * nvfp4_attn_weigh() is nvfp4_attn_decode() and, in the same pass over the cache,
 *   weights_out[b][h][i] = decay * weights[b][h][i] + sum exp(s_j - lse)
 * over the query heads of kv head h and the tokens j of page i that they attend to, for all i < table_width: a page's
 * share of what its readers looked at, each query head adding up to 1.  Terms and sums are fp32, as
 * the attention's are.  A score, d products summed in fp32, is off by up to e_j = (d + 4) 2^-24 scale sum |q_c k_jc|, so that a
 * share is off by up to e_j + max e of itself; beyond that, whatever the scores' size, by (n + 64 + page_size / 16) 2^-24 of
 * its query head's 1 (n: the tokens that it attends to).  A query head whose lse is -inf adds nothing, one whose lse is NaN makes
 * the pages NaN that it attends to, but for those whose terms are all 0.  decay 0: weights is not read and may be NULL.  weights_out may
 * be weights.  q_heads, batch and table as in nvfp4_attn_decode(), and batch * kv_heads * table_width at most 2^31. */
typedef struct nvfp4_attn_weigh_args {
  nvfp4_attn_args attn;
  const float* weights;     /* [batch][kv_heads][table_width] */
  float decay;              /* finite, >= 0 */
  float* weights_out;       /* [batch][kv_heads][table_width] */
} nvfp4_attn_weigh_args;

/* (host) As nvfp4_attn_decode_workspace_bytes(). */
int nvfp4_attn_weigh_workspace_bytes(const nvfp4_attn_weigh_args* args /* host */, size_t* bytes /* host */);
int nvfp4_attn_weigh(const nvfp4_attn_weigh_args* args /* host */, void* stream);

/* nvfp4_kv_evict(): keeps up to `budget` of the N = ceil(n_b / page_size) pages of each sequence: first the last
 * `recent` places' pages, the newest first; then those of the first `sink` places; then the others by their
 * weights' sum over the kv heads (formed in fp64), the heaviest first, ties to the earlier page, NaN above everything.
 * Entries below 0 hold nothing: they are dropped from the table, but for the sequence's last one.
 *   table_out[b]    the kept pages' ids in the sequence's order, then -1;
 *   lens_out[b]     the length that goes with them: all are full but the last;
 *   weights_out     the kept pages' weights at their new places, then 0 (or NULL);
 *   freed[b]        the ids of the pages dropped, in order, then -1 (or NULL).
 * Keys keep the rotary positions that they were turned by.  The outputs overlap no input.  The workspace needs no
 * initial contents; what was zero of its first NVFP4_SELECT_COUNTER_BYTES is so again after the call: an attention's or a
 * selection's workspace may serve. */
typedef struct nvfp4_kv_evict_args {
  int64_t batch;            /* 0..65536 */
  int64_t kv_heads;         /* 1..1024 */
  int64_t page_size;        /* multiple of 16, 16..65536 */
  const float* weights;     /* [batch][kv_heads][table_width] */
  const int32_t* page_table;/* [batch][table_width] */
  int64_t table_width;      /* >= 0; table_width * page_size <= 2^30 */
  const int32_t* seq_lens;  /* [batch] */
  int64_t budget;           /* >= 1; budget * page_size <= 2^30 */
  int64_t sink;             /* >= 0 */
  int64_t recent;           /* >= 1 */
  int32_t* table_out;       /* [batch][budget] */
  int32_t* lens_out;        /* [batch] */
  float* weights_out;       /* [batch][kv_heads][budget], or NULL */
  int32_t* freed;           /* [batch][table_width], or NULL */
  void* workspace;          /* 16-byte aligned */
  size_t workspace_bytes;
} nvfp4_kv_evict_args;

/* (host) Depends on batch and table_width. */
int nvfp4_kv_evict_workspace_bytes(const nvfp4_kv_evict_args* args /* host */, size_t* bytes /* host */);
int nvfp4_kv_evict(const nvfp4_kv_evict_args* args /* host */, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* NVFP4_ATTN_LONG_H_ */
