/*
 * cache.h — C ABI of the paged key/value cache on GB300 (sm_103a): appending the
 * keys and values of new tokens (with the position rotation applied on the
 * way), and the attention of new queries over the cached keys.
 * Status codes, the stream handle and the device error-word bits are those of
 * attn.h, and every convention listed there holds here too (caller-owned
 * device pointers, no allocation, no host synchronization, every output element
 * written, a status other than ATTN_OK means nothing was enqueued), with one
 * difference: element offsets inside the cache are 64-bit.
 */
#ifndef CACHE_GB300_H
#define CACHE_GB300_H

#include "attn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  ATTN_CACHE_BF16 = 0, /* keys and values as bf16 */
  ATTN_CACHE_E4M3 = 1  /* as 8-bit e4m3 codes, one fp32 scale per (page, KV head) */
} attn_cache_type_t;

/*
 * A step over a paged cache.
 *
 * The cache: k_cache and v_cache are pools [num_pages, heads_kv, page_size,
 * head_dim] of bf16 or e4m3; an e4m3 pool comes with k_scale and v_scale, fp32
 * [num_pages, heads_kv] (positive, finite and not subnormal; attn_cache_append
 * writes powers of two), and a code c stands for c * scale.  Sequence n's key j
 * lies in row j % page_size of page page_table[n, j / page_size]; page_table is
 * int32 [num_seqs, max_pages].  Sequences may share pages that no call appends
 * to.  Rows and pages that no sequence's length reaches may hold anything.
 *
 * The step's tokens: q, k, v are bf16 [tokens, heads, head_dim], sequence n's
 * new tokens are rows [cu_seqlens[n], cu_seqlens[n + 1]) (the THD packing of
 * attn.h; rows at or past cu_seqlens[num_seqs] are padding), and
 * seqlens_kv[n] is the sequence's length INCLUDING them: its new token i, of m,
 * has position seqlens_kv[n] - m + i.  cu_seqlens [num_seqs + 1], seqlens_kv
 * [num_seqs] and page_table are device memory and never read by the host, so a
 * captured graph may change them between replays.  max_new bounds the new
 * tokens of every sequence.  With tokens = 0 both calls do nothing, and the
 * pointers of rows (q, k, v, q_out, o, lse) and the workspace may be NULL.
 *
 * q_stride, k_stride and v_stride are the elements between two tokens' rows
 * (0: dense, heads * head_dim; else at least that and a multiple of 8), so that
 * slices of one fused projection can be passed; the heads of a token are dense.
 *
 * Supported: head_dim in {64, 128}; page_size in {16, 32, 64, 128}; heads_q a
 * multiple of heads_kv; num_pages * heads_kv * page_size < 2^31.
 *
 * Problems only the device sees are OR-ed into error_word: a page_table entry
 * outside [0, num_pages) (ATTN_DEVERR_INDEX_RANGE; keys there are not written
 * and not attended), a sequence longer than max_pages * page_size, with more
 * than max_new new tokens, with more new tokens than its length, or with
 * rotated positions at or past max_position (ATTN_DEVERR_SEQLEN; see each
 * call for what it does with it).
 */
typedef struct {
  int num_seqs;
  int tokens;       /* rows of q, k, v, q_out, o */
  int heads_q;
  int heads_kv;
  int head_dim;
  int cache_type;   /* attn_cache_type_t */
  int page_size;
  int num_pages;
  int max_pages;    /* columns of page_table */
  int max_new;
  int causal;       /* attn_cache_fwd */
  float scale;      /* attn_cache_fwd: multiplies the logits */
  int rot_dim;          /* attn_cache_append: rotated leading dims, 0 = none */
  int rot_interleaved;  /* pairs (2a, 2a + 1) instead of (a, a + rot_dim / 2) */
  int max_position;     /* rows of cos_sin */
  int64_t q_stride;
  int64_t k_stride;
  int64_t v_stride;
  const int32_t* cu_seqlens;
  const int32_t* seqlens_kv;
  const int32_t* page_table;
  int32_t* error_word; /* optional device int32 */
} attn_cache_problem_t;

/*
 * Append: writes the step's keys and values into the cache, and the rotated
 * queries to q_out (bf16 [tokens, heads_q, head_dim], dense; padding rows
 * exact zeros).  q and q_out may both be NULL; they may be the same dense
 * buffer.
 *
 * Rotation of q and k (rot_dim > 0; a multiple of 16, at most head_dim): with
 * c = cos_sin[pos, a] and s = cos_sin[pos, rot_dim / 2 + a] (fp32
 * [max_position, rot_dim], the table the caller's model uses), pair a = (x, y)
 * becomes (x c - y s, y c + x s), in fp32 with each product and sum rounded
 * once; dims at or past rot_dim and the values are not rotated.
 *
 * bf16: rounded once.  e4m3: the scale is a power of two, 2^e with the least
 * integer e >= -100 for which the largest finite magnitude that this call
 * brings to the (page, head) is at most 448 * 2^e.  A page that already holds
 * earlier keys of the sequence keeps the larger of its scale and this one; when
 * it grew, the earlier codes are rounded again under the new scale (exact
 * except for codes that become subnormal).  A power of two costs an e4m3 code
 * no precision and makes that second rounding exact almost always, so the
 * cache hardly depends on how a text was cut into calls.  Infinities are
 * stored as the largest code, NaN as NaN.
 *
 * Only the rows of the new tokens are written (and, where a scale grew, the
 * earlier rows of that page and head).  Tokens with a bad page or beyond the
 * limits above are skipped, flagged, and get a zero q_out row when they have
 * no position.  Two sequences must not append to the same page.
 */
attn_status_t attn_cache_append(const attn_cache_problem_t* p, const void* q, const void* k,
                                const void* v, const float* cos_sin, void* q_out, void* k_cache,
                                void* v_cache, float* k_scale, float* v_scale,
                                attn_stream_t stream);

/* Bytes of device workspace of attn_cache_fwd (0 for an invalid problem): the
 * fp32 partial results of the key ranges that one sequence and head was cut
 * into.  It holds nothing between calls; calls that may overlap on the GPU
 * (two streams, two graphs replayed at once) need one each. */
size_t attn_cache_fwd_workspace_size(const attn_cache_problem_t* p);

/*
 * Attention of the step's queries over the cache: for token i of sequence n
 * and query head h (KV head h / (heads_q / heads_kv)),
 *   o = sum_j softmax_j(scale <q, k_j>) v_j,  lse = ln sum_j exp(scale <q, k_j>)
 * over the keys j < seqlens_kv[n], and j <= position(i) when causal.  q bf16
 * [tokens, heads_q, head_dim] (already rotated), o bf16 dense, lse fp32
 * [heads_q, tokens].  A row without a visible key, and the padding rows, get
 * o = 0 and lse = -inf.  Keys past a sequence's length, in rows of a page that
 * was never written, do not affect any result whatever they hold.
 * A key that is infinite or NaN reaches the rows that see it; a value that is,
 * through 0 * NaN, also rows of its sequence in the same call that causality
 * keeps from it.
 * P is rounded before the product with V: bf16 caches, to bf16 (within 2^-8 of it)
 * by the kernel for many query rows per KV head and to a sum of two bf16 (2^-16) by
 * that for few; e4m3 caches, times the scale of its value's page, to fp16 (within
 * 2^-11 of it, or within 2^-33 of the largest P times scale of the keys that the row
 * sees).  Which kernel serves a call follows from the problem alone: a row of a bf16
 * cache is held to 2^-16 in a batch of sequences with few new tokens, and to 2^-8
 * where a prompt's chunk shares the call.
 * Over an e4m3 cache q is held in fp16 times a power of two for each row: exact for
 * elements of at least 2^-31 of the row's largest, off by 2^-39 of that below.  The
 * kernel for many rows expects logits of such a cache below 2^25 in magnitude.
 * Any number of new tokens per sequence, one included; sequences of different
 * kinds may share a call.  The result is bitwise reproducible on one device.
 */
attn_status_t attn_cache_fwd(const attn_cache_problem_t* p, const void* q, const void* k_cache,
                             const void* v_cache, const float* k_scale, const float* v_scale,
                             void* o, float* lse, void* workspace, size_t workspace_bytes,
                             attn_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* CACHE_GB300_H */
