/*
 * rotary.h — C ABI of the rotation by position (rotary position embedding) on
 * GB300 (sm_103a): the table of cosines and sines, scaled for long contexts, the
 * rotation of queries and keys, and its backward pass.
 * Status codes, the stream handle and the device error-word bits are those of
 * attn.h, and every convention listed there holds here too (caller-owned
 * device pointers, no allocation, no host synchronization, every output element
 * written, a status other than ATTN_OK means nothing was enqueued), with one
 * difference: element offsets are 64-bit.
 */
#ifndef ROTARY_GB300_H
#define ROTARY_GB300_H

#include "attn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  ATTN_ROTARY_NONE = 0,   /* f_a = base^(-2a / rot_dim) */
  ATTN_ROTARY_LINEAR = 1, /* f_a / factor: positions squeezed into the trained range */
  ATTN_ROTARY_BASE = 2,   /* the base times factor^(rot_dim / (rot_dim - 2)): the lowest
                             frequency divided by factor, the highest kept */
  ATTN_ROTARY_PARTS = 3   /* f_a (w + (1 - w) / factor) with w the ramp from 0 to 1 of the turns
                             original f_a / 2 pi between `slow` and `fast`: frequencies that turn
                             often over the trained range are kept, those that hardly turn are
                             divided (the "by parts" interpolation of B. Peng et al., "YaRN:
                             Efficient Context Window Extension", 2023, section 3.2) */
} attn_rotary_scaling_t;

/* The frequencies of a table.  rot_dim a multiple of 16 up to 256; base and
 * factor positive and finite; fast > slow (ATTN_ROTARY_PARTS). */
typedef struct {
  int max_position; /* rows of the table */
  int rot_dim;
  double base;
  int scaling;     /* attn_rotary_scaling_t */
  double factor;
  int original;    /* ATTN_ROTARY_PARTS: positions of the trained range */
  double fast;
  double slow;
  double magnitude; /* multiplies every cosine and sine; finite in fp32 */
} attn_rotary_table_t;

/* cos_sin fp32 [max_position, rot_dim]: row p holds magnitude cos(p f_a) for
 * a < rot_dim / 2, then magnitude sin(p f_a).  The table that attn_rotary_fwd and
 * attn_cache_append read.  An angle is a product of integers modulo one turn, so
 * its error is p 2^-65 turns beside p times that of f_a / 2 pi in fp64, at any
 * position.  Its cosine and sine are summed in fp32: an entry is off by up to 6 2^-24
 * magnitude, in the mean square 1.1 to 1.3 times what one rounding to fp32 is. */
attn_status_t attn_rotary_table(const attn_rotary_table_t* t, float* cos_sin, attn_stream_t stream);

/*
 * Rows to rotate: q bf16 [tokens, heads_q, head_dim] and k bf16 [tokens, heads_k,
 * head_dim] (k may be NULL, with k_out).  q_stride and k_stride are the elements
 * between two tokens' rows (0: dense; else at least heads * head_dim and a
 * multiple of 8), so that slices of a fused projection can be passed; the heads
 * of a token are dense.  The outputs are dense and may be the inputs where those
 * are dense; else they share no memory with another argument or with each other
 * (ATTN_ERR_INVALID_ARG).
 *
 * A token's position: positions[t] where `positions` is given (device int32
 * [tokens]; -1 marks a padding row); else its place in its sequence of the THD
 * packing (cu_seqlens device int32 [num_seqs + 1], rows at or past
 * cu_seqlens[num_seqs] are padding); else t mod seqlen.  Padding rows of the
 * outputs are zeros.  A position outside [0, max_position) is flagged
 * ATTN_DEVERR_INDEX_RANGE (given positions) or ATTN_DEVERR_SEQLEN and its rows are
 * zeros.
 *
 * Supported: head_dim a multiple of 8 up to 1024; rot_dim a multiple of 16 up to
 * 256, rot_offset a multiple of 8, rot_offset + rot_dim <= head_dim;
 * tokens * (heads_q + heads_k) * head_dim < 2^40.
 */
typedef struct {
  int tokens;
  int heads_q;
  int heads_k;
  int head_dim;
  int rot_dim;
  int rot_offset;   /* the first rotated dim */
  int interleaved;  /* pairs (2a, 2a + 1) instead of (a, a + rot_dim / 2) */
  int max_position; /* rows of cos_sin */
  int seqlen;       /* dense: tokens of a sequence */
  int num_seqs;     /* THD */
  int64_t q_stride;
  int64_t k_stride;
  const int32_t* cu_seqlens;
  const int32_t* positions;
  int32_t* error_word; /* optional device int32 */
} attn_rotary_problem_t;

/* With c = cos_sin[pos, a] and s = cos_sin[pos, rot_dim / 2 + a], pair a = (x, y)
 * becomes (x c - y s, y c + x s), in fp32 with each product and sum rounded once,
 * then rounded to bf16; the other dims are copied. */
attn_status_t attn_rotary_fwd(const attn_rotary_problem_t* p, const void* q, const void* k,
                              const float* cos_sin, void* q_out, void* k_out, attn_stream_t stream);

/* Backward: the gradients dq, dk of the rotated rows become those of the rows,
 * (x c + y s, y c - x s); the arguments are those of attn_rotary_fwd. */
attn_status_t attn_rotary_bwd(const attn_rotary_problem_t* p, const void* dq, const void* dk,
                              const float* cos_sin, void* dq_out, void* dk_out,
                              attn_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* ROTARY_GB300_H */
