/*
 * linear.h — C ABI of linear attention with a decay for each head on GB300
 * (sm_103a): the chunked form for training and prompts, its backward pass, and
 * the recurrent step for single tokens.
 * Status codes, the stream handle and the device error-word bits are those of
 * attn.h, and every convention listed there holds here too (caller-owned
 * device pointers, no allocation, no host synchronization, every output element
 * written, a status other than ATTN_OK means nothing was enqueued), with one
 * difference: element offsets are 64-bit.
 */
#ifndef LINEAR_GB300_H
#define LINEAR_GB300_H

#include "attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Device error-word bits */
#define ATTN_DEVERR_DECAY 0x10 /* a log_decay is positive or NaN (taken as 0) */

/*
 * For every sequence and KV head, with l = exp(log_decay) <= 1 and the state S
 * [head_dim, head_dim] (rows: dims of the keys, columns: of the values),
 *   S_t = l S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t,
 * q of query head h meeting KV head h / (heads_q / heads_kv); S before the first
 * token is the sequence's initial state (zeros where none is given), S after the
 * last its final state.
 *
 * Layouts: q, o, dout, dq bf16 [tokens, heads_q, head_dim], k, v, dk, dv bf16
 * [tokens, heads_kv, head_dim], states fp32 [num_seqs, heads_kv, head_dim,
 * head_dim].  Sequence n occupies rows [cu_seqlens[n], cu_seqlens[n + 1])
 * (device int32 [num_seqs + 1], non-decreasing from 0, at most `tokens`; read on
 * the device only, so a captured graph may change it between replays), or, with
 * cu_seqlens NULL, rows [n seqlen, (n + 1) seqlen).  Rows at or past
 * cu_seqlens[num_seqs] are padding: outputs there are exact zeros, inputs there
 * do not affect any result.  A sequence may be empty.  A cu_seqlens that does not
 * begin with 0, decreases or passes `tokens` is flagged ATTN_DEVERR_SEQLEN; the rows of the
 * sequences concerned are unspecified, and no memory beside the outputs and the workspace is
 * written whatever it holds.
 *
 * q_stride .. dout_stride are the elements between two tokens' rows (0: dense,
 * heads * head_dim; else at least that and a multiple of 8), so that slices of one
 * fused projection can be passed; the heads of a token are dense, and so are all
 * outputs.
 *
 * log_decay is device fp32 [heads_kv], the natural logarithm of the decay: 0
 * keeps everything, -inf keeps only the present token.  It is a property of the
 * layer, not differentiated.
 *
 * No output, nor the workspace, may share memory with another argument (ATTN_ERR_INVALID_ARG).
 *
 * Supported: head_dim in {64, 128}; heads_q a multiple of heads_kv, at most 65535;
 * tokens * heads_q < 2^31, num_seqs * heads_q < 2^29.
 */
typedef struct {
  int num_seqs;
  int seqlen;   /* dense: tokens of a sequence, tokens = num_seqs * seqlen */
  int tokens;
  int heads_q;
  int heads_kv;
  int head_dim;
  float scale;
  int64_t q_stride;
  int64_t k_stride;
  int64_t v_stride;
  int64_t dout_stride; /* linear_attn_bwd */
  const int32_t* cu_seqlens;
  const float* log_decay;
  int32_t* error_word; /* optional device int32 */
} linear_attn_problem_t;

/* Bytes of device workspace (0 for an invalid problem, and where none is
 * needed): the fp32 states between the segments that long sequences are cut
 * into.  It holds nothing between calls; calls that may overlap on the GPU need
 * one each. */
size_t linear_attn_fwd_workspace_size(const linear_attn_problem_t* p);
size_t linear_attn_bwd_workspace_size(const linear_attn_problem_t* p);

/*
 * Forward.  initial_state and final_state may be NULL (zeros; not wanted).
 * The products run on bf16 operands with fp32 sums.  Within a chunk of 128 tokens
 * the decayed scores are rounded to bf16 (off by up to 2^-8 of each).  The state is kept in
 * fp32, and for the chunks behind either the keys times their decays or the
 * state that meets a chunk's rows is rounded so, the other held in two
 * terms (2^-17).  A state that is returned comes of keys in three terms (2^-25), its
 * error below that of a sum over the tokens in fp32.  Where no sequence can be longer
 * than 8 tokens (seqlen, or with cu_seqlens `tokens`) all is fp32 but o.
 * A value that is infinite or NaN reaches the rows that see it as either and, through
 * 0 * NaN, earlier rows of its chunk.
 * The result is bitwise reproducible on one device.
 */
attn_status_t linear_attn_fwd(const linear_attn_problem_t* p, const void* q, const void* k,
                              const void* v, const float* initial_state, void* o,
                              float* final_state, void* workspace, size_t workspace_bytes,
                              attn_stream_t stream);

/*
 * Backward, from q, k, v and dout = dL/do alone (o is not needed):
 *   dq_t = scale S_t dout_t,   D_t = l D_{t+1} + scale q_t dout_t^T (summed over the KV
 *   head's query heads),   dk_t = D_t v_t,   dv_t = D_t^T k_t,
 * D past the last token standing for dL/d(final state), dfinal_state (NULL: zeros),
 * which meets the last token undecayed; dL/d(initial state) = l D_first goes to
 * dinitial_state unless that is NULL.
 * Rounding as in the forward pass, the three terms where dinitial_state is wanted.
 * Bitwise reproducible.
 */
attn_status_t linear_attn_bwd(const linear_attn_problem_t* p, const void* q, const void* k,
                              const void* v, const void* dout, const float* initial_state,
                              const float* dfinal_state, void* dq, void* dk, void* dv,
                              float* dinitial_state, void* workspace, size_t workspace_bytes,
                              attn_stream_t stream);

/*
 * One new token for each of num_seqs sequences, whose states lie in a pool fp32
 * [num_slots, heads_kv, head_dim, head_dim]: sequence n's in slot slots[n] (device
 * int32 [num_seqs]; NULL: slot n).  The states are updated in place and o (bf16
 * [num_seqs, heads_q, head_dim]) is written, all in fp32 but for the rounding of
 * o; the decay is held in two fp32 terms, so that its error does not grow with the steps.  An infinite
 * or NaN element of a state stays one of either.  A slot of -1 marks a padding row: its o is zeros.  Slots outside
 * [-1, num_slots) and slots that an earlier sequence of the call has are flagged
 * ATTN_DEVERR_INDEX_RANGE; their rows of o are zeros and they touch no state.
 * Other slots are left as they are.  o and the states share no memory with another
 * argument (ATTN_ERR_INVALID_ARG).
 */
typedef struct {
  int num_seqs;
  int num_slots;
  int heads_q;
  int heads_kv;
  int head_dim; /* 64 or 128 */
  float scale;
  int64_t q_stride; /* as in linear_attn_problem_t */
  int64_t k_stride;
  int64_t v_stride;
  const int32_t* slots;
  const float* log_decay;
  int32_t* error_word; /* optional device int32 */
} linear_attn_step_t;

attn_status_t linear_attn_step(const linear_attn_step_t* p, const void* q, const void* k,
                               const void* v, float* state, void* o, attn_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LINEAR_GB300_H */
