/*
 * mfl_attention.h — C ABI of attention: the back-to-back GEMM of
 * mfl_chain.h with the softmax between its products, for packed sequences
 * with grouped heads, its gradients, and its form for decoding behind a
 * shared prefix.
 *
 * For query token t and query head h of a sequence with lq query tokens and
 * lk keys, kv head g = h / (heads_q / heads_kv):
 *
 *   s_j   = scale * sum_d q(t, h, d) k(j, g, d)        over the visible keys j
 *   lse   = log sum_j exp(s_j)
 *   out_d = sum_j exp(s_j - lse) v(j, g, d)
 *
 * causal: t sees keys j <= t + lk - lq (both counted from 0 in the sequence:
 * the last query token sees every key); otherwise every key of the sequence.
 * A query that sees no key has out = 0 and lse = -infinity.
 *
 * Types.  Inputs, out and gradients are all MFL_F16 or all MFL_BF16.  Scores,
 * maxima, sums and accumulators are fp32; the weights are rounded once (to
 * nearest even) to the input type as the second product's operand, results
 * once at the end.  lse is fp32.
 *
 * Addressing (elements): x(t, h, d) = X[t * x_token + h * x_head + d].  Every
 * pointer is 16-byte aligned and every stride a multiple of 8 (else
 * MFL_E_MISALIGNED); strides are not negative (MFL_E_LEADING_DIM), 0 lets an
 * input be shared, and those between tokens are at most 2^23 (q, k, v, dout,
 * and the prefix; MFL_E_TOO_LARGE).  No two elements of an output share an
 * address (MFL_E_ALIAS).
 * head_dim is a multiple of 8 up to 256 (else MFL_E_UNSUPPORTED).
 *
 * Sizes.  total_q * heads_q (batch * q_tokens * heads_q) is below 2^31 - 2^16,
 * and no launch has 2^24 workgroups or more (else MFL_E_TOO_LARGE, before
 * anything is launched): FLAT takes one per kv head, split and 16 rows (a
 * sequence's last ones may be fewer), TALL and dQ per 128 rows, dK and dV per
 * 128 or 256 keys, joining splits per 8 rows of a tile and per 4
 * rows of the prefix form.
 *
 * Packed sequences.  seq_q and seq_k hold batch + 1 offsets each in device
 * memory, the first of them 0, growing: sequence s owns query tokens
 * seq_q[s] .. seq_q[s+1] - 1 and keys seq_k[s] .. seq_k[s+1] - 1; lengths of
 * 0 are allowed.  Both NULL: one sequence.  The offsets are read by the
 * kernels and held inside [0, total_q] and [0, total_k] whatever they are.
 * Query tokens behind the last sequence are no rows: their out and lse stay
 * as they were, their gradients are set to 0.
 *
 * Values of keys outside a sequence never reach it, whatever they are.  A
 * key inside it whose v holds infinities or NaNs can make NaN of out in the
 * rows the causal mask hides it from: a weight of 0 times NaN.  Likewise q, k,
 * v and dout in the gradients of what they are hidden from.  In the backward
 * functions a score gradient is rounded to the inputs' type: in fp16 one
 * beyond 65504 becomes infinite.
 *
 * Ownership and execution are gemm_tn's (mfl_gemm.h): nothing is allocated,
 * kept or synchronised; work runs on `stream`.  A workspace belongs to one
 * call until that call's work is done; its size comes from the *_plan
 * function, which makes the same checks without touching the GPU.  Outputs
 * must not overlap inputs or the workspace.  Results are the same bits for
 * the same arguments: no sum depends on the order workgroups run in.
 */
#ifndef MFL_ATTENTION_H
#define MFL_ATTENTION_H

#include <stdint.h>

#include "mfl_gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MFL_BF16 3            /* mfl_dtype of these functions, beside MFL_F16 */
#define MFL_E_WORKSPACE (-10) /* workspace NULL, misaligned or too small */

/* Kernel of the forward functions: AUTO chooses by sizes.  TALL: four
 * waves of 32 rows (a row is a token of one query head) share each chunk of
 * keys; FLAT: 16 rows per workgroup, whose four waves take turns over the
 * keys.  The lengths are on the device, so AUTO and splits = 0 go by their
 * means: for one long sequence among many short ones the caller does better
 * to give both (TALL for a prompt among single tokens, splits for one
 * sequence with most of the keys). */
#define MFL_ATTENTION_AUTO 0
#define MFL_ATTENTION_TALL 1
#define MFL_ATTENTION_FLAT 2

typedef struct {
  int32_t dtype;                /* MFL_F16 or MFL_BF16 */
  int32_t causal;               /* 0 or 1 */
  int64_t batch;                /* sequences, >= 1 */
  int64_t total_q, total_k;     /* tokens of q and out, of k and v */
  int64_t heads_q, heads_kv;    /* heads_q a multiple of heads_kv */
  int64_t head_dim;
  int64_t q_token, q_head, k_token, k_head, v_token, v_head, out_token, out_head;
  float scale;                  /* > 0, scale * log2(e) finite */
  int32_t algo;                 /* MFL_ATTENTION_* */
  int32_t splits;               /* parts the keys are split into, 0: by sizes */
} mfl_attention_t;

/* out, and lse (total_q x heads_q, contiguous) unless NULL. */
int attention_packed(const mfl_attention_t* a, const void* q, const void* k, const void* v,
                     const int32_t* seq_q, const int32_t* seq_k, void* out, float* lse,
                     void* workspace, int64_t workspace_bytes, void* stream);
/* the same checks; on success the kernel, the splits and the workspace's size
 * (0: none needed).  Any out pointer may be NULL.
 * With dc = head_dim rounded up to 64, 128 or 256 the workspace of n > 1
 * splits is n * total_q * heads_q * (4 dc + 8) bytes; for splits = 0 n is at
 * most 64 and the workspace at most 256 MiB. */
int attention_packed_plan(const mfl_attention_t* a, const void* q, const void* k, const void* v,
                          const int32_t* seq_q, const int32_t* seq_k, const void* out,
                          const float* lse, int32_t* algo, int32_t* splits,
                          int64_t* workspace_bytes);

/* Gradients of sum(out * dout) with respect to q, k and v, from the forward
 * call's out and lse; `f` as in that call (algo and splits are not read).
 * With more than one token q_token and dout_token are at least head_dim
 * (MFL_E_LEADING_DIM).  Gradients of tokens behind the last sequence are 0.
 *
 * The workspace: 8 bytes per token and query head, and, where tiles of keys
 * are cut between workgroups (up to 256 sequences and some 2000 tiles over
 * the kv heads), fp32 sums of dK and dV for every workgroup and tile, and
 * never more than two per workgroup: 64 KiB each up to head_dim 64, else
 * 256 KiB.  The workgroups are about 256, or up to 1024 where the kv heads
 * do not divide 256 well; fewer for few tokens.  8192 tokens in four sequences
 * of 32/8 heads of 128 take 136 MB, 1045 tokens in three of 16/4 heads 74 MB. */
typedef struct {
  mfl_attention_t f;
  int64_t dout_token, dout_head, dq_token, dq_head, dk_token, dk_head, dv_token, dv_head;
} mfl_attention_grad_t;

int attention_packed_backward(const mfl_attention_grad_t* a, const void* dout, const void* q,
                              const void* k, const void* v, const void* out, const float* lse,
                              const int32_t* seq_q, const int32_t* seq_k, void* dq, void* dk,
                              void* dv, void* workspace, int64_t workspace_bytes, void* stream);
int attention_packed_backward_plan(const mfl_attention_grad_t* a, const void* dout,
                                   const void* q, const void* k, const void* v, const void* out,
                                   const float* lse, const int32_t* seq_q, const int32_t* seq_k,
                                   const void* dq, const void* dk, const void* dv,
                                   int64_t* workspace_bytes);

/* Decoding behind a shared prefix: `batch` sequences of q_tokens query
 * tokens each.  Every query sees all `prefix` keys of prefix_k / prefix_v;
 * query token t of sequence b also sees the keys j <= lengths[b] - q_tokens + t
 * of its own cache k(b, j, g, d) = K[b * k_batch + j * k_token + g * k_head + d],
 * which holds lengths[b] keys (device memory, held inside [0, capacity]), the
 * new tokens' among them.  Prefix keys are held and fetched once for all
 * sequences' rows together, per tile of 128 rows of a kv head (16 in FLAT). */
typedef struct {
  int32_t dtype;
  int32_t algo;                 /* of the prefix's part: AUTO, TALL or FLAT */
  int64_t batch, q_tokens;
  int64_t prefix, capacity;
  int64_t heads_q, heads_kv, head_dim;
  int64_t q_batch, q_token, q_head, prefix_k_token, prefix_k_head, prefix_v_token,
      prefix_v_head;
  int64_t k_batch, k_token, k_head, v_batch, v_token, v_head, out_batch, out_token, out_head;
  float scale;
  int32_t splits_prefix, splits_own;   /* 0: by sizes */
} mfl_attention_prefix_t;

/* lse: batch x q_tokens x heads_q, contiguous, or NULL */
int attention_prefix(const mfl_attention_prefix_t* a, const void* q, const void* prefix_k,
                     const void* prefix_v, const void* k, const void* v, const int32_t* lengths,
                     void* out, float* lse, void* workspace, int64_t workspace_bytes,
                     void* stream);
int attention_prefix_plan(const mfl_attention_prefix_t* a, const void* q, const void* prefix_k,
                          const void* prefix_v, const void* k, const void* v,
                          const int32_t* lengths, const void* out, const float* lse,
                          int32_t* algo, int32_t* splits_prefix, int32_t* splits_own,
                          int64_t* workspace_bytes);

#ifdef __cplusplus
}
#endif
#endif /* MFL_ATTENTION_H */
