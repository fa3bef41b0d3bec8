/*
 * mla_prompt.h -- C ABI of libmla_decode.so: the attention of a prompt, head by
 * head, over keys and values up-projected from the latent rows (those that
 * mla_cache_gather gives back, or a prompt's own before they are stored).
 *
 * The documents of a batch lie side by side, as qo_indptr and kv_indptr say.
 * With n = qo_indptr[b + 1] - qo_indptr[b] query tokens and m = kv_indptr[b + 1]
 * - kv_indptr[b] keys, query token i of document b sees its key j < m if
 *   not causal, or j <= m - n + i (the last n keys are the tokens' own), or
 *   j < prefix[b] (a prefix that every token sees),
 * and no key of another document.  For head h, over the keys that it sees,
 *   s_j = sm_scale * (q_nope[i, h, :128] . k_nope[j, h, :128] + q_pe[i, h, :64] . k_pe[j, :64])
 *   out[i, h, :128] = sum_j softmax(s)_j v[j, h, :128]
 *   lse[i, h]       = ln sum_j exp(s_j)                      (natural log)
 * A token that sees nothing gets out = 0 and lse = -inf.  The position part k_pe
 * is one for all heads.  A single token's form is the decode (mla_decode.h).
 *
 * Conventions are those of mla_decode.h: an mla_status from every entry point,
 * nothing allocated, no synchronisation, launches on `stream` of the current
 * device.  Document bounds that do not fit (decreasing, negative, past num_q or
 * num_kv) set MLA_ERR_DEVICE_INDEX in the workspace's first word, which
 * mla_decode_poll_error(workspace, stream) reads and clears; that document's rows
 * of out and lse are then not written, and nothing outside the tensors is read.
 * The other documents are computed (of more than 32, some of their rows may stay as
 * they were too), where no two of them claim the same rows.
 */
#ifndef MLA_PROMPT_H
#define MLA_PROMPT_H

#include "mla_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MLA_PROMPT_NOPE 128
#define MLA_PROMPT_PE 64
#define MLA_PROMPT_V 128
#define MLA_PROMPT_MAX_HEADS 128

/* One call.  Rows are consecutive in their last dimension; strides are in
 * elements, multiples of 8 and positive (of dimensions of size 1 not looked at).
 * The inputs are device memory, 16-byte aligned, and do not overlap out or lse. */
typedef struct {
  const void* q_nope;        /* bf16 [num_q, heads, 128] */
  const void* q_pe;          /* bf16 [num_q, heads, 64] */
  const void* k_nope;        /* bf16 [num_kv, heads, 128] */
  const void* k_pe;          /* bf16 [num_kv, 64] */
  const void* v;             /* bf16 [num_kv, heads, 128]; the keys' values are finite, seen or not (what lies
                                past a document's last key may be anything) */
  const int32_t* qo_indptr;  /* device [batch + 1] */
  const int32_t* kv_indptr;  /* device [batch + 1] */
  const int32_t* prefix;     /* device [batch], or NULL: none; below 0 counts as 0, past the keys as all */
  void* out;                 /* bf16 [num_q, heads, 128], 16-byte aligned; rows of no document stay */
  float* lse;                /* fp32 [num_q, heads], contiguous, or NULL */
  int64_t q_nope_token_stride, q_nope_head_stride;
  int64_t q_pe_token_stride, q_pe_head_stride;
  int64_t k_nope_token_stride, k_nope_head_stride;
  int64_t k_pe_token_stride;
  int64_t v_token_stride, v_head_stride;
  int64_t out_token_stride, out_head_stride;
  int32_t num_q, num_kv;     /* rows of the tensors, below 2^30 */
  int32_t batch;             /* documents, 0..MLA_MAX_BATCH */
  int32_t heads;             /* 1..MLA_PROMPT_MAX_HEADS */
  int32_t causal;            /* 1, or 0: every key of the document is seen */
  float sm_scale;            /* finite, > 0 */
} mla_prompt_args;

/* Bytes of device workspace of a call of these sizes (only num_q, num_kv, batch
 * and heads are read; 0 on null or bad sizes). */
MLA_API size_t mla_prompt_workspace_bytes(const mla_prompt_args* args);

/*
 * mla_prompt_fwd -- enqueues one call.  workspace: device, 256-byte aligned, at
 * least mla_prompt_workspace_bytes(args) bytes, its first word zeroed before the
 * first use; calls that share it must be ordered on the GPU.
 */
MLA_API int mla_prompt_fwd(const mla_prompt_args* args, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MLA_PROMPT_H */
