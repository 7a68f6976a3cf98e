/*
 * spec_serve.h -- C ABI of libspecverify, part two: the operators a serving loop needs around the
 * speculative round of spec_verify.h, on the same GPU and with the same conventions.
 *
 *   spec_paged_attn      Attention of a ragged batch of new-token chunks over a PAGED KV cache: one
 *                        token per sequence (decode), gamma + 1 (verify), or a chunk of its prompt,
 *                        mixed freely in one call; optionally appends the chunk's K/V to the pages.
 *   spec_prefill_attn    Causal attention over whole prompts packed one after the other.
 *   spec_token_logprobs  Log probabilities of given tokens, with each row's entropy and its top
 *                        alternatives.
 *
 * Conventions are those of spec_verify.h: device pointers owned by the caller, strides in ELEMENTS
 * with the innermost dimension contiguous, asynchronous calls on the given stream of the calling
 * thread's current device, no allocation, no global mutable state, host validation before any
 * launch, negative return codes, a caller workspace (256-byte aligned; calls that share one must
 * not overlap, and that includes replays of captured graphs) whose first 32-bit word is the call's
 * device status, cleared by the call.  A call can be captured into a CUDA graph; everything it
 * reads from device memory (lengths, tables, data) is read anew by each replay.
 * spec_commit(SPEC_COMMIT_CHAIN) works on a paged cache as it is: it moves only kv_len.
 */
#ifndef SPEC_SERVE_H_
#define SPEC_SERVE_H_

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* further flags of the device status word */
enum {
  SPEC_STATUS_BAD_RANGE = 16, /* q_start: negative, decreasing, above T, or a chunk above max_q */
  SPEC_STATUS_BAD_PAGE = 32   /* a needed page id outside [0, num_pages) */
};

/* ------------------------------------------------------------------------------------------
 * spec_paged_attn
 *
 * The batch's new tokens lie one after the other: sequence b owns rows q_start[b] ..
 * q_start[b + 1] - 1 of q, o, k_new and v_new (n_b of them; n_b = 0 is allowed).  Its cache holds
 * kv_len[b] tokens, of which the last n_b are the new ones, so row q_start[b] + j is position
 * p = kv_len[b] - n_b + j and
 *     o[row, h, :] = softmax_t(scale * q[row, h, :] . k[t, g, :]) @ v[t, g, :],  g = h / (Hq / Hkv),
 * over t in (p - window, p] (window > 0) or [0, p] (window == 0).  Token t of sequence b is slot
 * t % page_size of page page_table[b, t / page_size].
 *   k_new / v_new set (both or neither): the call also writes the new tokens' rows into their
 *   slots; the attention uses them.  A slot written to must be one new token's and seen by its
 *   sequence alone (pages that sequences share hold earlier tokens only).  NULL: the caller has
 *   written them.
 *   window: K/V of tokens below kv_len[b] - n_b + 1 - window are not read, nor are their table
 *   entries, so their pages may have been given back.
 *
 * Layout: q, o [T, Hq, D] (strides _t, _h); k_new, v_new [T, Hkv, D] (new_stride_t, new_stride_h);
 *   k_pages, v_pages [num_pages, Hkv, page_size, D] with any strides for page, head and token
 *   (kv_stride_p, kv_stride_h, kv_stride_t), equal for both; page_table [B, table_cols] int32 with
 *   row stride table_stride; q_start [B + 1] and kv_len [B] int32.
 * Types: kv_dtype SPEC_BF16 or SPEC_F32, q and k_new / v_new of the same; o_dtype SPEC_F32 or
 *   SPEC_BF16.  All strides but o's are multiples of 16 bytes, all pointers but o's (element
 *   aligned) and the int32 ones are 16-byte aligned.
 * Limits: D in {64, 128}; Hq % Hkv == 0, Hq / Hkv <= 32; 1 <= B <= 4096; 0 <= T <= 2^22 (T == 0:
 *   nothing is launched); max_q >= 1; 1 <= page_size <= 65536; table_cols >= 1;
 *   table_cols * page_size <= 2^30; window >= 0; scale >= 0, scale * log2(e) finite.  max_q is an upper
 *   bound on every n_b and chooses the kernel; a tight one is faster.
 * No output overlaps an input: not o, nor the pages with k_new / v_new.
 * Rows of q at or past q_start[B], or before q_start[0], are not read and their o is left as it was.
 * Data errors: a sequence whose q_start is out of order (SPEC_STATUS_BAD_RANGE) has no rows, and
 *   its o is left as it was (ranges that overlap, so that they add up to more than T rows, can cost the
 *   others theirs too); kv_len[b] < n_b or > table_cols * page_size (SPEC_STATUS_BAD_KV_LEN)
 *   gives zeros and no append; a needed page id out of range (SPEC_STATUS_BAD_PAGE) is never
 *   followed: its tokens read as zeros (o of the rows that see them is not meaningful) and are not
 *   written (appended rows then take part from k_new / v_new, or as zeros).
 * K and V of the tokens that some row of the chunk sees have to be finite, and so do a row's scores times
 *   scale * log2(e) in fp32 (else that row's o is unspecified); slots past kv_len and pages before the
 *   window may hold anything.
 * Accumulation is fp32 (scores, softmax statistics, P.V); for bf16 K/V the probabilities are
 *   rounded to bf16 before P.V, as in spec_verify_attn.  A call's result is the same every time; it
 *   can differ in the last bits between batches (and devices), whose work is cut differently.
 * ---------------------------------------------------------------------------------------- */
typedef struct spec_paged_args {
  int32_t B, Hq, Hkv, D, T, max_q;
  int32_t q_dtype, kv_dtype, o_dtype;
  int32_t page_size, num_pages, table_cols;
  int32_t window;
  float scale;                /* 0: 1/sqrt(D) */
  const void* q;
  int64_t q_stride_t, q_stride_h;
  void* k_pages;              /* written only with k_new / v_new */
  void* v_pages;
  int64_t kv_stride_p, kv_stride_h, kv_stride_t;
  const int32_t* page_table;
  int64_t table_stride;
  const int32_t* q_start;
  const int32_t* kv_len;
  const void* k_new;
  const void* v_new;
  int64_t new_stride_t, new_stride_h;
  void* o;
  int64_t o_stride_t, o_stride_h;
  void* workspace;
  size_t workspace_bytes;
} spec_paged_args;

/* Bytes of workspace (host only, pure; reads the sizes, types and max_q).  0: invalid sizes. */
size_t spec_paged_attn_workspace(const spec_paged_args* args);
int spec_paged_attn(const spec_paged_args* args, spec_stream_t stream);

/* ------------------------------------------------------------------------------------------
 * spec_prefill_attn
 *
 * Prompts packed one after the other: sequence b owns rows seq_start[b] .. seq_start[b + 1] - 1 of
 * q, k, v and o.  Row seq_start[b] + j attends causally to the rows seq_start[b] .. of its own
 * sequence, the last `window` of them if window > 0 (what spec_draft_window_attn later sees of its
 * ring).  Sequences of length 0 are allowed.
 * Layout: q, o [T, Hq, D]; k, v [T, Hkv, D] with equal strides; seq_start [B + 1] int32.
 * Types, alignment, limits, overlap, rows outside the sequences, finiteness (of a sequence's own
 *   rows: neighbours may hold anything) and accumulation as spec_paged_attn; a sequence whose seq_start is out of order is skipped
 *   (SPEC_STATUS_BAD_RANGE).
 * ---------------------------------------------------------------------------------------- */
typedef struct spec_prefill_args {
  int32_t B, Hq, Hkv, D, T, window;
  int32_t q_dtype, kv_dtype, o_dtype;
  float scale;
  const void* q;
  int64_t q_stride_t, q_stride_h;
  const void* k;
  const void* v;
  int64_t kv_stride_t, kv_stride_h;
  const int32_t* seq_start;
  void* o;
  int64_t o_stride_t, o_stride_h;
  void* workspace;
  size_t workspace_bytes;
} spec_prefill_args;

size_t spec_prefill_attn_workspace(const spec_prefill_args* args);
int spec_prefill_attn(const spec_prefill_args* args, spec_stream_t stream);

/* ------------------------------------------------------------------------------------------
 * spec_token_logprobs
 *
 * For every row r of logits [N, V], with lse = log sum_v exp(logits[r, v]):
 *     logprobs[r]        = logits[r, tokens[r]] - lse
 *     entropy[r]         = -sum_v p_v log p_v,  p_v = exp(logits[r, v] - lse)      (optional)
 *     top_ids[r, 0..K-1] = the K ids of largest logit in descending order, the lower id first among
 *                          equals, and top_logprobs[r, i] = logits[r, top_ids[r, i]] - lse (optional)
 * Layout: logits fp32 or bf16 (SPEC_F32 / SPEC_BF16), rows of V contiguous, row stride
 *   logits_stride >= V, element-aligned (any V, any stride); tokens [N] int32 or NULL (with logprobs
 *   NULL: neither); logprobs, entropy [N] fp32; top_ids int32 and top_logprobs fp32 [N, K]
 *   contiguous (both, or neither with K == 0).
 * Limits: 0 <= N <= 2^24 (0: nothing is launched); 1 <= V <= 2^24; 0 <= K <= min(32, V).
 * Values: -inf entries are allowed (log probability -inf, no part of the entropy).  A row of nothing
 *   but -inf has no distribution: its log probabilities are -inf, its entropy 0 and its top ids 0,
 *   1, ....  NaN and +inf entries leave that row's outputs unspecified.
 * A token outside [0, V) gives logprobs[r] = 0 and SPEC_STATUS_BAD_TOKEN; the row's other outputs are
 *   computed.
 * Sums are fp32, in a fixed order; exponentials are 2^x of the scaled, max-subtracted logit with a
 *   relative error of about 2^-22.
 * ---------------------------------------------------------------------------------------- */
typedef struct spec_logprob_args {
  int32_t N, V, K, dtype;
  const void* logits;
  int64_t logits_stride;
  const int32_t* tokens;
  float* logprobs;
  float* entropy;
  int32_t* top_ids;
  float* top_logprobs;
  void* workspace;
  size_t workspace_bytes;
} spec_logprob_args;

size_t spec_token_logprobs_workspace(const spec_logprob_args* args);
int spec_token_logprobs(const spec_logprob_args* args, spec_stream_t stream);

/* sizeof() of this header's structs as compiled: which = 0 spec_paged_args, 1 spec_prefill_args,
 * 2 spec_logprob_args; else 0. */
size_t spec_serve_struct_size(int which);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_SERVE_H_ */
