/*
 * kq_prompt.h -- C ABI of libkq.so for a prompt: the norms of query and key
 * heads with their rotary positions, causal attention of whole prompts, and
 * the log probabilities of given tokens.
 *
 * The conventions are those of kq.h and kq_decode.h: asynchronous on the
 * caller's stream, capturable in a CUDA graph, every argument checked on the
 * host first (a call that returns an error has enqueued nothing, except
 * KQ_ERR_CUDA from a later launch of several), all memory owned by the caller,
 * no pointer kept after the call.  Pointers are memory of the current device
 * or managed memory; anything else is KQ_ERR_MEMORY.  Starts, positions and
 * tokens are read on the device, and a bad one never reads or writes outside
 * the caller's buffers.  Results are deterministic: bitwise the same for the
 * same inputs on the same device model.
 *
 * Activations are f32, or 16-bit where a type is an argument.
 */
#ifndef KQ_PROMPT_H
#define KQ_PROMPT_H

#include <stdint.h>

#include "kq.h"
#include "kq_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Types of activations (type codes as kq_fmt has them). */
#define KQ_F32 0
#define KQ_F16 1
#define KQ_BF16 30

#define KQ_MAX_NORM_PARTS 4
#define KQ_MAX_TOP 32 /* alternatives of kq_token_logprobs */

/*
 * One tensor of a kq_norm_rope call: x [ntok][heads][dim], `stride` values
 * from token to token, its weight f32 [dim] (NULL: ones) and its output.
 * Strides are multiples of 16 bytes and at least heads * dim; x and out are
 * 16-byte aligned, weight too.
 */
typedef struct kq_norm_part {
    const void *x;
    int64_t stride;
    const float *weight;
    void *out; /* x itself (same type and stride), or no overlap */
    int64_t out_stride;
    int32_t heads;    /* 1..KQ_MAX_HEADS */
    int32_t reserved; /* must be 0 */
} kq_norm_part;

/*
 * Norm of each head, and its rotary positions, in one pass over up to
 * KQ_MAX_NORM_PARTS tensors of the same tokens (queries and keys):
 *
 *   y = x * (mean(x^2) + eps)^-1/2 * weight        over a head's dim values
 *
 * then, with a table (not NULL), the first rot values are turned by the
 * token's position as kq_rope does.  type: of x, KQ_F32, KQ_F16 or KQ_BF16;
 * out_type: the same, or any of the three where type is KQ_F32.  Everything
 * is computed in f32 and rounded once, to nearest even.  Magnitudes whose
 * squares f32 does not hold are scaled first.
 *
 *   dim  multiple of 8, 8..1024;  eps finite, >= 0
 *   pos  device int32 [ntok]; a position outside 0..positions-1 gives a token
 *        of NaN (with a table; otherwise pos is not looked at)
 *   rot  multiple of 8, 8..dim
 */
kq_status kq_norm_rope(const kq_norm_part *parts, int n, int type, int out_type, int64_t ntok,
                       int dim, float eps, const int32_t *pos, const float *table,
                       int64_t positions, int rot, int interleaved, void *stream);

/*
 * Causal attention of whole prompts, packed one behind the other:
 *
 *   out[t][h] = sum_j p_j v_j,  p = softmax over j of scale * (q[t][h] . k_j)
 *
 * Sequence b has the queries start[b] .. start[b+1]-1 (n of them) and the keys
 * and values key_start[b] .. key_start[b+1]-1 (m of them); its queries are the
 * last n of its m tokens, so that query i attends keys j <= i + m - n.  Where m
 * < n the first queries attend nothing, and their rows are zero.  key_start
 * NULL: start (no tokens before the prompt; nkeys must be ntok).
 *
 * A start counts as the largest so far, within 0..ntok (0..nkeys), so that
 * sequences never overlap, whatever the starts are.  Rows of no sequence are
 * left as they were.  NaN and infinities in keys and values that a
 * row does not attend do not reach it.
 *
 *   type  of q, k, v and out: KQ_F32, KQ_F16 or KQ_BF16
 *   q     device [ntok][q_heads][dim], q_stride values from token to token;
 *         q_heads a multiple of kv_heads, query head h reads key head
 *         h / (q_heads / kv_heads); dim 64, 128 or 256
 *   k, v  device [nkeys][kv_heads][dim], their strides from token to token
 *   out   device [ntok][q_heads][dim], dense
 *   ws    device workspace of kq_prompt_workspace_bytes(...) bytes or more,
 *         256-byte aligned; NULL: a stream-ordered temporary.  One that is too
 *         small is KQ_ERR_LIMIT.
 *
 * q, k, v and out are 16-byte aligned, strides multiples of 16 bytes.  scale is
 * finite, of either sign (16-bit types: below 2.35e38, so that its product with
 * log2(e) is finite too; KQ_ERR_SHAPE).  Sums, maxima and corrections are f32.  16-bit types:
 * products are exact, probabilities are rounded to the type (the error is
 * then 1.25 to 1.4 times that of the output's own rounding).  KQ_F32: queries,
 * keys, values and probabilities are held as two f16 terms (22 bits, after a
 * scaling by a power of two: of a query's row, and of a sequence's 64 or 32
 * keys or values, or of each of these where their largest values lie further
 * apart than 2^12; what is below 2^-27 of the largest value of its key, value
 * or query, or 2^-39 of a row's largest probability times value, is dropped),
 * so logits may be as large as 2e38, as long as scale * q is below that too.
 * However large a key or value is, rows that do not attend it, or whose
 * probability for it is small enough, are as exact as without it.  A row is
 * divided by its probabilities' sum at the end, so a value's size times the
 * number of keys (bf16: and 2^8) has to be within f32.  A
 * row that attends a key with an infinity may be NaN where the formula has a
 * weight of zero, and so may one that attends an infinite value of a 16-bit
 * type where its probability is too small for the type.
 */
kq_status kq_prompt_attention(int type, int nseq, int64_t ntok, int64_t nkeys,
                              const int32_t *start, const int32_t *key_start, const void *q,
                              int64_t q_stride, int q_heads, const void *k, int64_t k_stride,
                              const void *v, int64_t v_stride, int kv_heads, int dim, float scale,
                              void *out, void *ws, int64_t ws_bytes, void *stream);

/* Workspace bytes of kq_prompt_attention on the current device, from sizes
 * alone (0: none is needed), or a negative kq_status. */
int64_t kq_prompt_workspace_bytes(int type, int nseq, int64_t ntok, int64_t nkeys, int q_heads,
                                  int kv_heads, int dim);

/*
 * Log probabilities from logits x, row by row: with m = max x and
 * S = sum exp(x - m),
 *
 *   logp    = x[token] - m - log S
 *   entropy = log S - sum exp(x - m) (x - m) / S      (0 * -inf is 0)
 *   top     the `top` largest logits, largest first, of equal ones the lower
 *           token first: their tokens, and their log probabilities
 *
 * A logit of -infinity has probability zero.  A row that holds a NaN or
 * +infinity, or nothing but -infinity, has NaN for logp, entropy and the log
 * probabilities of its alternatives, whose tokens are still those of the
 * largest logits (a NaN counts as larger than any).  A token outside the
 * vocabulary has a logp of NaN.
 *
 *   type    KQ_F32, KQ_F16 or KQ_BF16
 *   logits  device [n][vocab], stride values from row to row, aligned to the
 *           type's size; vocab 1..KQ_MAX_VOCAB, n 0..2^24
 *   token   device int32 [n], with logp f32 [n]; both NULL: not computed
 *   entropy device f32 [n] or NULL
 *   top     0..min(KQ_MAX_TOP, vocab); top_logp f32 [n][top], top_token int32
 *           [n][top] (not looked at for 0)
 */
kq_status kq_token_logprobs(int type, int64_t n, int vocab, const void *logits, int64_t stride,
                            const int32_t *token, int top, float *logp, float *entropy,
                            float *top_logp, int32_t *top_token, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* KQ_PROMPT_H */
