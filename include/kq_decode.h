/*
 * kq_decode.h -- C ABI of libkq.so for what a decode step does around its
 * matvecs: rotary positions, a quantised key/value cache, attention of the
 * new tokens over that cache, and the verification of drafted tokens.
 *
 * The operators share two descriptors: kq_kv, the cache, and kq_batch, the
 * sequences of a step.  They follow kq.h's conventions: f32 activations,
 * asynchronous on the caller's stream, capturable in a CUDA graph, every
 * argument checked on the host first (a call that returns an error has
 * enqueued nothing, except KQ_ERR_CUDA from a later launch of several), all
 * memory owned by the caller, no pointer kept after the call.  Pointers are
 * memory of the current device or managed memory; anything else is
 * KQ_ERR_MEMORY.  Lengths, page tables and positions are read on the
 * device, so a captured graph serves a growing sequence.  What they hold is
 * checked there: a bad entry never reads or writes outside the caller's
 * buffers, and what it gives is said at each function.
 *
 * Results are deterministic: bitwise the same for the same inputs on the
 * same device model.
 */
#ifndef KQ_DECODE_H
#define KQ_DECODE_H

#include <stdint.h>

#include "kq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Cache formats, with the type codes that kq_fmt uses too.  Quantised
 * formats hold groups of 32 consecutive values of a head, one f16 scale d
 * each, with value = code * d:
 *   KQ_KV_F16  f16, rounded to nearest
 *   KQ_KV_Q8   8 bits: d = max|x| / 127, code = round(x / d) in -127..127
 *   KQ_KV_Q4   4 bits: d = m / -8, m the value of largest magnitude (the
 *              positive one of a tie), code = round(x / d) in -8..7
 * d is rounded to f16 (magnitudes above 65504 become 65504) before the codes
 * are formed from it; rounding is to nearest, ties to even, and every step
 * is one f32 operation.  A group that holds a NaN or an infinity reads back
 * as NaN. */
#define KQ_KV_F16 1
#define KQ_KV_Q4 2
#define KQ_KV_Q8 8

#define KQ_KV_PAGE 64        /* tokens of a cache page                      */
#define KQ_MAX_SEQS 4096     /* sequences of a batch                        */
#define KQ_MAX_DRAFT 64      /* new tokens of one sequence in an attention
                                or verification call                        */
#define KQ_MAX_HEADS 1024
#define KQ_MAX_VOCAB (1 << 19)

/*
 * A paged key/value cache of one layer: `pages` pages of 64 tokens of
 * kv_heads heads of head_dim (64, 128 or 256) values.  One page and head is
 * one contiguous block of kq_kv_page_bytes / kv_heads bytes, laid out for
 * the attention kernel's loads:
 *   keys' codes    [slab][token][64 bytes]: a slab is 1 (F16), 2 (Q8) or 4
 *                  (Q4; 2 and 32 bytes for head_dim 64) groups of 32
 *                  values; octet c (8 values) of the slab's group g lies at
 *                  place c * groups + g of the token's bytes
 *   keys' scales   [token][group] f16            (quantised formats)
 *   values' codes  [token slab][value][tokens of the slab]: 32 (F16) or 64
 *                  tokens a slab
 *   values' scales [group][token] f16            (quantised formats)
 * 4-bit codes are two's complement, the lower-numbered one in the low
 * nibble.  Page p, head h starts at data + (p * kv_heads + h) * block.
 */
typedef struct kq_kv {
    int32_t fmt;      /* KQ_KV_F16, KQ_KV_Q8 or KQ_KV_Q4 */
    int32_t kv_heads; /* 1..KQ_MAX_HEADS */
    int32_t head_dim; /* 64, 128 or 256 */
    int32_t reserved; /* must be 0 */
    void *data;       /* kq_kv_page_bytes * pages bytes, 16-byte aligned */
    int64_t pages;    /* 1..2^31-1 */
} kq_kv;

/*
 * The sequences of a step and their new tokens.  Sequence b holds ctx[b]
 * committed tokens; its new tokens are tokens start[b] .. start[b+1]-1 of
 * the step, and new token j sits at place ctx[b] + j of the sequence.  Place
 * t lies in page pages[b * max_pages + t / 64], token t % 64.
 *
 * Sequences whose start is not within 0..ntok in rising order, whose new
 * tokens pass max_new, or whose ctx is negative are cut to what is.  (Starts
 * that fall and rise again can give a token to two sequences; what a call
 * writes for it is then either's.)  A call that writes the cache needs a page of
 * its own for each entry of its tables; calls that read it do not.
 */
typedef struct kq_batch {
    int32_t nseq;         /* 1..KQ_MAX_SEQS */
    int32_t max_new;      /* most new tokens of one sequence, 1..2^24 */
    int64_t ntok;         /* new tokens in all, 0..2^24 (0: nothing is done) */
    const int32_t *start; /* device [nseq + 1] */
    const int32_t *ctx;   /* device [nseq] */
    const int32_t *pages; /* device [nseq][max_pages] */
    int64_t max_pages;    /* 1..2^24 */
} kq_batch;

/* Bytes of one page (all heads, keys and values), or -1 for bad arguments. */
int64_t kq_kv_page_bytes(int fmt, int kv_heads, int head_dim);

/* How rotary positions are stretched for contexts longer than the model was
 * trained on.  theta_i = base^(-2i / rot) is pair i's angle a position. */
typedef struct kq_rope_scaling {
    int32_t kind; /* 0 none; 1 linear: theta / factor; 2 base: base becomes
                     base * factor^(rot / (rot - 2)); 3 ramp: pairs that turn
                     more than `fast` times in `orig` positions keep theta,
                     those that turn less than `slow` times get theta /
                     factor, those between a blend that is linear in their
                     turns (one that is linear in the pair's index, as some
                     models have it, needs a table of the caller's) */
    int32_t orig; /* ramp: positions the model was trained on, >= 1 */
    double factor; /* > 0 (kinds 1..3) */
    double fast, slow; /* ramp: fast > slow >= 0 */
    double magnitude;  /* cos and sin are multiplied by it; 1 leaves them */
} kq_rope_scaling;

/*
 * Table of (cos, sin) pairs: table f32 [positions][rot / 2][2], angles and
 * functions formed in 64 bits and rounded once, so that far positions are as
 * exact as near ones.  rot: multiple of 8, 8..1024; scaling may be NULL.
 */
kq_status kq_rope_table(int64_t positions, int rot, double base, const kq_rope_scaling *scaling,
                        float *table, void *stream);

/*
 * Rotary positions: of each head's first rot values, pair i
 *   (a, b) -> (a c - b s, b c + a s),  (c, s) = table[pos[t]][i]
 * with a, b the values i and i + rot/2 (interleaved = 0) or 2i and 2i + 1
 * (interleaved = 1); the others are copied.  inverse != 0 turns back (s
 * negated), which is also the gradient.  Both products and the sum are
 * rounded, without a fused step, so that kq_kv_append sees the same keys.
 *
 *   x    device f32 [ntok][heads][dim], `stride` values (multiple of 4) from
 *        token to token; 16-byte aligned.  dim: multiple of 8, 8..1024.
 *   out  device f32 [ntok][heads][dim], out_stride from token to token;
 *        either x itself with the same stride (in place) or no overlap.
 *   pos  device int32 [ntok]; a position outside 0..positions-1 gives a
 *        token of NaN.
 */
kq_status kq_rope(const float *x, int64_t stride, float *out, int64_t out_stride, int64_t ntok,
                  int heads, int dim, const int32_t *pos, const float *table, int64_t positions,
                  int rot, int interleaved, int inverse, void *stream);

/*
 * Quantise the new tokens' keys and values into the cache at places ctx[b] +
 * j.  With a table (not NULL) the keys are rotated first, as kq_rope does,
 * with position pos[t] of each new token (in a tree of drafts that is not
 * its place); without a table pos is not looked at.  k and v: device f32
 * [ntok][kv_heads][head_dim], strides (multiples of 4) from token to token,
 * 16-byte aligned.  Tokens whose place has no valid page are skipped; a bad
 * position stores a key of NaN, all of it.
 */
kq_status kq_kv_append(const kq_kv *kv, const kq_batch *batch, const float *k, int64_t k_stride,
                       const float *v, int64_t v_stride, const int32_t *pos, const float *table,
                       int64_t positions, int rot, int interleaved, void *stream);

/*
 * Read places ctx[b] + j back as f32: k, v device [ntok][kv_heads][head_dim]
 * dense, 16-byte aligned; either may be NULL.  (With ctx = 0 and the whole
 * length as new tokens this reads a sequence.)  A place without a valid page
 * reads as NaN; tokens of no sequence are left as they were.
 */
kq_status kq_kv_read(const kq_kv *kv, const kq_batch *batch, float *k, float *v, void *stream);

/*
 * Close the gaps that rejected drafts leave: copies place ctx[b] + path[i]
 * to ctx[b] + i for i < count[b], path = path + start[b], as kq_verify_tree
 * writes them (path rising).  Entries that are not rising or not new tokens
 * of the sequence, and those after them, are ignored.  Codes are copied, not
 * quantised again.  path: device int32 [ntok], count: device int32 [nseq].
 * max_new <= KQ_MAX_DRAFT.
 */
kq_status kq_kv_move(const kq_kv *kv, const kq_batch *batch, const int32_t *path,
                     const int32_t *count, void *stream);

/*
 * Attention of the new tokens over the cache, the new tokens' own keys and
 * values included (kq_kv_append comes first):
 *
 *   out[t][h] = sum_s p_s v_s,  p = softmax over s of scale * (q[t][h] . k_s)
 *
 * s runs over the sequence's ctx[b] committed places and over those new
 * tokens j whose bit j is set in mask[t] (a tree of drafts: a token's
 * ancestors and itself; any other set works too).  mask NULL: all new tokens
 * up to t itself.  A row that attends nothing is zero.  NaN and infinities
 * in places that a row does not attend do not reach it.
 *
 *   q    device f32 [ntok][q_heads][head_dim], q_stride values (multiple of
 *        4) from token to token; 16-byte aligned.  q_heads: a multiple of
 *        kv_heads; query head h reads key head h / (q_heads / kv_heads).
 *   mask device uint64 [ntok] or NULL, 8-byte aligned.
 *   out  device f32 [ntok][q_heads][head_dim] dense, 16-byte aligned; tokens
 *        of no sequence are left as they were.
 *   ws   device workspace of kq_attn_workspace_bytes(...) bytes or more,
 *        256-byte aligned; NULL: a stream-ordered temporary.  One that is
 *        too small is KQ_ERR_LIMIT.
 *
 * A row that attends a place without a valid page is NaN.  max_new <=
 * KQ_MAX_DRAFT.  Queries and probabilities are held as two f16 terms (22
 * bits; queries after scaling a row by a power of two, and with many rows by
 * the fraction of `scale` too, rounded to f32), and so is code * scale, or a
 * probability times its value's scale, where that is formed before the product
 * (what is dropped is below 2^-22 of it, or 2^-39 of the page's largest).
 * Products are exact, sums are f32.  Logits may be as large as f32 holds, as
 * long as scale * q is finite too.  A row that attends an infinity (an f16 key
 * or value past 65504) may be NaN where the formula gives it an infinite value
 * or a weight of zero.
 */
kq_status kq_tree_attention(const kq_kv *kv, const kq_batch *batch, const float *q,
                            int64_t q_stride, int q_heads, const uint64_t *mask, float scale,
                            float *out, void *ws, int64_t ws_bytes, void *stream);

/* Workspace bytes of kq_tree_attention on the current device, from the
 * descriptors' sizes alone, or a negative kq_status. */
int64_t kq_attn_workspace_bytes(const kq_kv *kv, const kq_batch *batch, int q_heads);

/*
 * Verification of drafted tokens, from given random numbers: each sequence's
 * new tokens are a tree, node 0 the last committed token, the others drafts,
 * each after its parent.  p[i] is the target's distribution after node i,
 * q[i] the one node i's children were drawn from.  From cur = 0, r = p[0],
 * z = 1, the children of cur are tried in order of their index, child x of
 * token t being accepted if
 *     u[x] * (q[cur][t] * z) < r[t]
 * (then cur = x, r = p[x], z = 1); otherwise r becomes max(r - z * q[cur],
 * 0) and z its sum (unless that sum is zero: then r and z stay).  After the
 * last child the next token is drawn from r by its running sum with
 * u_next[b].  q NULL: the drafts came without a distribution; a child is
 * tried with u[x] * z < r[t], and a rejected token is taken out of r.  The
 * tokens that come out are distributed as if drawn from p one by one,
 * provided that a node's children are independent draws from q.
 *
 * Products and differences are f32 operations; sums are taken over
 * multiples of 2^-44 (smaller parts are dropped), so that they do not depend
 * on any order: the token is the first x whose running sum passes
 * floor(u * sum), u in multiples of 2^-31.  Probabilities outside 0..1 are
 * taken as the nearer bound, NaN as 0; the same for u, which stays below 1.
 *
 *   start   device int32 [nseq + 1] as in kq_batch; 1..KQ_MAX_DRAFT nodes a
 *           sequence (max_new), one with none gets count 0 and next -1 (with
 *           ntok = 0 all of them; token, parent, p, u and path may be NULL)
 *   token   device int32 [ntok]; a draft outside the vocabulary is rejected
 *           (and nothing is taken out for it)
 *   parent  device int32 [ntok], a node of lower index in the sequence; a
 *           node with another parent is never tried
 *   p, q    device f32 [ntok][vocab], p_stride and q_stride values from row
 *           to row; 4-byte aligned.  vocab 1..KQ_MAX_VOCAB
 *   path    device int32 [ntok]: of each sequence the accepted nodes, 0
 *           first, then -1
 *   count   device int32 [nseq]: accepted nodes, node 0 included
 *   next    device int32 [nseq]
 */
kq_status kq_verify_tree(int nseq, int64_t ntok, int max_new, const int32_t *start,
                         const int32_t *token, const int32_t *parent, const float *p,
                         int64_t p_stride, const float *q, int64_t q_stride, int vocab,
                         const float *u, const float *u_next, int32_t *path, int32_t *count,
                         int32_t *next, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* KQ_DECODE_H */
