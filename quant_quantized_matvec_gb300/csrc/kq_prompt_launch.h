// kq_prompt_launch.h -- launch entry points of the prompt's kernels, called by
// kq_prompt_api.cu after it has checked the arguments.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "kq_prompt.h"

namespace kqp {

struct NormArgs {
    kq_norm_part part[KQ_MAX_NORM_PARTS];
    int32_t upto[KQ_MAX_NORM_PARTS];  // runs of a token's heads up to and with each part
    int64_t ntok, positions;
    const int32_t *pos;
    const float *table;  // (NULL: no rotation, rot 0)
    float eps;
    int32_t runs, dim, rot, inter;
};
// (sets the runs: upto and runs)
cudaError_t norm_rope(NormArgs &a, int parts, int type, int out_type, cudaStream_t s);

struct ScoreArgs {
    const void *x;
    int64_t n, stride;
    const int32_t *token;
    float *logp, *entropy, *top_logp;
    int32_t *top_token;
    int32_t vocab, top;
};
cudaError_t token_logprobs(const ScoreArgs &a, int type, cudaStream_t s);

// A kq_prompt_attention call: its workspace bytes (-1: too many items), and its
// launches.
struct PromptCall {
    const int32_t *start, *key_start;
    const void *q, *k, *v;
    void *out;
    int64_t q_stride, k_stride, v_stride;
    int32_t type, nseq, ntok, nkeys, q_heads, kv_heads, dim;
    float scale;
};
int64_t prompt_workspace(const PromptCall &c, int sms);
cudaError_t prompt_attention(const PromptCall &c, void *ws, int sms, unsigned int *err,
                             unsigned long long wait_ns, cudaStream_t s);

}  // namespace kqp
