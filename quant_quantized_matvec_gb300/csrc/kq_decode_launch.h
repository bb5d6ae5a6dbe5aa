// kq_decode_launch.h -- launch entry points of the decode-step kernels, called
// by kq_decode_api.cu after it has checked the arguments.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "kq_decode.h"

namespace kqd {

struct Seqs;

cudaError_t rope_table(int64_t positions, int rot, double base, const kq_rope_scaling &sc,
                       float *table, cudaStream_t s);
cudaError_t rope(const float *x, int64_t stride, float *out, int64_t out_stride, int64_t ntok,
                 int heads, int dim, const int32_t *pos, const float *table, int64_t positions,
                 int rot, bool interleaved, bool inverse, cudaStream_t s);

// New keys and values of a step, and how the keys are rotated (table NULL:
// not at all).
struct AppendArgs {
    const float *k, *v;
    int64_t k_stride, v_stride;
    const int32_t *pos;
    const float *table;
    int64_t positions;
    int32_t rot, inter;
};
cudaError_t kv_append(int fmt, int dim, const Seqs &q, const AppendArgs &a, cudaStream_t s);
cudaError_t kv_read(int fmt, int dim, const Seqs &q, float *k, float *v, cudaStream_t s);
cudaError_t kv_move(int fmt, int dim, const Seqs &q, const int32_t *path, const int32_t *count,
                    cudaStream_t s);

// Attention: workspace bytes and the launches.
int64_t attn_workspace(int fmt, int dim, const Seqs &q, int q_heads, int sms);
cudaError_t attn(int fmt, int dim, const Seqs &q, const float *x, int64_t x_stride, int q_heads,
                 const uint64_t *mask, float scale, float *out, void *ws, int sms,
                 unsigned int *err, unsigned long long wait_ns, cudaStream_t s);

struct VerifyArgs {
    const int32_t *start, *token, *parent;
    const float *p, *q, *u, *u_next;
    int64_t p_stride, q_stride;
    int32_t *path, *count, *next;
    int32_t nseq, ntok, max_new, vocab;
};
cudaError_t verify(const VerifyArgs &a, cudaStream_t s);

}  // namespace kqd
