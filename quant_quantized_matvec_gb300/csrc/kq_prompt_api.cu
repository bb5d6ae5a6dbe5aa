// kq_prompt_api.cu -- the C ABI of include/kq_prompt.h: argument checks and
// launches.  Checks are pure host logic first, then the pointers' memory, so a
// rejected call enqueues nothing.
#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>

#include "kq_host.h"
#include "kq_prompt_launch.h"
#include "kq_types.cuh"

using kqhost::aligned;
using kqhost::launched;
using kqhost::Pointers;
using kqp::is_type;
using kqp::type_size;

namespace {

constexpr int64_t kMaxCount = 1 << 24;      // tokens
constexpr int64_t kMaxPositions = 1 << 28;  // of a rotary table
constexpr int64_t kMaxStride = 1LL << 32;

// Rows of `row` values, multiples of 16 bytes apart.
bool bad_stride(int64_t stride, int64_t row, int size) {
    return stride < row || stride % (16 / size) != 0 || stride > kMaxStride;
}
int64_t rows_bytes(int64_t n, int64_t stride, int64_t row, int size) {
    return n < 1 ? 0 : size * ((n - 1) * stride + row);
}

// Whether two arrays of n rows meet.  Rows that lie equally far apart may lie
// between each other's (slices of a fused projection).
struct Strided {
    const void *p;
    int64_t stride, row;  // bytes
    int64_t n;
};
bool meet(const Strided &a, const Strided &b) {
    const kqhost::Span x = kqhost::span(a.p, (a.n - 1) * a.stride + a.row);
    const kqhost::Span y = kqhost::span(b.p, (b.n - 1) * b.stride + b.row);
    if (!kqhost::meet(x, y)) return false;
    if (a.stride != b.stride || a.n == 1 || b.n == 1) return true;
    const int64_t d = ((int64_t)(y.lo - x.lo) % a.stride + a.stride) % a.stride;
    return !(d >= a.row && d + b.row <= a.stride);
}

kq_status check_prompt(const kqp::PromptCall &c, int64_t ntok, int64_t nkeys) {
    if (!is_type(c.type)) return KQ_ERR_FORMAT;
    if (c.nseq < 1 || c.nseq > KQ_MAX_SEQS) return KQ_ERR_COUNT;
    if (ntok < 0 || ntok > kMaxCount || nkeys < 0 || nkeys > kMaxCount) return KQ_ERR_NTOK;
    if (c.kv_heads < 1 || c.q_heads < 1 || c.q_heads > KQ_MAX_HEADS || c.q_heads % c.kv_heads != 0 ||
        (c.dim != 64 && c.dim != 128 && c.dim != 256))
        return KQ_ERR_SHAPE;
    return KQ_OK;
}

}  // namespace

extern "C" {

kq_status kq_norm_rope(const kq_norm_part *parts, int n, int type, int out_type, int64_t ntok,
                       int dim, float eps, const int32_t *pos, const float *table,
                       int64_t positions, int rot, int interleaved, void *stream) {
    if (!parts) return KQ_ERR_NULL;
    if (n < 1 || n > KQ_MAX_NORM_PARTS) return KQ_ERR_COUNT;
    if (!is_type(type) || !is_type(out_type) || (type != KQ_F32 && out_type != type))
        return KQ_ERR_FORMAT;
    if (dim < 8 || dim > 1024 || dim % 8 != 0 || !(eps >= 0.f) || !std::isfinite(eps))
        return KQ_ERR_SHAPE;
    if (table && (rot < 8 || rot > dim || rot % 8 != 0 || positions < 1 || positions > kMaxPositions))
        return KQ_ERR_SHAPE;
    const int size = type_size(type), out_size = type_size(out_type);
    kqp::NormArgs a{};
    for (int i = 0; i < n; ++i) {
        const kq_norm_part &p = parts[i];
        if (p.heads < 1 || p.heads > KQ_MAX_HEADS || p.reserved != 0) return KQ_ERR_SHAPE;
        const int64_t row = (int64_t)p.heads * dim;
        if (bad_stride(p.stride, row, size) || bad_stride(p.out_stride, row, out_size))
            return KQ_ERR_SHAPE;
        a.part[i] = p;
    }
    if (ntok < 0 || ntok > kMaxCount) return KQ_ERR_NTOK;
    if (ntok == 0) return KQ_OK;
    for (int i = 0; i < n; ++i)
        if (!parts[i].x || !parts[i].out) return KQ_ERR_NULL;
    if (table && !pos) return KQ_ERR_NULL;
    for (int i = 0; i < n; ++i)
        if (!aligned(parts[i].x, 16) || !aligned(parts[i].out, 16) || !aligned(parts[i].weight, 16))
            return KQ_ERR_ALIGN;
    if (table && (!aligned(table, 16) || !aligned(pos, 4))) return KQ_ERR_ALIGN;
    Pointers mem;
    for (int i = 0; i < n; ++i) {
        const kq_norm_part &p = parts[i];
        const int64_t row = (int64_t)p.heads * dim;
        const Strided out{p.out, p.out_stride * out_size, row * out_size, ntok};
        auto clear = [&](const void *q, int64_t bytes) { return !meet(out, Strided{q, bytes, bytes, 1}); };
        for (int j = 0; j < n; ++j) {
            const kq_norm_part &o = parts[j];
            const int64_t orow = (int64_t)o.heads * dim;
            const bool in_place =
                i == j && o.x == p.out && o.stride == p.out_stride && type == out_type;
            if (!in_place && meet(out, Strided{o.x, o.stride * size, orow * size, ntok}))
                return KQ_ERR_ALIAS;
            if (j < i && meet(out, Strided{o.out, o.out_stride * out_size, orow * out_size, ntok}))
                return KQ_ERR_ALIAS;
            if (o.weight && !clear(o.weight, 4 * dim)) return KQ_ERR_ALIAS;
        }
        if (table && (!clear(table, 4 * positions * rot) || !clear(pos, 4 * ntok))) return KQ_ERR_ALIAS;
        mem.p[mem.np++] = p.x, mem.p[mem.np++] = p.out;
        if (p.weight) mem.p[mem.np++] = p.weight;
    }
    if (table) mem.p[mem.np++] = table, mem.p[mem.np++] = pos;
    const kq_status st = mem.memory();
    if (st != KQ_OK) return st;
    a.ntok = ntok, a.positions = positions, a.pos = pos, a.table = table, a.eps = eps;
    a.dim = dim, a.rot = table ? rot : 0, a.inter = interleaved != 0;
    return launched(kqp::norm_rope(a, n, type, out_type, (cudaStream_t)stream));
}

int64_t kq_prompt_workspace_bytes(int type, int nseq, int64_t ntok, int64_t nkeys, int q_heads,
                                  int kv_heads, int dim) {
    kqp::PromptCall c{};
    c.type = type, c.nseq = nseq, c.q_heads = q_heads, c.kv_heads = kv_heads, c.dim = dim;
    const kq_status st = check_prompt(c, ntok, nkeys);
    if (st != KQ_OK) return -(int64_t)st;
    if (ntok == 0) return 0;
    c.ntok = (int32_t)ntok, c.nkeys = (int32_t)nkeys;
    kqhost::Device dev{};
    const cudaError_t e = kqhost::device(dev);
    if (e != cudaSuccess) return -(int64_t)kqhost::cuda_failed(e);
    const int64_t bytes = kqp::prompt_workspace(c, dev.sms);
    return bytes < 0 ? -(int64_t)KQ_ERR_NTOK : bytes;
}

kq_status kq_prompt_attention(int type, int nseq, int64_t ntok, int64_t nkeys,
                              const int32_t *start, const int32_t *key_start, const void *q,
                              int64_t q_stride, int q_heads, const void *k, int64_t k_stride,
                              const void *v, int64_t v_stride, int kv_heads, int dim, float scale,
                              void *out, void *ws, int64_t ws_bytes, void *stream) {
    kqp::PromptCall c{};
    c.type = type, c.nseq = nseq, c.q_heads = q_heads, c.kv_heads = kv_heads, c.dim = dim;
    c.scale = scale;
    kq_status st = check_prompt(c, ntok, nkeys);
    if (st != KQ_OK) return st;
    if (!key_start && nkeys != ntok) return KQ_ERR_NTOK;
    const int size = type_size(type);
    const int64_t row = (int64_t)q_heads * dim, kv_row = (int64_t)kv_heads * dim;
    if (bad_stride(q_stride, row, size) || bad_stride(k_stride, kv_row, size) ||
        bad_stride(v_stride, kv_row, size) || !std::isfinite(scale))
        return KQ_ERR_SHAPE;
    // (16 bits: the scale's product with log2(e) is one number)
    if (type != KQ_F32 && !std::isfinite(scale * 1.44269504f)) return KQ_ERR_SHAPE;
    if (ntok == 0) return KQ_OK;
    if (!start || !q || !out || (nkeys > 0 && (!k || !v))) return KQ_ERR_NULL;
    if (!aligned(start, 4) || !aligned(key_start, 4) || !aligned(q, 16) || !aligned(k, 16) ||
        !aligned(v, 16) || !aligned(out, 16) || !aligned(ws, 256))
        return KQ_ERR_ALIGN;
    c.start = start, c.key_start = key_start, c.q = q, c.k = k, c.v = v, c.out = out;
    c.q_stride = q_stride, c.k_stride = k_stride, c.v_stride = v_stride;
    c.ntok = (int32_t)ntok, c.nkeys = (int32_t)nkeys;
    kqhost::Device dev{};
    cudaError_t e = kqhost::device(dev);
    if (e != cudaSuccess) return kqhost::cuda_failed(e);
    const int64_t need = kqp::prompt_workspace(c, dev.sms);
    if (need < 0) return KQ_ERR_NTOK;
    if (ws && ws_bytes < need) return KQ_ERR_LIMIT;
    Pointers p;
    p.read(start, 4 * ((int64_t)nseq + 1));
    if (key_start) p.read(key_start, 4 * ((int64_t)nseq + 1));
    p.read(q, rows_bytes(ntok, q_stride, row, size));
    if (nkeys > 0) {
        p.read(k, rows_bytes(nkeys, k_stride, kv_row, size));
        p.read(v, rows_bytes(nkeys, v_stride, kv_row, size));
    }
    p.write(out, ntok * row * size);
    if (ws && ws_bytes > 0) p.write(ws, ws_bytes);
    st = p.check();
    if (st != KQ_OK) return st;
    const cudaStream_t s = (cudaStream_t)stream;
    void *tmp = nullptr;
    if (!ws && need > 0) {
        e = cudaMallocAsync(&tmp, (size_t)need, s);
        if (e != cudaSuccess) return kqhost::cuda_failed(e);
    }
    e = kqp::prompt_attention(c, ws ? ws : tmp, dev.sms, dev.err, dev.wait_ns, s);
    if (tmp) {
        const cudaError_t f = cudaFreeAsync(tmp, s);
        if (e == cudaSuccess) e = f;
    }
    return launched(e);
}

kq_status kq_token_logprobs(int type, int64_t n, int vocab, const void *logits, int64_t stride,
                            const int32_t *token, int top, float *logp, float *entropy,
                            float *top_logp, int32_t *top_token, void *stream) {
    if (!is_type(type)) return KQ_ERR_FORMAT;
    if (n < 0 || n > kMaxCount) return KQ_ERR_NTOK;
    if (vocab < 1 || vocab > KQ_MAX_VOCAB || stride < vocab || stride > kMaxStride || top < 0 ||
        top > KQ_MAX_TOP || top > vocab)
        return KQ_ERR_SHAPE;
    if ((token == nullptr) != (logp == nullptr) && n > 0) return KQ_ERR_NULL;
    if (n == 0) return KQ_OK;
    if (!logits || (top > 0 && (!top_logp || !top_token)) || (!logp && !entropy && top == 0))
        return KQ_ERR_NULL;
    const int size = type_size(type);
    if (!aligned(logits, size) || !aligned(token, 4) || !aligned(logp, 4) || !aligned(entropy, 4) ||
        (top > 0 && (!aligned(top_logp, 4) || !aligned(top_token, 4))))
        return KQ_ERR_ALIGN;
    Pointers p;
    p.read(logits, rows_bytes(n, stride, vocab, size));
    if (token) p.read(token, 4 * n), p.write(logp, 4 * n);
    if (entropy) p.write(entropy, 4 * n);
    if (top > 0) p.write(top_logp, 4 * n * top), p.write(top_token, 4 * n * top);
    const kq_status st = p.check();
    if (st != KQ_OK) return st;
    const kqp::ScoreArgs a{logits, n, stride, token, logp, entropy, top_logp, top_token, vocab, top};
    return launched(kqp::token_logprobs(a, type, (cudaStream_t)stream));
}

}  // extern "C"
