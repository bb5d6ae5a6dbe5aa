// kq_decode_api.cu -- the C ABI of include/kq_decode.h: argument checks and
// launches.  Checks are pure host logic first, then the pointers' memory, so
// a rejected call enqueues nothing.
#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>

#include "kq_decode.cuh"
#include "kq_decode_launch.h"
#include "kq_host.h"

using kqhost::meet;
using kqhost::Span;
using kqhost::span;

namespace {

constexpr int64_t kMaxCount = 1 << 24;      // tokens, pages of a table, positions of a step
constexpr int64_t kMaxPositions = 1 << 28;  // of a rotary table
constexpr int64_t kMaxStride = 1LL << 32;

bool aligned(const void *p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

// Pointers of a call, for the alias and memory checks.
struct Pointers {
    Span in[12], out[4];
    const void *p[16];
    int ni = 0, no = 0, np = 0;
    void read(const void *q, int64_t bytes) { in[ni++] = span(q, bytes), p[np++] = q; }
    void write(const void *q, int64_t bytes) { out[no++] = span(q, bytes), p[np++] = q; }
    kq_status check() const {
        for (int i = 0; i < no; ++i) {
            for (int j = 0; j < ni; ++j)
                if (meet(out[i], in[j])) return KQ_ERR_ALIAS;
            for (int j = 0; j < i; ++j)
                if (meet(out[i], out[j])) return KQ_ERR_ALIAS;
        }
        int dev = 0;
        const cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return kqhost::cuda_failed(e);
        for (int i = 0; i < np; ++i) {
            const kq_status s = kqhost::on_device(p[i], dev);
            if (s != KQ_OK) return s;
        }
        return KQ_OK;
    }
};

kq_status launched(cudaError_t e) { return e == cudaSuccess ? KQ_OK : kqhost::cuda_failed(e); }

kq_status check_kv(const kq_kv *kv) {
    if (!kv) return KQ_ERR_NULL;
    if (kv->fmt != KQ_KV_F16 && kv->fmt != KQ_KV_Q8 && kv->fmt != KQ_KV_Q4) return KQ_ERR_FORMAT;
    if (kv->kv_heads < 1 || kv->kv_heads > KQ_MAX_HEADS || kv->reserved != 0 ||
        (kv->head_dim != 64 && kv->head_dim != 128 && kv->head_dim != 256) || kv->pages < 1 ||
        kv->pages > 0x7FFFFFFF)
        return KQ_ERR_SHAPE;
    if (!kv->data) return KQ_ERR_NULL;
    if (!aligned(kv->data, 16)) return KQ_ERR_ALIGN;
    return KQ_OK;
}

kq_status check_batch(const kq_batch *b, int most) {
    if (!b) return KQ_ERR_NULL;
    if (b->nseq < 1 || b->nseq > KQ_MAX_SEQS) return KQ_ERR_COUNT;
    if (b->ntok < 0 || b->ntok > kMaxCount || b->max_new < 1 || b->max_new > most)
        return KQ_ERR_NTOK;
    if (b->max_pages < 1 || b->max_pages > kMaxCount) return KQ_ERR_SHAPE;
    if (!b->start || !b->ctx || !b->pages) return KQ_ERR_NULL;
    if (!aligned(b->start, 4) || !aligned(b->ctx, 4) || !aligned(b->pages, 4)) return KQ_ERR_ALIGN;
    return KQ_OK;
}

int64_t kv_bytes(const kq_kv *kv) {
    return kq_kv_page_bytes(kv->fmt, kv->kv_heads, kv->head_dim) * kv->pages;
}
void read_batch(Pointers &p, const kq_batch *b) {
    p.read(b->start, 4 * ((int64_t)b->nseq + 1));
    p.read(b->ctx, 4 * (int64_t)b->nseq);
    p.read(b->pages, 4 * b->nseq * b->max_pages);
}
kqd::Seqs seqs_of(const kq_kv *kv, const kq_batch *b) {
    kqd::Seqs q;
    q.data = static_cast<uint8_t *>(kv->data);
    q.npages = kv->pages;
    q.start = b->start, q.ctx = b->ctx, q.table = b->pages;
    q.max_pages = b->max_pages;
    q.nseq = b->nseq, q.max_new = b->max_new, q.heads = kv->kv_heads;
    q.ntok = (int32_t)b->ntok;
    return q;
}

// Bytes from the first to the last value of n rows of `row` f32 values.
int64_t rows_bytes(int64_t n, int64_t stride, int64_t row) { return 4 * ((n - 1) * stride + row); }
bool bad_stride(int64_t stride, int64_t row) {
    return stride < row || stride % 4 != 0 || stride > kMaxStride;
}
bool bad_rot(int rot, int64_t positions) {
    return rot < 8 || rot > 1024 || rot % 8 != 0 || positions < 1 || positions > kMaxPositions;
}

}  // namespace

extern "C" {

int64_t kq_kv_page_bytes(int fmt, int kv_heads, int head_dim) {
    if ((fmt != KQ_KV_F16 && fmt != KQ_KV_Q8 && fmt != KQ_KV_Q4) || kv_heads < 1 ||
        kv_heads > KQ_MAX_HEADS || (head_dim != 64 && head_dim != 128 && head_dim != 256))
        return -1;
    return kqd::kv_block_bytes(fmt, head_dim) * kv_heads;
}

kq_status kq_rope_table(int64_t positions, int rot, double base, const kq_rope_scaling *scaling,
                        float *table, void *stream) {
    kq_rope_scaling sc{};
    sc.magnitude = 1.0;
    if (scaling) sc = *scaling;
    if (bad_rot(rot, positions) || !std::isfinite(base) || base <= 0) return KQ_ERR_SHAPE;
    if (sc.kind < 0 || sc.kind > 3 || !std::isfinite(sc.magnitude)) return KQ_ERR_SHAPE;
    if (sc.kind >= 1 && !(std::isfinite(sc.factor) && sc.factor > 0)) return KQ_ERR_SHAPE;
    if (sc.kind == 3 && !(sc.orig >= 1 && std::isfinite(sc.fast) && sc.slow >= 0 && sc.fast > sc.slow))
        return KQ_ERR_SHAPE;
    if (!table) return KQ_ERR_NULL;
    if (!aligned(table, 16)) return KQ_ERR_ALIGN;
    Pointers p;
    p.write(table, 4 * positions * rot);
    const kq_status st = p.check();
    if (st != KQ_OK) return st;
    return launched(kqd::rope_table(positions, rot, base, sc, table, (cudaStream_t)stream));
}

kq_status kq_rope(const float *x, int64_t stride, float *out, int64_t out_stride, int64_t ntok,
                  int heads, int dim, const int32_t *pos, const float *table, int64_t positions,
                  int rot, int interleaved, int inverse, void *stream) {
    if (heads < 1 || heads > KQ_MAX_HEADS || dim < 8 || dim > 1024 || dim % 8 != 0 ||
        bad_rot(rot, positions) || rot > dim)
        return KQ_ERR_SHAPE;
    const int64_t row = (int64_t)heads * dim;
    if (bad_stride(stride, row) || bad_stride(out_stride, row)) return KQ_ERR_SHAPE;
    if (ntok < 0 || ntok > kMaxCount) return KQ_ERR_NTOK;
    if (ntok == 0) return KQ_OK;
    if (!x || !out || !pos || !table) return KQ_ERR_NULL;
    if (!aligned(x, 16) || !aligned(out, 16) || !aligned(table, 16) || !aligned(pos, 4))
        return KQ_ERR_ALIGN;
    Pointers p;
    const bool in_place = x == out && stride == out_stride;
    if (!in_place) p.read(x, rows_bytes(ntok, stride, row));
    p.read(pos, 4 * ntok);
    p.read(table, 4 * positions * rot);
    p.write(out, rows_bytes(ntok, out_stride, row));
    const kq_status st = p.check();
    if (st != KQ_OK) return st;
    return launched(kqd::rope(x, stride, out, out_stride, ntok, heads, dim, pos, table, positions,
                              rot, interleaved != 0, inverse != 0, (cudaStream_t)stream));
}

kq_status kq_kv_append(const kq_kv *kv, const kq_batch *batch, const float *k, int64_t k_stride,
                       const float *v, int64_t v_stride, const int32_t *pos, const float *table,
                       int64_t positions, int rot, int interleaved, void *stream) {
    kq_status st = check_kv(kv);
    if (st == KQ_OK) st = check_batch(batch, (int)kMaxCount);
    if (st != KQ_OK) return st;
    const int64_t row = (int64_t)kv->kv_heads * kv->head_dim;
    if (bad_stride(k_stride, row) || bad_stride(v_stride, row)) return KQ_ERR_SHAPE;
    if (table && (bad_rot(rot, positions) || rot > kv->head_dim)) return KQ_ERR_SHAPE;
    if (batch->ntok == 0) return KQ_OK;
    if (!k || !v || (table && !pos)) return KQ_ERR_NULL;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(table, 16) || (table && !aligned(pos, 4)))
        return KQ_ERR_ALIGN;
    Pointers p;
    read_batch(p, batch);
    p.read(k, rows_bytes(batch->ntok, k_stride, row));
    p.read(v, rows_bytes(batch->ntok, v_stride, row));
    if (table) {
        p.read(pos, 4 * batch->ntok);
        p.read(table, 4 * positions * rot);
    }
    p.write(kv->data, kv_bytes(kv));
    st = p.check();
    if (st != KQ_OK) return st;
    const kqd::AppendArgs a{k, v, k_stride, v_stride, pos, table, positions, rot, interleaved != 0};
    return launched(kqd::kv_append(kv->fmt, kv->head_dim, seqs_of(kv, batch), a, (cudaStream_t)stream));
}

kq_status kq_kv_read(const kq_kv *kv, const kq_batch *batch, float *k, float *v, void *stream) {
    kq_status st = check_kv(kv);
    if (st == KQ_OK) st = check_batch(batch, (int)kMaxCount);
    if (st != KQ_OK) return st;
    if (batch->ntok == 0) return KQ_OK;
    if (!k && !v) return KQ_ERR_NULL;
    if (!aligned(k, 16) || !aligned(v, 16)) return KQ_ERR_ALIGN;
    Pointers p;
    read_batch(p, batch);
    p.read(kv->data, kv_bytes(kv));
    const int64_t bytes = 4 * batch->ntok * kv->kv_heads * kv->head_dim;
    if (k) p.write(k, bytes);
    if (v) p.write(v, bytes);
    st = p.check();
    if (st != KQ_OK) return st;
    return launched(kqd::kv_read(kv->fmt, kv->head_dim, seqs_of(kv, batch), k, v, (cudaStream_t)stream));
}

kq_status kq_kv_move(const kq_kv *kv, const kq_batch *batch, const int32_t *path,
                     const int32_t *count, void *stream) {
    kq_status st = check_kv(kv);
    if (st == KQ_OK) st = check_batch(batch, KQ_MAX_DRAFT);
    if (st != KQ_OK) return st;
    if (batch->ntok == 0) return KQ_OK;
    if (!path || !count) return KQ_ERR_NULL;
    if (!aligned(path, 4) || !aligned(count, 4)) return KQ_ERR_ALIGN;
    Pointers p;
    read_batch(p, batch);
    p.read(path, 4 * batch->ntok);
    p.read(count, 4 * (int64_t)batch->nseq);
    p.write(kv->data, kv_bytes(kv));
    st = p.check();
    if (st != KQ_OK) return st;
    return launched(kqd::kv_move(kv->fmt, kv->head_dim, seqs_of(kv, batch), path, count,
                                 (cudaStream_t)stream));
}

int64_t kq_attn_workspace_bytes(const kq_kv *kv, const kq_batch *batch, int q_heads) {
    kq_status st = check_kv(kv);
    if (st == KQ_OK) st = check_batch(batch, KQ_MAX_DRAFT);
    if (st == KQ_OK && (q_heads < 1 || q_heads > KQ_MAX_HEADS || q_heads % kv->kv_heads != 0))
        st = KQ_ERR_SHAPE;
    if (st != KQ_OK) return -(int64_t)st;
    kqhost::Device dev{};
    const cudaError_t e = kqhost::device(dev);
    if (e != cudaSuccess) return -(int64_t)kqhost::cuda_failed(e);
    return kqd::attn_workspace(kv->fmt, kv->head_dim, seqs_of(kv, batch), q_heads, dev.sms);
}

kq_status kq_tree_attention(const kq_kv *kv, const kq_batch *batch, const float *q,
                            int64_t q_stride, int q_heads, const uint64_t *mask, float scale,
                            float *out, void *ws, int64_t ws_bytes, void *stream) {
    kq_status st = check_kv(kv);
    if (st == KQ_OK) st = check_batch(batch, KQ_MAX_DRAFT);
    if (st != KQ_OK) return st;
    if (q_heads < 1 || q_heads > KQ_MAX_HEADS || q_heads % kv->kv_heads != 0) return KQ_ERR_SHAPE;
    const int64_t row = (int64_t)q_heads * kv->head_dim;
    if (bad_stride(q_stride, row) || !std::isfinite(scale)) return KQ_ERR_SHAPE;
    if (batch->ntok == 0) return KQ_OK;
    if (!q || !out) return KQ_ERR_NULL;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(mask, 8) || !aligned(ws, 256))
        return KQ_ERR_ALIGN;
    kqhost::Device dev{};
    cudaError_t e = kqhost::device(dev);
    if (e != cudaSuccess) return kqhost::cuda_failed(e);
    const kqd::Seqs seqs = seqs_of(kv, batch);
    const int64_t need = kqd::attn_workspace(kv->fmt, kv->head_dim, seqs, q_heads, dev.sms);
    if (ws && ws_bytes < need) return KQ_ERR_LIMIT;
    Pointers p;
    read_batch(p, batch);
    p.read(kv->data, kv_bytes(kv));
    p.read(q, rows_bytes(batch->ntok, q_stride, row));
    if (mask) p.read(mask, 8 * batch->ntok);
    p.write(out, 4 * batch->ntok * row);
    if (ws) p.write(ws, ws_bytes);
    st = p.check();
    if (st != KQ_OK) return st;
    const cudaStream_t s = (cudaStream_t)stream;
    void *tmp = nullptr;
    if (!ws && need > 0) {
        e = cudaMallocAsync(&tmp, (size_t)need, s);
        if (e != cudaSuccess) return kqhost::cuda_failed(e);
    }
    e = kqd::attn(kv->fmt, kv->head_dim, seqs, q, q_stride, q_heads, mask, scale, out,
                  ws ? ws : tmp, dev.sms, dev.err, dev.wait_ns, s);
    if (tmp) {
        const cudaError_t f = cudaFreeAsync(tmp, s);
        if (e == cudaSuccess) e = f;
    }
    return launched(e);
}

kq_status kq_verify_tree(int nseq, int64_t ntok, int max_new, const int32_t *start,
                         const int32_t *token, const int32_t *parent, const float *p,
                         int64_t p_stride, const float *q, int64_t q_stride, int vocab,
                         const float *u, const float *u_next, int32_t *path, int32_t *count,
                         int32_t *next, void *stream) {
    if (nseq < 1 || nseq > KQ_MAX_SEQS) return KQ_ERR_COUNT;
    if (ntok < 0 || ntok > kMaxCount || max_new < 1 || max_new > KQ_MAX_DRAFT) return KQ_ERR_NTOK;
    if (vocab < 1 || vocab > KQ_MAX_VOCAB || p_stride < vocab || p_stride > kMaxStride ||
        (q && (q_stride < vocab || q_stride > kMaxStride)))
        return KQ_ERR_SHAPE;
    // (without nodes token, parent, p, u and path have no elements to point at)
    if (!start || !u_next || !count || !next ||
        (ntok > 0 && (!token || !parent || !p || !u || !path)))
        return KQ_ERR_NULL;
    const void *four[] = {start, token, parent, p, q, u, u_next, path, count, next};
    for (const void *a : four)
        if (!aligned(a, 4)) return KQ_ERR_ALIGN;
    int devices = 0;
    if (ntok == 0 && (cudaGetDeviceCount(&devices) != cudaSuccess || devices == 0)) {
        cudaGetLastError();
        return KQ_OK;  // no memory that a result could be written to
    }
    Pointers a;
    a.read(start, 4 * ((int64_t)nseq + 1));
    if (ntok > 0) {
        a.read(token, 4 * ntok);
        a.read(parent, 4 * ntok);
        a.read(p, rows_bytes(ntok, p_stride, vocab));
        if (q) a.read(q, rows_bytes(ntok, q_stride, vocab));
        a.read(u, 4 * ntok);
        a.write(path, 4 * ntok);
    }
    a.read(u_next, 4 * (int64_t)nseq);
    a.write(count, 4 * (int64_t)nseq);
    a.write(next, 4 * (int64_t)nseq);
    const kq_status st = a.check();
    if (st != KQ_OK) return st;
    const kqd::VerifyArgs v{start, token, parent, p, q, u, u_next, p_stride, q_stride,
                            path, count, next, nseq, (int32_t)ntok, max_new, vocab};
    return launched(kqd::verify(v, (cudaStream_t)stream));
}

}  // extern "C"
