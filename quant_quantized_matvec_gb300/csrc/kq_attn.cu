// kq_attn.cu -- kq_tree_attention's launches: the format's kernel
// (kq_attn.cuh) and the workspace it needs.
#include "kq_attn.cuh"

#include <cmath>

namespace kqd {

cudaError_t attn_f16(int dim, const AttnArgs &a, int sms, cudaStream_t s, int64_t *floats);
cudaError_t attn_q8(int dim, const AttnArgs &a, int sms, cudaStream_t s, int64_t *floats);
cudaError_t attn_q4(int dim, const AttnArgs &a, int sms, cudaStream_t s, int64_t *floats);
cudaError_t attn_rows_f16(int dim, const AttnArgs &a, int64_t rows, int sms, cudaStream_t s,
                          int64_t *floats);
cudaError_t attn_rows_q8(int dim, const AttnArgs &a, int64_t rows, int sms, cudaStream_t s,
                         int64_t *floats);
cudaError_t attn_rows_q4(int dim, const AttnArgs &a, int64_t rows, int sms, cudaStream_t s,
                         int64_t *floats);

namespace {
// Rows that a key head of a sequence may have.
int64_t q_rows(const AttnArgs &a) { return (int64_t)a.q.max_new * a.per; }

cudaError_t of_format(int fmt, int dim, const AttnArgs &a, int sms, cudaStream_t s,
                      int64_t *floats) {
    const int64_t rows = q_rows(a);
    // Up to 16 rows fit one block of mma.sync tiles; more are tcgen05's, but for
    // width 256, which its tensor memory does not hold.  Measured, mma.sync /
    // tcgen05, 16 rows (16 sequences of 16384 at most, 2 key heads of 128): 8-bit
    // 56.2 / 72.2 us, 4-bit 58.3 / 69.6; 12 rows 47.6 / 70.2.  f16 goes the same
    // way although 16 rows took 51.2 us with tcgen05 and 59.3 here (12 rows
    // 50.2 / 50.5).
    if (dim <= 128 && rows > 16)
        return fmt == KQ_KV_F16  ? attn_rows_f16(dim, a, rows, sms, s, floats)
               : fmt == KQ_KV_Q8 ? attn_rows_q8(dim, a, rows, sms, s, floats)
                                 : attn_rows_q4(dim, a, rows, sms, s, floats);
    return fmt == KQ_KV_F16  ? attn_f16(dim, a, sms, s, floats)
           : fmt == KQ_KV_Q8 ? attn_q8(dim, a, sms, s, floats)
                             : attn_q4(dim, a, sms, s, floats);
}
}  // namespace

int64_t attn_workspace(int fmt, int dim, const Seqs &q, int q_heads, int sms) {
    AttnArgs a{};
    a.q = q, a.q_heads = q_heads, a.per = q_heads / q.heads;
    int64_t floats = 0;
    of_format(fmt, dim, a, sms, nullptr, &floats);
    // the partial results, and two int4 a CTA (at most four CTAs an SM)
    return (4 * floats + 32 * 4 * (int64_t)sms + 255) / 256 * 256;
}

cudaError_t attn(int fmt, int dim, const Seqs &q, const float *x, int64_t x_stride, int q_heads,
                 const uint64_t *mask, float scale, float *out, void *ws, int sms,
                 unsigned int *err, unsigned long long wait_ns, cudaStream_t s) {
    AttnArgs a{};
    a.q = q;
    a.x = x, a.x_stride = x_stride, a.mask = mask, a.out = out;
    a.part = static_cast<float *>(ws);
    a.err = err, a.wait_ns = wait_ns;
    a.suspend_ns = wait_ns < kq::kSuspendNs ? (uint32_t)wait_ns : kq::kSuspendNs;
    a.q_heads = q_heads, a.per = q_heads / q.heads;
    int e = 0;
    a.scale_m = (float)std::frexp(scale * 1.44269504088896340736, &e);
    a.scale_e = e;
    int64_t floats = 0;
    return of_format(fmt, dim, a, sms, s, &floats);
}

}  // namespace kqd
