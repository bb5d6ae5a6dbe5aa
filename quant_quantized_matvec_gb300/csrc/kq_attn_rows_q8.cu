// kq_attn_rows_q8.cu -- kq_attn_rows.cuh for KQ_KV_Q8 caches.
#include "kq_attn_rows.cuh"

namespace kqd {
cudaError_t attn_rows_q8(int dim, const AttnArgs &a, int64_t rows, int sms, cudaStream_t s,
                         int64_t *floats) {
    return dim == 64 ? launch_rows<KQ_KV_Q8, 64>(a, rows, sms, s, floats)
                     : launch_rows<KQ_KV_Q8, 128>(a, rows, sms, s, floats);
}
}  // namespace kqd
