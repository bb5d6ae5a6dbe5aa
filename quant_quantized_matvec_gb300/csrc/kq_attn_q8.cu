// kq_attn_q8.cu -- kq_attn.cuh for KQ_KV_Q8 caches.
#include "kq_attn.cuh"

namespace kqd {
cudaError_t attn_q8(int dim, const AttnArgs &a, int sms, cudaStream_t s, int64_t *floats) {
    return attn_format<KQ_KV_Q8>(dim, a, sms, s, floats);
}
}  // namespace kqd
