// kq_attn_f16.cu -- kq_attn.cuh for KQ_KV_F16 caches.
#include "kq_attn.cuh"

namespace kqd {
cudaError_t attn_f16(int dim, const AttnArgs &a, int sms, cudaStream_t s, int64_t *floats) {
    return attn_format<KQ_KV_F16>(dim, a, sms, s, floats);
}
}  // namespace kqd
