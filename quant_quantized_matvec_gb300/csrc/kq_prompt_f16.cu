// kq_prompt_f16.cu -- attention of whole prompts, f16.
#include "kq_prompt_pairs.cuh"

namespace kqp {
cudaError_t prompt_f16(int d, PromptArgs &a, cudaStream_t s) {
    return d == 64    ? launch_pairs<__half, 64>(a, s)
           : d == 128 ? launch_pairs<__half, 128>(a, s)
                      : launch_rows<__half, 256>(a, s);
}
}  // namespace kqp
