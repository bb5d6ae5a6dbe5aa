// kq_prompt_bf16.cu -- attention of whole prompts, bf16.
#include "kq_prompt_pairs.cuh"

namespace kqp {
cudaError_t prompt_bf16(int d, PromptArgs &a, cudaStream_t s) {
    return d == 64    ? launch_pairs<__nv_bfloat16, 64>(a, s)
           : d == 128 ? launch_pairs<__nv_bfloat16, 128>(a, s)
                      : launch_rows<__nv_bfloat16, 256>(a, s);
}
}  // namespace kqp
