// kq_prompt_f32.cu -- attention of whole prompts, f32.
#include "kq_prompt_attn.cuh"

namespace kqp {
cudaError_t prompt_f32(int d, PromptArgs &a, cudaStream_t s) {
    return d == 64    ? launch_rows<float, 64>(a, s)
           : d == 128 ? launch_rows<float, 128>(a, s)
                      : launch_rows<float, 256>(a, s);
}
}  // namespace kqp
