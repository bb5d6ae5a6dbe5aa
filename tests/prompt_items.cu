// prompt_items.cu -- how the prompt's attention finds the items of numbers that
// come in any order (test_prompt_items_gpu.py): the walk and first_found as the
// kernels have them, with numbers from an array.
#include "kq_prompt_attn.cuh"

namespace {

// The numbers' items in their order: number, sequence, first token, tokens, key
// head, first head, keys; then a number of -1.
__global__ void order_kernel(const __grid_constant__ kqp::PromptArgs a, const int32_t *numbers, int n, int32_t *out) {
    __shared__ kqp::Item it;
    kqp::Place place;
    const int lane = threadIdx.x;
    int next = 0, rows = 0;
    auto given = [&]() { return next < n ? numbers[next++] : -1; };
    auto find = [&](int u) { return kqp::find_item(a, u / a.splits, it, lane, place); };
    while (true) {
        const int u = kqp::first_found(given, find);
        if (lane == 0) {
            int32_t *to = out + 7 * rows;
            to[0] = u;
            if (u >= 0)
                to[1] = it.seq, to[2] = it.tok0, to[3] = it.nt, to[4] = it.head, to[5] = it.hq, to[6] = it.keys();
        }
        __syncwarp();
        if (u < 0) return;
        ++rows;
    }
}

}  // namespace

// out [n + 1][7]; everything on the device.  Returns a CUDA error code.
extern "C" int prompt_items(const int32_t *start, int nseq, int ntok, int tok, int kv_heads, int per, int hb,
                            int splits, const int32_t *numbers, int n, int32_t *out) {
    kqp::PromptArgs a{};
    a.start = start, a.nseq = nseq, a.ntok = a.nkeys = ntok, a.tok = tok, a.kv_heads = kv_heads;
    a.per = per, a.hb = hb, a.hblocks = (per + hb - 1) / hb, a.splits = splits;
    order_kernel<<<1, 32>>>(a, numbers, n, out);
    const cudaError_t e = cudaGetLastError();
    return (int)(e != cudaSuccess ? e : cudaDeviceSynchronize());
}
