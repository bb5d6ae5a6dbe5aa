// kq_prompt_attn.cu -- kq_prompt_attention's launches: what chooses the kernel
// and divides its work, and the kernel that joins the parts of cut keys.
#include "kq_prompt_attn.cuh"

#include <algorithm>

namespace kqp {

cudaError_t prompt_f32(int d, PromptArgs &a, cudaStream_t s);
cudaError_t prompt_f16(int d, PromptArgs &a, cudaStream_t s);
cudaError_t prompt_bf16(int d, PromptArgs &a, cudaStream_t s);

constexpr int kJoinThreads = 256;

// One CTA per item: its rows' parts in their order.
template <class T>
__global__ void __launch_bounds__(kJoinThreads)
    kq_prompt_join(const __grid_constant__ PromptArgs a, int d, int rows) {
    __shared__ Item item;
    if (threadIdx.x < 32) find_item(a, blockIdx.x, item, threadIdx.x);
    kq::wait_prerequisites();
    __syncthreads();
    const Item it = item;
    if (!it.found) return;
    const float factor = std::is_same<T, float>::value ? 1.f : fabsf(a.scale) * kLog2E;
    const float up = std::is_same<T, float>::value ? 32768.f : 1.f;
    const int64_t each = (int64_t)rows * (d + 2);
    const float *part = a.part + (int64_t)blockIdx.x * a.splits * each;
    for (int i = threadIdx.x; i < rows * (d / 4); i += kJoinThreads) {
        const int r = i / (d / 4), e = 4 * (i % (d / 4));
        int tok, h;
        if (!it.row(a.hb, r, tok, h)) continue;
        const float *m = part + rows * d + r, *l = m + rows;
        float top = -INFINITY;
        for (int k = 0; k < a.splits; ++k) top = fmaxf(top, m[k * each]);
        float sum = 0.f;
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < a.splits; ++k) {
            const float mk = m[k * each];
            const float f = mk == top ? 1.f : mk == -INFINITY ? 0.f : exp2_fast((mk - top) * factor);
            const float4 v = *reinterpret_cast<const float4 *>(part + k * each + r * d + e);
            sum = fmaf(f, l[k * each], sum);
            y.x = fmaf(f, v.x, y.x), y.y = fmaf(f, v.y, y.y);
            y.z = fmaf(f, v.z, y.z), y.w = fmaf(f, v.w, y.w);
        }
        // (an expired wait left a sum of NaN, also in rows that attend nothing)
        const float inv = it.limit(tok) < 0 && sum == 0.f ? 0.f : __fdiv_rn(up, sum);
        store4(static_cast<T *>(a.out) + ((int64_t)(it.first + tok) * a.q_heads + it.hq + h) * d + e,
               make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv));
    }
}

// Tokens of an item, items at most, and parts of the keys where items are few.
void divide(PromptArgs &a, int rows, int tile, int sms) {
    a.per = a.q_heads / a.kv_heads;
    a.hb = std::min(a.per, rows);
    a.hblocks = (a.per + a.hb - 1) / a.hb;
    a.tok = rows / a.hb;
    const int64_t blocks =
        std::min<int64_t>(a.ntok, (int64_t)a.ntok / a.tok + std::min(a.nseq, a.ntok));
    const int64_t items = blocks * a.kv_heads * a.hblocks;
    a.items = (int32_t)std::min<int64_t>(items, 0x7FFFFFFF);
    // each part has four tiles or more (of a sequence of mean length)
    const int64_t tiles = (int64_t)a.nkeys / a.nseq / tile;
    a.splits = (int32_t)std::max<int64_t>(1, std::min<int64_t>(sms / std::max(a.items, 1), tiles / 4));
}

namespace {
int rows_of(int type, int d) { return kRows; }
int tile_of(int type, int d) { return type == KQ_F32 ? f32_tile_tokens(d) : 64; }

PromptArgs args_of(const PromptCall &c, int sms) {
    PromptArgs a{};
    a.start = c.start, a.kstart = c.key_start;
    a.q = c.q, a.k = c.k, a.v = c.v, a.out = c.out;
    a.q_stride = c.q_stride, a.k_stride = c.k_stride, a.v_stride = c.v_stride;
    a.nseq = c.nseq, a.ntok = c.ntok, a.nkeys = c.nkeys;
    a.q_heads = c.q_heads, a.kv_heads = c.kv_heads, a.scale = c.scale;
    divide(a, rows_of(c.type, c.dim), tile_of(c.type, c.dim), sms);
    return a;
}
}  // namespace

int64_t prompt_workspace(const PromptCall &c, int sms) {
    const PromptArgs a = args_of(c, sms);
    if ((int64_t)a.items * a.splits >= 0x7FFFFFFF) return -1;
    return space_of(a, c.type == KQ_F32, c.dim).bytes;
}

cudaError_t prompt_attention(const PromptCall &c, void *ws, int sms, unsigned int *err,
                             unsigned long long wait_ns, cudaStream_t s) {
    PromptArgs a = args_of(c, sms);
    const Space at = space_of(a, c.type == KQ_F32, c.dim);
    a.tiles = static_cast<uint8_t *>(ws);
    a.info = reinterpret_cast<TileInfo *>(a.tiles + at.info);
    a.part = reinterpret_cast<float *>(a.tiles + at.part);
    a.err = err, a.wait_ns = wait_ns;
    a.suspend_ns = wait_ns < kq::kSuspendNs ? (uint32_t)wait_ns : kq::kSuspendNs;
    cudaError_t e = c.type == KQ_F32   ? prompt_f32(c.dim, a, s)
                    : c.type == KQ_F16 ? prompt_f16(c.dim, a, s)
                                       : prompt_bf16(c.dim, a, s);
    if (e != cudaSuccess || a.splits == 1) return e;
    const dim3 grid((unsigned)a.items);
    const int rows = rows_of(c.type, c.dim);
    return c.type == KQ_F32 ? launch_early(kq_prompt_join<float>, grid, kJoinThreads, 0, s, a, c.dim, rows)
           : c.type == KQ_F16
               ? launch_early(kq_prompt_join<__half>, grid, kJoinThreads, 0, s, a, c.dim, rows)
               : launch_early(kq_prompt_join<__nv_bfloat16>, grid, kJoinThreads, 0, s, a, c.dim, rows);
}

}  // namespace kqp
