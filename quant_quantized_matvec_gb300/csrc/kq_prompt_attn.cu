// kq_prompt_attn.cu -- kq_prompt_attention's launches: what chooses the kernel
// and divides its work, and the kernel that joins the parts of cut keys.
#include "kq_prompt_pairs.cuh"

#include <algorithm>
#include <cmath>

namespace kqp {

cudaError_t prompt_f32(int d, PromptArgs &a, cudaStream_t s);
cudaError_t prompt_f16(int d, PromptArgs &a, cudaStream_t s);
cudaError_t prompt_bf16(int d, PromptArgs &a, cudaStream_t s);

constexpr int kJoinThreads = 256, kJoinRows = 32;

// 32 rows of an item a CTA, a lane each; a warp has some of their values and
// joins the parts in their order.  Rows go out through shared memory.  (A CTA
// an item: 130 us against 8, 40 items of 256 rows of width 128 in 7 parts.)
template <class T, int D>
__global__ void __launch_bounds__(kJoinThreads)
    kq_prompt_join(const __grid_constant__ PromptArgs a, int blocks) {
    constexpr int V = D / (kJoinThreads / 32);  // values of a thread
    __shared__ Item item;
    __shared__ float tile[kJoinRows][D + 1];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    Place from;
    if (w == 0) find_item(a, blockIdx.x, item, lane, from);
    kq::wait_prerequisites();
    __syncthreads();
    const Item it = item;
    if (!it.found) return;
    const float factor = std::is_same<T, float>::value ? 1.f : fabsf(a.scale) * kLog2E;
    const float up = std::is_same<T, float>::value ? 32768.f : 1.f;
    const int rows = blocks * kRows, half = a.tok / blocks;
    // row r's place among the item's tokens and heads; -1: none
    auto place = [&](int r, int &at, int &h) {
        const int t = r % kRows / a.hb;
        h = r % kRows - t * a.hb, at = r / kRows * half + t;
        return t < half && at < it.nt && h < it.nh;
    };
    const int64_t each = (int64_t)rows * (D + 2);
    const float *part = a.part + (int64_t)blockIdx.x * a.splits * each;
    const int r0 = blockIdx.y * kJoinRows;
    const float *m = part + rows * D + r0 + lane, *l = m + rows;
    const float *o = part + (r0 * D + w * V * 32) + lane;
    // (the reference moves as the parts come, by 2^0 most of the time)
    float top = -INFINITY, sum = 0.f, y[V];
#pragma unroll
    for (int e = 0; e < V; ++e) y[e] = 0.f;
    for (int k = 0; k < a.splits; ++k) {
        const float mk = m[k * each], lk = l[k * each];
        float v[V];
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = o[k * each + 32 * e];
        const float now = fmaxf(top, mk);
        const float g = top == now ? 1.f : top == -INFINITY ? 0.f : exp2_fast((top - now) * factor);
        const float f = mk == now ? 1.f : mk == -INFINITY ? 0.f : exp2_fast((mk - now) * factor);
        top = now;
        sum = fmaf(f, lk, sum * g);
#pragma unroll
        for (int e = 0; e < V; ++e) y[e] = fmaf(f, v[e], y[e] * g);
    }
    int at, h;
    const bool on = place(r0 + lane, at, h);
    // (an expired wait left a sum of NaN, also in rows that attend nothing)
    const float inv = on && it.limit(it.tok0 + at) < 0 && sum == 0.f ? 0.f : __fdiv_rn(up, sum);
#pragma unroll
    for (int e = 0; e < V; ++e) tile[lane][w * V + e] = y[e] * inv;
    __syncthreads();
    for (int i = threadIdx.x; i < kJoinRows * (D / 4); i += kJoinThreads) {
        const int r = i / (D / 4), e = 4 * (i % (D / 4));
        if (!place(r0 + r, at, h)) continue;
        store4(static_cast<T *>(a.out) +
                   ((int64_t)(it.first + it.tok0 + at) * a.q_heads + it.hq + h) * D + e,
               make_float4(tile[r][e], tile[r][e + 1], tile[r][e + 2], tile[r][e + 3]));
    }
}

template <class T>
cudaError_t launch_join(const PromptArgs &a, int d, int blocks, cudaStream_t s) {
    const dim3 grid((unsigned)a.items, blocks * kRows / kJoinRows);
    return d == 64    ? launch_early(kq_prompt_join<T, 64>, grid, kJoinThreads, 0, s, a, blocks)
           : d == 128 ? launch_early(kq_prompt_join<T, 128>, grid, kJoinThreads, 0, s, a, blocks)
                      : launch_early(kq_prompt_join<T, 256>, grid, kJoinThreads, 0, s, a, blocks);
}

// Tokens of an item of `blocks` blocks, items at most, and the parts into which
// their keys are cut.
void divide(PromptArgs &a, int blocks, int tile, int sms) {
    a.per = a.q_heads / a.kv_heads;
    a.hb = std::min(a.per, kRows);
    a.hblocks = (a.per + a.hb - 1) / a.hb;
    a.tok = kRows / a.hb * blocks;
    const int64_t runs =
        std::min<int64_t>(a.ntok, (int64_t)a.ntok / a.tok + std::min(a.nseq, a.ntok));
    const int64_t items = runs * a.kv_heads * a.hblocks;
    a.items = (int32_t)std::min<int64_t>(items, 0x7FFFFFFF);
    // The cut that ends first, in tiles: of the longest item, or of rounds of
    // mean ones, each with what a part costs beside its tiles (about 400 keys'
    // time to begin and to end, and as much again to write partial results and
    // join them: figures of 16 bits at width 128).  This number of parts, half and
    // twice as many, on the GPU: 300 tokens behind 32001, 32 / 8 heads, f16 134, 141
    // and 152 us, f32 481, 666 and 513; 16 / 4 heads of 256, bf16 142, 147 and 174,
    // f32 591, 648 and 632; 64 tokens behind 4000, f16 23, 26 and 24.  One token
    // behind 8000 would rather have half as many (bf16 of 256: 30 and 26).  Lengths
    // count by their means: a long one among short ones is cut too little (300
    // behind 32001 beside seven prompts of 16: 380 us).
    a.splits = 1;
    if (items >= 2 * (int64_t)sms) return;
    const double keys = (double)a.nkeys / a.nseq, mine = (double)a.ntok / a.nseq;
    const double most = keys / tile, mean = std::max(keys - mine / 2, 1.0) / tile;
    double best = 1e30;
    for (int n = 1; n <= 32 && (n == 1 || n * 2 <= most); ++n) {
        const double extra = (n > 1 ? 800.0 : 400.0) / tile;
        const double rounds = (double)((items * n + sms - 1) / sms);
        const double cost = std::max(most / n + extra, rounds * (mean / n + extra));
        if (cost < 0.97 * best) best = cost, a.splits = n;
    }
}

namespace {
// Whether the kernel of two blocks takes a call, keys of a tile, blocks.
bool pairs(int type, int d) { return type != KQ_F32 && d <= 128; }
int tile_of(int type, int d) { return pairs(type, d) ? pair_tile(d) : type == KQ_F32 ? f32_tile_tokens(d) : 64; }
int blocks_of(int type, int d) { return pairs(type, d) ? 2 : 1; }

PromptArgs args_of(const PromptCall &c, int sms) {
    PromptArgs a{};
    a.start = c.start, a.kstart = c.key_start;
    a.q = c.q, a.k = c.k, a.v = c.v, a.out = c.out;
    a.q_stride = c.q_stride, a.k_stride = c.k_stride, a.v_stride = c.v_stride;
    a.nseq = c.nseq, a.ntok = c.ntok, a.nkeys = c.nkeys;
    a.q_heads = c.q_heads, a.kv_heads = c.kv_heads, a.scale = c.scale;
    int e = 0;
    a.scale_m = (float)std::frexp(c.scale * 1.44269504088896340736, &e);
    a.scale_e = e;
    divide(a, blocks_of(c.type, c.dim), tile_of(c.type, c.dim), sms);
    return a;
}
}  // namespace

int64_t prompt_workspace(const PromptCall &c, int sms) {
    const PromptArgs a = args_of(c, sms);
    if ((int64_t)a.items * a.splits >= 0x7FFF0000) return -1;  // (numbers go a round past)
    return space_of(a, blocks_of(c.type, c.dim), c.type == KQ_F32, c.dim).bytes;
}

cudaError_t prompt_attention(const PromptCall &c, void *ws, int sms, unsigned int *err,
                             unsigned long long wait_ns, cudaStream_t s) {
    PromptArgs a = args_of(c, sms);
    const int blocks = blocks_of(c.type, c.dim);
    const Space at = space_of(a, blocks, c.type == KQ_F32, c.dim);
    a.tiles = static_cast<uint8_t *>(ws);
    a.info = reinterpret_cast<TileInfo *>(a.tiles + at.info);
    a.powers = reinterpret_cast<TilePowers *>(a.tiles + at.powers);
    a.part = reinterpret_cast<float *>(a.tiles + at.part);
    a.err = err, a.wait_ns = wait_ns;
    a.suspend_ns = wait_ns < kq::kSuspendNs ? (uint32_t)wait_ns : kq::kSuspendNs;
    cudaError_t e = c.type == KQ_F32   ? prompt_f32(c.dim, a, s)
                    : c.type == KQ_F16 ? prompt_f16(c.dim, a, s)
                                       : prompt_bf16(c.dim, a, s);
    if (e != cudaSuccess || a.splits == 1) return e;
    return c.type == KQ_F32   ? launch_join<float>(a, c.dim, blocks, s)
           : c.type == KQ_F16 ? launch_join<__half>(a, c.dim, blocks, s)
                              : launch_join<__nv_bfloat16>(a, c.dim, blocks, s);
}

}  // namespace kqp
