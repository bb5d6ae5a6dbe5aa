// kq_attn.cu -- attention of new tokens over the paged cache
// (kq_tree_attention).
//
// One CTA per (new token, query head): eight warps take the tokens in turn,
// a lane holding D / 32 values of the head; each warp keeps a running
// maximum, sum and weighted values, which are joined at the end.
#include "kq_decode.cuh"
#include "kq_decode_launch.h"

namespace kqd {

constexpr int kAttnWarps = 8;

template <int FMT, int D>
__device__ __forceinline__ float kv_value(const uint8_t *block, bool value, int t, int e) {
    using L = Kv<FMT, D>;
    const uint8_t *p;
    int bit;
    if (value) {
        p = block + L::v_word(e, t / L::kVPerWord);
        bit = (t % L::kVPerWord) * L::kBits;
    } else {
        p = block + L::k_octet(t, e / 8);
        bit = (e % 8) * L::kBits;
        p += bit / 32 * 4, bit %= 32;
    }
    const uint32_t w = *reinterpret_cast<const uint32_t *>(p);
    if constexpr (FMT == KQ_KV_F16) return __half2float(__ushort_as_half((uint16_t)(w >> bit)));
    const float d = __half2float(*reinterpret_cast<const __half *>(
        block + (value ? L::v_scale(t, e / kGroup) : L::k_scale(t, e / kGroup))));
    return (float)((int)(w << (32 - L::kBits - bit)) >> (32 - L::kBits)) * d;
}

template <int FMT, int D>
__global__ void __launch_bounds__(32 * kAttnWarps)
    kq_attn_kernel(const __grid_constant__ Seqs q, const float *__restrict__ x, int64_t x_stride,
                   int q_heads, const uint64_t *__restrict__ mask, float scale,
                   float *__restrict__ out) {
    using L = Kv<FMT, D>;
    constexpr int N = D / 32;
    __shared__ float sm[kAttnWarps], sl[kAttnWarps], so[kAttnWarps][D];
    const int tok = blockIdx.x, head = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int b = 0;
    Seq s;
    for (; b < q.nseq; ++b) {
        s = seq_of(q, b);
        if (tok >= s.first && tok < s.first + s.n) break;
    }
    if (b == q.nseq) return;
    const int j = tok - s.first;
    uint64_t m = mask ? __ldg(mask + tok) : ~0ull >> (63 - j);
    const int kvh = head / (q_heads / q.heads);
    float qv[N], o[N];
    for (int i = 0; i < N; ++i) {
        qv[i] = x[(int64_t)tok * x_stride + head * D + lane + 32 * i] * scale;
        o[i] = 0.f;
    }
    float top = -INFINITY, sum = 0.f;
    for (int t = warp; t < s.ctx + s.n; t += kAttnWarps) {
        if (t >= s.ctx && !((m >> (t - s.ctx)) & 1)) continue;
        const int64_t page = page_of(q, b, t / kPage);
        float dot = 0.f;
        const uint8_t *block = q.data + (page * q.heads + kvh) * L::kBlock;
        if (page < 0) dot = quiet_nan();
        else
            for (int i = 0; i < N; ++i)
                dot += qv[i] * kv_value<FMT, D>(block, false, t % kPage, lane + 32 * i);
        for (int k = 16; k; k /= 2) dot += __shfl_xor_sync(~0u, dot, k);
        const float now = fmaxf(top, dot);
        const float a = now == -INFINITY ? 1.f : expf(top - now);
        const float p = dot == -INFINITY ? 0.f : expf(dot - now);
        sum = sum * a + p;
        for (int i = 0; i < N; ++i)
            o[i] = o[i] * a +
                   (page < 0 ? p : p * kv_value<FMT, D>(block, true, t % kPage, lane + 32 * i));
        top = now;
    }
    if (lane == 0) sm[warp] = top, sl[warp] = sum;
    for (int i = 0; i < N; ++i) so[warp][lane + 32 * i] = o[i];
    __syncthreads();
    float all = -INFINITY;
    for (int w = 0; w < kAttnWarps; ++w) all = fmaxf(all, sm[w]);
    for (int e = threadIdx.x; e < D; e += 32 * kAttnWarps) {
        float y = 0.f, l = 0.f;
        for (int w = 0; w < kAttnWarps; ++w) {
            const float a = sm[w] == -INFINITY && sl[w] == 0.f ? 0.f : expf(sm[w] - all);
            y += a * so[w][e];
            l += a * sl[w];
        }
        out[((int64_t)tok * q_heads + head) * D + e] = l == 0.f ? 0.f : y / l;
    }
}

int64_t attn_workspace(int, const Seqs &, int, int) { return 0; }

namespace {
template <int FMT, int D>
cudaError_t go(const Seqs &q, const float *x, int64_t x_stride, int q_heads, const uint64_t *mask,
               float scale, float *out, cudaStream_t s) {
    kq_attn_kernel<FMT, D><<<dim3(q.ntok, q_heads), 32 * kAttnWarps, 0, s>>>(
        q, x, x_stride, q_heads, mask, scale, out);
    return cudaGetLastError();
}
}  // namespace

cudaError_t attn(int fmt, int dim, const Seqs &q, const float *x, int64_t x_stride, int q_heads,
                 const uint64_t *mask, float scale, float *out, void *, int, unsigned int *,
                 cudaStream_t s) {
#define KQ_GO(F, D) \
    if (fmt == F && dim == D) return go<F, D>(q, x, x_stride, q_heads, mask, scale, out, s);
    KQ_GO(KQ_KV_F16, 64) KQ_GO(KQ_KV_F16, 128) KQ_GO(KQ_KV_F16, 256)
    KQ_GO(KQ_KV_Q8, 64) KQ_GO(KQ_KV_Q8, 128) KQ_GO(KQ_KV_Q8, 256)
    KQ_GO(KQ_KV_Q4, 64) KQ_GO(KQ_KV_Q4, 128) KQ_GO(KQ_KV_Q4, 256)
#undef KQ_GO
    return cudaErrorInvalidValue;
}

}  // namespace kqd
