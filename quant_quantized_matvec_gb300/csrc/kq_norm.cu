// kq_norm.cu -- norms of heads and their rotary positions in one pass.
//
// A head is a group of G lanes, the power of two that gives a lane 8 values
// (or up to 32 in heads wider than 256): four pairs of the rotation, as in
// kq_rope.cu, or eight values that are not turned.  The squares' sum goes
// round the group by shuffles, so x is read once and kept in registers.
// Queries and keys are one launch: a head's number says which tensor it is of.
//
// Bound by memory: 4 + 4 bytes a value in f32, 4 + 2 to 16 bits.  8191 tokens of
// 40 heads of 128, f32 to bf16, 64 values turned: 42.4 us, 88% of the copy rate;
// one token of 34 heads: 2.0 us.  (Weights, cos and sin fetched ahead of the
// values' sums: 67 us, as fewer warps fit.)
#include "kq_decode.cuh"
#include "kq_prompt_launch.h"
#include "kq_types.cuh"

namespace kqp {

using kqd::quiet_nan;
using kqd::rot_a;
using kqd::rot_b;

constexpr int kNormThreads = 128;

// The factor of the values, (mean + eps)^-1/2, where f32 holds neither the
// squares nor their sum: values are scaled by a power of two first.  (All
// lanes of a warp come here together; `group` of them share a head.)
template <int N>
__device__ __forceinline__ float scaled_factor(const float (&v)[N], int group, int dim, float eps) {
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) top = fmaxf(top, fabsf(v[i]));
    for (int o = group / 2; o; o /= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    // 2^-e: `top` to about 1 (with an eps, tiny values need not come that far)
    const int e = min(max((int)(__float_as_uint(top) >> 23 & 255) - 127, eps > 0.f ? -60 : -126), 126);
    const float down = __uint_as_float((uint32_t)(127 - e) << 23);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) sum = fmaf(v[i] * down, v[i] * down, sum);
    for (int o = group / 2; o; o /= 2) sum += __shfl_xor_sync(~0u, sum, o);
    return __fdiv_rn(down, __fsqrt_rn(__fdiv_rn(sum, (float)dim) + eps * down * down));
}

// U: units of eight values of a lane; H: heads that a group of lanes goes
// through, of one tensor and token.
template <class TI, class TO, int U, int H>
__global__ void __launch_bounds__(kNormThreads)
    kq_norm_kernel(const __grid_constant__ NormArgs a, int log2_group, int wide) {
    const int group = 1 << log2_group, lane = threadIdx.x & (group - 1);
    const int64_t i = ((int64_t)blockIdx.x * kNormThreads + threadIdx.x) >> log2_group;
    const int64_t all = a.ntok * a.runs;
    const int64_t it = i < all ? i : all - 1;  // (lanes past the end take part in the shuffles)
    int64_t t;
    int h;
    if (wide) {
        t = it / a.runs, h = (int)(it - t * a.runs);
    } else {
        const uint32_t q = (uint32_t)it / (uint32_t)a.runs;
        t = q, h = (int)((uint32_t)it - q * (uint32_t)a.runs);
    }
    int p = 0;
    while (h >= a.upto[p]) ++p;
    if (p) h -= a.upto[p - 1];
    const kq_norm_part &part = a.part[p];
    h *= H;
    const int heads = min(H, part.heads - h);
    const TI *x = static_cast<const TI *>(part.x) + t * part.stride + (int64_t)h * a.dim;
    TO *out = static_cast<TO *>(part.out) + t * part.out_stride + (int64_t)h * a.dim;
    const int units = a.dim / 8, turned = a.rot / 8;
    const int pos = a.table ? __ldg(a.pos + t) : 0;

    // values of a unit: two runs of four, pairs of the rotation where it turns
    auto run0 = [&](int u) { return u < turned && !a.inter ? 4 * u : 8 * u; };
    auto run1 = [&](int u) { return u < turned && !a.inter ? 4 * u + a.rot / 2 : 8 * u + 4; };
    float v[H][8 * U];
#pragma unroll
    for (int n = 0; n < H; ++n)
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int u = lane + k * group;
            float4 v0 = make_float4(0.f, 0.f, 0.f, 0.f), v1 = v0;
            if (u < units && n < heads)
                v0 = load4(x + n * a.dim + run0(u)), v1 = load4(x + n * a.dim + run1(u));
            float *e = v[n] + 8 * k;
            e[0] = v0.x, e[1] = v0.y, e[2] = v0.z, e[3] = v0.w;
            e[4] = v1.x, e[5] = v1.y, e[6] = v1.z, e[7] = v1.w;
        }
    float sum[H], r[H];
#pragma unroll
    for (int n = 0; n < H; ++n) {
        sum[n] = 0.f;
#pragma unroll
        for (int k = 0; k < 8 * U; ++k) sum[n] = fmaf(v[n][k], v[n][k], sum[n]);
    }
    for (int o = group / 2; o; o /= 2)
#pragma unroll
        for (int n = 0; n < H; ++n) sum[n] += __shfl_xor_sync(~0u, sum[n], o);
#pragma unroll
    for (int n = 0; n < H; ++n) {
        const float mean = __fdiv_rn(sum[n], (float)a.dim) + a.eps;
        r[n] = __fdiv_rn(1.f, __fsqrt_rn(mean));
        // the head's squares may be past f32: its own factor
        const bool odd = !(mean > 1e-30f && mean < INFINITY);
        if (__any_sync(~0u, odd && n < heads)) {
            const float f = scaled_factor(v[n], group, a.dim, a.eps);
            if (odd) r[n] = f;
        }
    }
    if (i >= all) return;
    const bool bad = a.table && (pos < 0 || pos >= a.positions);
#pragma unroll
    for (int k = 0; k < U; ++k) {
        const int u = lane + k * group;
        if (u >= units) continue;
        const int e0 = run0(u), e1 = run1(u);
        float4 w0 = make_float4(1.f, 1.f, 1.f, 1.f), w1 = w0, c0 = w0, c1 = w0;
        if (part.weight) {
            w0 = __ldg(reinterpret_cast<const float4 *>(part.weight + e0));
            w1 = __ldg(reinterpret_cast<const float4 *>(part.weight + e1));
        }
        const bool turns = u < turned && !bad;
        if (turns) {
            const float4 *cs = reinterpret_cast<const float4 *>(a.table + (int64_t)pos * a.rot + 8 * u);
            c0 = __ldg(cs), c1 = __ldg(cs + 1);
        }
#pragma unroll
        for (int n = 0; n < H; ++n) {
            if (n >= heads) break;
            const float *e = v[n] + 8 * k;
            float4 v0 = make_float4(e[0] * r[n] * w0.x, e[1] * r[n] * w0.y, e[2] * r[n] * w0.z, e[3] * r[n] * w0.w);
            float4 v1 = make_float4(e[4] * r[n] * w1.x, e[5] * r[n] * w1.y, e[6] * r[n] * w1.z, e[7] * r[n] * w1.w);
            if (bad) {
                const float z = quiet_nan();
                v0 = v1 = make_float4(z, z, z, z);
            } else if (turns) {
                const float4 y0 = v0, y1 = v1;
                if (a.inter) {
                    v0 = make_float4(rot_a(y0.x, y0.y, c0.x, c0.y), rot_b(y0.x, y0.y, c0.x, c0.y),
                                     rot_a(y0.z, y0.w, c0.z, c0.w), rot_b(y0.z, y0.w, c0.z, c0.w));
                    v1 = make_float4(rot_a(y1.x, y1.y, c1.x, c1.y), rot_b(y1.x, y1.y, c1.x, c1.y),
                                     rot_a(y1.z, y1.w, c1.z, c1.w), rot_b(y1.z, y1.w, c1.z, c1.w));
                } else {
                    v0 = make_float4(rot_a(y0.x, y1.x, c0.x, c0.y), rot_a(y0.y, y1.y, c0.z, c0.w),
                                     rot_a(y0.z, y1.z, c1.x, c1.y), rot_a(y0.w, y1.w, c1.z, c1.w));
                    v1 = make_float4(rot_b(y0.x, y1.x, c0.x, c0.y), rot_b(y0.y, y1.y, c0.z, c0.w),
                                     rot_b(y0.z, y1.z, c1.x, c1.y), rot_b(y0.w, y1.w, c1.z, c1.w));
                }
            }
            TO *o = out + n * a.dim;
            if (sizeof(TO) == 2 && e1 == e0 + 4) store8(o + e0, v0, v1);
            else store4(o + e0, v0), store4(o + e1, v1);
        }
    }
}

namespace {
template <class TI, class TO, int U, int H>
cudaError_t launch_heads(NormArgs &a, int parts, int lg, cudaStream_t s) {
    a.runs = 0;
    for (int i = 0; i < parts; ++i) a.upto[i] = a.runs += (a.part[i].heads + H - 1) / H;
    const int group = 1 << lg;
    const int64_t all = a.ntok * a.runs;
    const int wide = all > 0x7FFFFFFF;
    const int64_t blocks = (all + kNormThreads / group - 1) / (kNormThreads / group);
    // (2^24 tokens of 4096 heads: 2^36 heads, 2^33 blocks of 8)
    if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    kq_norm_kernel<TI, TO, U, H><<<(unsigned)blocks, kNormThreads, 0, s>>>(a, lg, wide);
    return cudaGetLastError();
}
template <class TI, class TO>
cudaError_t launch(NormArgs &a, int parts, cudaStream_t s) {
    int lg = 0;
    while (lg < 5 && 8 << lg < a.dim) ++lg;
    const int each = (a.dim / 8 + (1 << lg) - 1) >> lg;
    int64_t heads = 0;
    for (int i = 0; i < parts; ++i) heads += a.part[i].heads;
    // Four heads a group once there are four rounds of warps over the chip: a
    // token's cos and sin and the weights are fetched for all of them, and four
    // loads are on their way (8191 tokens of 40 heads of 128 from f32 to bf16:
    // one 53.5 us, four 49.4, in CTAs of 128 threads 45.2; two 50.9, eight 54.5).
    if (each > 2) return launch_heads<TI, TO, 4, 1>(a, parts, lg, s);
    if (each > 1) return launch_heads<TI, TO, 2, 1>(a, parts, lg, s);
    if (a.ntok * heads << lg >= 152 * 2048 * 4) return launch_heads<TI, TO, 1, 4>(a, parts, lg, s);
    return launch_heads<TI, TO, 1, 1>(a, parts, lg, s);
}
}  // namespace

cudaError_t norm_rope(NormArgs &a, int parts, int type, int out_type, cudaStream_t s) {
    if (type == KQ_F16) return launch<__half, __half>(a, parts, s);
    if (type == KQ_BF16) return launch<__nv_bfloat16, __nv_bfloat16>(a, parts, s);
    return out_type == KQ_F32   ? launch<float, float>(a, parts, s)
           : out_type == KQ_F16 ? launch<float, __half>(a, parts, s)
                                : launch<float, __nv_bfloat16>(a, parts, s);
}

}  // namespace kqp
