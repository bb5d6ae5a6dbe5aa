// kq_rope.cu -- rotary positions: the table of (cos, sin) and the rotation.
//
// Rotation: one thread per eight values of a head, i.e. four pairs (a, b):
// two float4 of x, two float4 of the table, two float4 out.  Bound by
// memory: 8 bytes a value for x and out; a token's table row is shared by
// its heads and comes from cache after the first.  8191 tokens of 32 heads of
// 128, 64 of them turned: 45 us, 89% of the copy rate; one token: 2.0 us.
#include "kq_decode.cuh"
#include "kq_decode_launch.h"

namespace kqd {

constexpr int kRopeThreads = 256;

// One thread per (position, pair); f64 throughout, once per table.
__global__ void kq_rope_table_kernel(float2 *__restrict__ table, int64_t positions, int half,
                                     double base, kq_rope_scaling sc) {
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= positions * half) return;
    const int64_t t = i / half;
    const int p = (int)(i - t * half);
    const double rot = 2.0 * half;
    if (sc.kind == 2) base *= pow(sc.factor, rot / (rot - 2));
    double f = pow(base, -2.0 * p / rot);
    if (sc.kind == 1) f /= sc.factor;
    if (sc.kind == 3) {
        const double turns = sc.orig * f / 6.283185307179586476925286766559;
        const double keep = fmin(fmax((turns - sc.slow) / (sc.fast - sc.slow), 0.0), 1.0);
        f = f / sc.factor * (1 - keep) + f * keep;
    }
    double s, c;
    sincos((double)t * f, &s, &c);
    table[i] = make_float2((float)(c * sc.magnitude), (float)(s * sc.magnitude));
}

__global__ void __launch_bounds__(kRopeThreads)
    kq_rope_kernel(const float *x, int64_t stride, float *out, int64_t out_stride, int64_t ntok,
                   int heads, int dim, const int32_t *__restrict__ pos,
                   const float *__restrict__ table, int64_t positions, int rot, int inter,
                   float sign) {
    const int per = heads * (dim / 8);
    const int64_t i = (int64_t)blockIdx.x * kRopeThreads + threadIdx.x;
    if (i >= ntok * per) return;
    const int64_t t = i / per;
    const int r = (int)(i - t * per);
    const int h = r / (dim / 8), u = r - h * (dim / 8);
    const float *xi = x + t * stride + (int64_t)h * dim;
    float *oi = out + t * out_stride + (int64_t)h * dim;
    const int p = __ldg(pos + t);
    const bool turn = u < rot / 8;
    // values of the thread: two runs of four
    const int e0 = turn && !inter ? 4 * u : 8 * u;
    const int e1 = turn && !inter ? 4 * u + rot / 2 : 8 * u + 4;
    if (p < 0 || p >= positions) {
        const float n = quiet_nan();
        *reinterpret_cast<float4 *>(oi + e0) = make_float4(n, n, n, n);
        *reinterpret_cast<float4 *>(oi + e1) = make_float4(n, n, n, n);
        return;
    }
    const float4 v0 = *reinterpret_cast<const float4 *>(xi + e0);
    const float4 v1 = *reinterpret_cast<const float4 *>(xi + e1);
    if (!turn) {
        *reinterpret_cast<float4 *>(oi + e0) = v0;
        *reinterpret_cast<float4 *>(oi + e1) = v1;
        return;
    }
    const float4 *cs = reinterpret_cast<const float4 *>(table + (int64_t)p * rot + 8 * u);
    float4 c0 = __ldg(cs), c1 = __ldg(cs + 1);
    c0.y *= sign, c0.w *= sign, c1.y *= sign, c1.w *= sign;
    float4 y0, y1;
    if (inter) {
        y0 = make_float4(rot_a(v0.x, v0.y, c0.x, c0.y), rot_b(v0.x, v0.y, c0.x, c0.y),
                         rot_a(v0.z, v0.w, c0.z, c0.w), rot_b(v0.z, v0.w, c0.z, c0.w));
        y1 = make_float4(rot_a(v1.x, v1.y, c1.x, c1.y), rot_b(v1.x, v1.y, c1.x, c1.y),
                         rot_a(v1.z, v1.w, c1.z, c1.w), rot_b(v1.z, v1.w, c1.z, c1.w));
    } else {
        y0 = make_float4(rot_a(v0.x, v1.x, c0.x, c0.y), rot_a(v0.y, v1.y, c0.z, c0.w),
                         rot_a(v0.z, v1.z, c1.x, c1.y), rot_a(v0.w, v1.w, c1.z, c1.w));
        y1 = make_float4(rot_b(v0.x, v1.x, c0.x, c0.y), rot_b(v0.y, v1.y, c0.z, c0.w),
                         rot_b(v0.z, v1.z, c1.x, c1.y), rot_b(v0.w, v1.w, c1.z, c1.w));
    }
    *reinterpret_cast<float4 *>(oi + e0) = y0;
    *reinterpret_cast<float4 *>(oi + e1) = y1;
}

cudaError_t rope_table(int64_t positions, int rot, double base, const kq_rope_scaling &sc,
                       float *table, cudaStream_t s) {
    const int64_t n = positions * (rot / 2);
    kq_rope_table_kernel<<<(unsigned)((n + 127) / 128), 128, 0, s>>>(
        reinterpret_cast<float2 *>(table), positions, rot / 2, base, sc);
    return cudaGetLastError();
}

cudaError_t rope(const float *x, int64_t stride, float *out, int64_t out_stride, int64_t ntok,
                 int heads, int dim, const int32_t *pos, const float *table, int64_t positions,
                 int rot, bool interleaved, bool inverse, cudaStream_t s) {
    const int64_t n = ntok * heads * (dim / 8);
    kq_rope_kernel<<<(unsigned)((n + kRopeThreads - 1) / kRopeThreads), kRopeThreads, 0, s>>>(
        x, stride, out, out_stride, ntok, heads, dim, pos, table, positions, rot,
        interleaved ? 1 : 0, inverse ? -1.f : 1.f);
    return cudaGetLastError();
}

}  // namespace kqd
