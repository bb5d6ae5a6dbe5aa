// kq_verify.cu -- verification of drafted tokens (kq_verify_tree).
//
// One CTA per sequence walks the tree; r, the residual distribution, is
// never stored: it is p[cur] less z_1 q[cur], less z_2 q[cur] ... for the
// children rejected so far, formed again from p and q and the few z where
// it is needed.  Sums are over whole multiples of 2^-44, so any order gives
// the same.
#include "kq_decode.cuh"
#include "kq_decode_launch.h"

namespace kqd {

constexpr int kVerifyThreads = 1024;

__device__ __forceinline__ float unit(float x) { return fminf(fmaxf(x, 0.f), 1.f); }

// r at token x: row p less what each rejected child took out.
struct Residual {
    const float *p, *q;  // rows of the current node; q NULL: no distribution
    int n;               // rejected children
    const float *z;      // with q: the sums before each
    const int32_t *out;  // without: their tokens
    __device__ __forceinline__ float at(int x) const {
        float r = unit(__ldg(p + x));
        if (q) {
            const float d = n ? unit(__ldg(q + x)) : 0.f;
            for (int i = 0; i < n; ++i) r = fmaxf(__fsub_rn(r, __fmul_rn(z[i], d)), 0.f);
        } else {
            for (int i = 0; i < n; ++i) r = out[i] == x ? 0.f : r;
        }
        return r;
    }
};
__device__ __forceinline__ unsigned long long fixed(float r) {
    return (unsigned long long)__float2ull_rz(r * 17592186044416.f);  // 2^44
}

__device__ unsigned long long block_sum(unsigned long long v, unsigned long long *tmp) {
#pragma unroll
    for (int o = 16; o; o /= 2) v += __shfl_xor_sync(~0u, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) tmp[threadIdx.x >> 5] = v;
    __syncthreads();
    unsigned long long s = 0;
    for (int i = 0; i < kVerifyThreads / 32; ++i) s += tmp[i];
    return s;
}

__global__ void __launch_bounds__(kVerifyThreads)
    kq_verify_kernel(const __grid_constant__ VerifyArgs a) {
    __shared__ unsigned long long tmp[kVerifyThreads / 32];
    __shared__ float z[KQ_MAX_DRAFT];
    __shared__ int32_t out[KQ_MAX_DRAFT];
    const int b = blockIdx.x, tid = threadIdx.x, V = a.vocab;
    const Seq s = seq_of(a.start, nullptr, a.ntok, a.max_new, b);
    if (s.n == 0) {
        if (tid == 0) a.count[b] = 0, a.next[b] = -1;
        return;
    }
    for (int i = tid; i < s.n; i += kVerifyThreads) a.path[s.first + i] = i ? -1 : 0;
    __syncthreads();
    int cur = 0, got = 1;
    float zc = 1.f;
    Residual r{a.p + (int64_t)s.first * a.p_stride, a.q ? a.q + (int64_t)s.first * a.q_stride : nullptr,
               0, z, out};
    for (int j = 1; j < s.n; ++j) {
        const int x = s.first + j;
        if (__ldg(a.parent + x) != cur) continue;
        const int t = __ldg(a.token + x);
        if (t < 0 || t >= V) continue;
        const float have = r.at(t);
        const float d = r.q ? __fmul_rn(unit(__ldg(r.q + t)), zc) : zc;
        if (__fmul_rn(unit(__ldg(a.u + x)), d) < have) {
            cur = j;
            r.p = a.p + (int64_t)x * a.p_stride;
            if (a.q) r.q = a.q + (int64_t)x * a.q_stride;
            r.n = 0, zc = 1.f;
            if (tid == 0) a.path[s.first + got] = j;
            ++got;
            continue;
        }
        // rejected: what is left without it
        __syncthreads();
        if (tid == 0) z[r.n] = zc, out[r.n] = t;
        __syncthreads();
        Residual left = r;
        left.n = r.n + 1;
        unsigned long long sum = 0;
        for (int i = tid; i < V; i += kVerifyThreads) sum += fixed(left.at(i));
        sum = block_sum(sum, tmp);
        if (sum) {
            r = left;
            zc = (float)((double)(long long)sum * 0x1p-44);
        }
    }
    // the first token whose running sum passes the goal: each thread sums a
    // run of tokens, the runs before it are added up, and the one run that
    // holds the goal is walked
    const int per = (V + kVerifyThreads - 1) / kVerifyThreads;
    const int lo = min(tid * per, V), hi = min(lo + per, V);
    unsigned long long mine = 0;
    for (int i = lo; i < hi; ++i) mine += fixed(r.at(i));
    const unsigned long long total = block_sum(mine, tmp);
    unsigned long long upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const unsigned long long v = __shfl_up_sync(~0u, upto, o);
        if ((tid & 31) >= o) upto += v;
    }
    // (block_sum left every warp's sum in tmp)
    for (int i = 0; i < (tid >> 5); ++i) upto += tmp[i];
    const unsigned long long u = min((unsigned long long)(unit(__ldg(a.u_next + b)) * 0x1p31f), 0x7FFFFFFFull);
    const unsigned long long goal = (total >> 31) * u + (((total & 0x7FFFFFFFull) * u) >> 31);
    if (tid == 0) {
        a.count[b] = got;
        if (total == 0) a.next[b] = V - 1;
    }
    if (goal >= upto - mine && goal < upto) {
        unsigned long long sum = upto - mine;
        int i = lo;
        for (; i < hi - 1; ++i) {
            sum += fixed(r.at(i));
            if (sum > goal) break;
        }
        a.next[b] = i;
    }
}

cudaError_t verify(const VerifyArgs &a, cudaStream_t s) {
    kq_verify_kernel<<<a.nseq, kVerifyThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace kqd
