// kq_logprob.cu -- log probabilities of given tokens, entropies and the best
// alternatives of rows of logits (kq_token_logprobs).
//
// One pass over a row: a thread keeps its running maximum m, S = sum e^(x - m)
// and T = sum e^(x - m) (x - m), corrected once a batch, and a warp its largest
// logits, a sorted list with one entry a lane.  An entry is a 64-bit number,
// the logit's bits turned to order like it above the token's complement, so
// all differ and any order of merging gives the same list.  A batch is looked
// at only where a value passes the list's last entry: few are merged in one by
// one, many by a sorting network of the lanes' largest and a merge.  Lists and
// sums are joined by warps, then over a cluster of CTAs that share a row.
//
// Bound by memory for many rows, by latency for few.
#include <cooperative_groups.h>

#include <mutex>

#include "kq_decode.cuh"
#include "kq_prompt_launch.h"
#include "kq_types.cuh"

namespace kqp {

namespace cg = cooperative_groups;
using kqd::quiet_nan;

constexpr int kScoreThreads = 512;
constexpr int kScoreWarps = kScoreThreads / 32;
constexpr int kScoreCluster = 16;  // most CTAs of a row
constexpr int kScoreCtas = 304;    // two an SM of this chip
constexpr int kBatchValues = 16;   // of a thread, loads in flight

using Key = unsigned long long;

// A number that orders like (x, lower token first): NaN above all, -0 as 0.
__device__ __forceinline__ Key key_of(float x, int token) {
    uint32_t b = __float_as_uint(x + 0.f);
    b = x != x ? 0xFFFFFFFFu : b ^ (b >> 31 ? 0xFFFFFFFFu : 0x80000000u);
    return (Key)b << 32 | (uint32_t)~token;
}
__device__ __forceinline__ float value_of(Key k) {
    const uint32_t b = (uint32_t)(k >> 32);
    return __uint_as_float(b >> 31 ? b ^ 0x80000000u : ~b);  // (NaN: 0x7FFFFFFF)
}
__device__ __forceinline__ int token_of(Key k) { return (int)~(uint32_t)k; }

__device__ __forceinline__ Key pick(Key mine, int o, bool larger) {
    const Key other = __shfl_xor_sync(~0u, mine, o);
    return (mine > other) == larger ? mine : other;
}
// The warp's 32 keys, largest in lane 0.
__device__ __forceinline__ Key sorted(Key k, int lane) {
#pragma unroll
    for (int n = 2; n <= 32; n *= 2)
#pragma unroll
        for (int o = n / 2; o; o /= 2) k = pick(k, o, ((lane & o) == 0) == ((lane & n) == 0 || n == 32));
    return k;
}
// The 32 largest of two sorted lists, sorted.
__device__ __forceinline__ Key merged(Key a, Key b, int lane) {
    const Key r = __shfl_sync(~0u, b, 31 - lane);
    Key k = a > r ? a : r;
#pragma unroll
    for (int o = 16; o; o /= 2) k = pick(k, o, (lane & o) == 0);
    return k;
}

struct Sums {
    float m, s, t;  // t in units of log2(e)
};
__device__ __forceinline__ float exp2_of(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.693147180559945309417f;
// -infinity times a weight of zero would be NaN: the least distance that is
// multiplied (e^(x - m) is zero long before).
constexpr float kFar = -1e30f;

// Sums about the reference `m` (not below s.m); an empty sum stays empty.
__device__ __forceinline__ Sums about(Sums s, float m) {
    if (s.m == m || s.m == -INFINITY) return {m, s.s, s.t};
    const float d = (s.m - m) * kLog2e, f = exp2_of(d);
    return {m, s.s * f, f * fmaf(fmaxf(d, kFar), s.s, s.t)};
}
__device__ __forceinline__ Sums joined(Sums a, Sums b) {
    const float m = fmaxf(a.m, b.m);
    a = about(a, m), b = about(b, m);
    return {m, a.s + b.s, a.t + b.t};
}

struct ScoreShared {
    Key list[kScoreWarps][32];
    Sums sums[kScoreWarps];
    // of the cluster's CTAs, gathered in the first
    Key lists[kScoreCluster][32];
    Sums parts[kScoreCluster];
};

// Lists of n warps (n a power of two) joined into the first.
__device__ __forceinline__ void join_lists(Key (*list)[32], int n, int w, int lane) {
    for (int half = n / 2; half; half /= 2) {
        __syncthreads();
        if (w < half) list[w][lane] = merged(list[w][lane], list[w + half][lane], lane);
    }
    __syncthreads();
}

template <class T>
__global__ void __launch_bounds__(kScoreThreads, 2)
    kq_score_kernel(const __grid_constant__ ScoreArgs a, int ctas, int chunk) {
    constexpr int V = 16 / sizeof(T);        // values of a load
    constexpr int R = kBatchValues / V;      // loads of a batch
    __shared__ ScoreShared sh;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int rank = ctas > 1 ? (int)(blockIdx.x % ctas) : 0;
    const int64_t row = ctas > 1 ? blockIdx.x / ctas : blockIdx.x;
    const T *x = static_cast<const T *>(a.x) + row * a.stride;
    // Words are counted from the 16-byte line that holds the row's first: word
    // j is value j - skew, and the CTA's words are whole lines.
    const int skew = (int)(((uintptr_t)x & 15) / sizeof(T));
    const T *line = x - skew;
    const int lo = rank * chunk, hi = min(lo + chunk, a.vocab + skew);
    // (every CTA of the cluster is there before another writes to it)
    if (ctas > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");

    Sums mine = {-INFINITY, 0.f, 0.f};
    Key list = 0;  // (below every key)
    Key last = 0;  // the list's entry that a candidate has to pass
    float bar = -INFINITY;
    for (int j0 = lo; j0 < hi; j0 += kScoreThreads * kBatchValues) {
        float v[kBatchValues];
        const int first = j0 + tid * V;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int j = first + r * kScoreThreads * V;
            if (j >= skew && j + V <= hi) {
                const uint4 q = __ldcs(reinterpret_cast<const uint4 *>(line + j));
                const uint32_t word[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (sizeof(T) == 4) {
                        v[V * r + i] = __uint_as_float(word[i]);
                    } else {
                        const float2 f = unpack2<T>(word[i]);
                        v[V * r + 2 * i] = f.x, v[V * r + 2 * i + 1] = f.y;
                    }
                }
            } else {  // the row's ends
#pragma unroll
                for (int i = 0; i < V; ++i)
                    v[V * r + i] = j + i >= skew && j + i < hi ? to_f32<T>(line[j + i]) : -INFINITY;
            }
        }
        float top = mine.m;
        bool found = false;
#pragma unroll
        for (int i = 0; i < kBatchValues; ++i) top = fmaxf(top, v[i]);
        mine = about(mine, top);
        const float from = top == -INFINITY ? 0.f : top;
        float s0 = 0.f, s1 = 0.f, t0 = 0.f, t1 = 0.f;
#pragma unroll
        for (int i = 0; i < kBatchValues; i += 2) {
            const float d0 = (v[i] - from) * kLog2e, d1 = (v[i + 1] - from) * kLog2e;
            const float e0 = exp2_of(d0), e1 = exp2_of(d1);
            s0 += e0, s1 += e1;
            t0 = fmaf(e0, fmaxf(d0, kFar), t0), t1 = fmaf(e1, fmaxf(d1, kFar), t1);
            // (not below: a NaN is a candidate too)
            found |= !(v[i] < bar) || !(v[i + 1] < bar);
        }
        mine.s += s0 + s1, mine.t += t0 + t1;
        if (a.top == 0 || !__any_sync(~0u, found)) continue;
        // ---- candidates: by turns each lane's largest that is not in yet
        uint32_t left = 0;
#pragma unroll
        for (int i = 0; i < kBatchValues; ++i) {
            const int j = first + (i / V) * kScoreThreads * V + i % V;
            if (j >= skew && j < hi && key_of(v[i], j - skew) > last) left |= 1u << i;
        }
        while (true) {
            Key best = 0;
            int at = 0;
#pragma unroll
            for (int i = 0; i < kBatchValues; ++i) {
                const int j = first + (i / V) * kScoreThreads * V + i % V;
                const Key k = key_of(v[i], j - skew);
                if (left >> i & 1) {
                    if (k <= last) left &= ~(1u << i);
                    else if (k > best) best = k, at = i;
                }
            }
            unsigned who = __ballot_sync(~0u, best != 0);
            if (who == 0) break;
            if (best) left &= ~(1u << at);
            if (__popc(who) > 6) {
                list = merged(list, sorted(best, lane), lane);
            } else {
                while (who) {
                    const Key k = __shfl_sync(~0u, best, __ffs(who) - 1);
                    who &= who - 1;
                    const Key up = __shfl_up_sync(~0u, list, 1);
                    const int place = __popc(__ballot_sync(~0u, list > k));
                    list = lane < place ? list : lane == place ? k : up;
                }
            }
            last = __shfl_sync(~0u, list, a.top - 1);
        }
        // (a NaN at the list's end lets no number pass, only another NaN)
        bar = last == 0 ? -INFINITY : value_of(last);
        if (bar != bar) bar = INFINITY;
    }
    // ---- joined over the warp, the CTA, the cluster
#pragma unroll
    for (int o = 16; o; o /= 2)
        mine = joined(mine, {__shfl_xor_sync(~0u, mine.m, o), __shfl_xor_sync(~0u, mine.s, o),
                             __shfl_xor_sync(~0u, mine.t, o)});
    if (lane == 0) sh.sums[w] = mine;
    sh.list[w][lane] = list;
    if (a.top) join_lists(sh.list, kScoreWarps, w, lane);
    else __syncthreads();
    Sums all = {-INFINITY, 0.f, 0.f};
    if (w == 0) {
        for (int i = 0; i < kScoreWarps; ++i) all = joined(all, sh.sums[i]);
        list = sh.list[0][lane];
    }
    if (ctas > 1) {
        cg::cluster_group cluster = cg::this_cluster();
        asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
        ScoreShared *to = cluster.map_shared_rank(&sh, 0);
        if (w == 0) {
            to->lists[rank][lane] = list;
            if (lane == 0) to->parts[rank] = all;
        }
        cluster.sync();
        if (rank != 0) return;
        if (a.top) join_lists(sh.lists, ctas, w, lane);
        if (w == 0) {
            all = {-INFINITY, 0.f, 0.f};
            for (int i = 0; i < ctas; ++i) all = joined(all, sh.parts[i]);
            list = sh.lists[0][lane];
        }
    }
    if (w != 0) return;
    // nothing but -infinity: 0 / 0
    const float s = all.m == -INFINITY ? quiet_nan() : all.s;
    const float log_s = logf(s);
    if (lane == 0) {
        if (a.logp) {
            const int t = __ldg(a.token + row);
            a.logp[row] =
                t >= 0 && t < a.vocab ? (to_f32<T>(x[t]) - all.m) - log_s : quiet_nan();
        }
        if (a.entropy) {
            const float h = log_s - kLn2 * __fdiv_rn(all.t, s);
            a.entropy[row] = h < 0.f ? 0.f : h;
        }
    }
    if (lane < a.top) {
        a.top_logp[row * a.top + lane] = (value_of(list) - all.m) - log_s;
        a.top_token[row * a.top + lane] = token_of(list);
    }
}

namespace {
template <class T>
cudaError_t launch(const ScoreArgs &a, cudaStream_t s) {
    // CTAs of a row: up to 16, each with 4096 words or more, and about two an SM
    // in all.
    int ctas = 1;
    while (ctas < kScoreCluster && ctas * 4096 < a.vocab && 2 * ctas * a.n <= kScoreCtas) ctas *= 2;
    constexpr int V = 16 / sizeof(T);
    // (V - 1: the words before a row's first in its line)
    const int chunk = ((a.vocab + V - 1 + ctas - 1) / ctas + V - 1) / V * V;
    static std::mutex mu;
    static bool configured[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (dev < 0 || dev >= 64 || !configured[dev]) {
            e = cudaFuncSetAttribute(kq_score_kernel<T>,
                                     cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e != cudaSuccess) return e;
            if (dev >= 0 && dev < 64) configured[dev] = true;
        }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.n * ctas));
    cfg.blockDim = dim3(kScoreThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kq_score_kernel<T>, a, ctas, chunk);
}
}  // namespace

cudaError_t token_logprobs(const ScoreArgs &a, int type, cudaStream_t s) {
    return type == KQ_F32   ? launch<float>(a, s)
           : type == KQ_F16 ? launch<__half>(a, s)
                            : launch<__nv_bfloat16>(a, s);
}

}  // namespace kqp
