// kq_logprob.cu -- log probabilities of given tokens, entropies and the best
// alternatives of rows of logits (kq_token_logprobs).
//
// One pass over a row: a thread keeps its running maximum m, S = sum e^(x - m)
// and T = sum e^(x - m) (x - m), corrected once a batch, and a warp its largest
// logits, a sorted list with one entry a lane.  An entry is a 64-bit number,
// the logit's bits turned to order like it above the token's complement, so
// all differ and any order of merging gives the same list.  A batch is looked
// at only where its largest reaches what some warp of the CTA holds `top` values
// of already: few are merged in one by one, many by a sorting network of the
// lanes' largest and a merge.  Lists and sums are joined by warps, then over a
// cluster of CTAs that share a row.
//
// Bound by memory for many rows: 1999 rows of 202048 f32 logits, 5 alternatives,
// 252 us, 95% of the copy rate (486 us with a bound of each warp's own, where two
// batches of three had to be looked at).  By latency for few: one row 8.7 us with
// 20 alternatives, 4.6 without; the load takes 1.1 us, and what the first batch
// holds, candidates and two joins, the rest.  Code that runs once is fetched as it
// is reached, so it is kept short: candidates in a loop and one copy of the join
// instead of all of it written out, 12.3 and 276 to 11.9 and 261 us.
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
// Candidates of a warp's batch that are merged in one by one (64 rows of 32000,
// 20 alternatives: 8 10.5 us, 12 to 32 9.4).
constexpr int kFew = 16;

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

// A value that orders as it does, for atomics; never a NaN.
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);
    return b ^ (b >> 31 ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float ordered(uint32_t k) {
    return __uint_as_float(k >> 31 ? k ^ 0x80000000u : ~k);
}

struct ScoreShared {
    int count;
    uint32_t bar;  // order_of a value that `top` values of some warp reach
    Key list[kScoreWarps][32];  // (0: no entry)
    Key pool[kScoreThreads];    // those that may be of the best
    uint32_t nth[kScoreWarps];  // of a warp's lanes, in the first batch
    Key best[32];
    Sums sums[kScoreWarps];
    // of the cluster's CTAs, gathered in the first
    Key lists[kScoreCluster][32];
    Sums parts[kScoreCluster];
};

// What `top` values of the CTA's first batch reach: in n warps, r lanes or more
// have a largest value at or above the n-th largest of all warps' r-th such, so
// that n r >= top values do.  r: of random logits, where the fewest pass.  (The
// least of the warps' second largest: one row 11.9 us against 8.7.)
__device__ __forceinline__ uint32_t first_bound(uint32_t *nth, float most, int top, int w, int lane) {
    static_assert(kScoreWarps == 16 && KQ_MAX_TOP <= 3 * kScoreWarps, "the first bound");
    const int r = top <= 12 ? 1 : top <= 24 ? 2 : 3, n = (top + r - 1) / r;
    uint32_t x = order_of(most != most ? -INFINITY : most), its = __reduce_max_sync(~0u, x);
#pragma unroll 1
    for (int i = 1; i < r; ++i) {
        if (lane == __ffs(__ballot_sync(~0u, x == its)) - 1) x = 0;
        its = __reduce_max_sync(~0u, x);
    }
    if (lane == 0) nth[w] = its;
    __syncthreads();
    its = nth[lane & 15];
    int before = 0;
#pragma unroll
    for (int o = 1; o < kScoreWarps; ++o) before += __shfl_xor_sync(~0u, its, o) > its;
    return __reduce_min_sync(~0u, before < n ? its : ~0u);
}

// The `top` largest of n sorted lists (of up to 16), in sh.best.  Entries that
// cannot be of them are left out: what the `top`-th of some list, or the r-th of
// every one (n r >= top), passes.  The others go to the place that the number of
// larger ones gives.  (A tree of merges: 1.7 us against 0.5.)  A function of its
// own, as both calls then run the same code.
__device__ __noinline__ void join_lists(ScoreShared &sh, const Key (*list)[32], int n, int top, int w,
                                        int lane) {
    __syncthreads();
    if (threadIdx.x == 0) sh.count = 0;
    if (threadIdx.x < 32) sh.best[lane] = 0;
    __syncthreads();
    const uint32_t last = lane < n ? (uint32_t)(list[lane][top - 1] >> 32) : 0u;
    const uint32_t each = lane < n ? (uint32_t)(list[lane][(top + n - 1) / n - 1] >> 32) : ~0u;
    const uint32_t least = max(__reduce_max_sync(~0u, last), __reduce_min_sync(~0u, each));
    const Key mine = w < n ? list[w][lane] : 0;
    const bool in = mine != 0 && lane < top && (uint32_t)(mine >> 32) >= least;
    const uint32_t who = __ballot_sync(~0u, in);
    int at = 0;
    if (lane == 0 && who) at = atomicAdd(&sh.count, __popc(who));
    at = __shfl_sync(~0u, at, 0);
    if (in) sh.pool[at + __popc(who & ((1u << lane) - 1))] = mine;
    __syncthreads();
    const int all = sh.count;
    // up to 128 keys: four threads count for each
    const int by = all <= kScoreThreads / 4 ? 4 : 1;
    const int i = threadIdx.x / by, part = threadIdx.x & (by - 1);
    if (w * 32 < all * by) {
        const Key k = i < all ? sh.pool[i] : ~0ull;
        int before = 0;
#pragma unroll 4
        for (int j = part; j < all; j += by) before += sh.pool[j] > k;
        if (by == 4) {
            before += __shfl_xor_sync(~0u, before, 1);
            before += __shfl_xor_sync(~0u, before, 2);
        }
        if (i < all && part == 0 && before < top) sh.best[before] = k;
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
    if (tid == 0) sh.bar = 0;
    __syncthreads();
    // A batch's values; the next one's are on their way while it is looked at.
    auto load = [&](int j0, float (&v)[kBatchValues]) {
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
    };
    constexpr int kStep = kScoreThreads * kBatchValues;
    float ahead[kBatchValues];
    load(lo, ahead);
    for (int j0 = lo; j0 < hi; j0 += kStep) {
        float v[kBatchValues];
#pragma unroll
        for (int i = 0; i < kBatchValues; ++i) v[i] = ahead[i];
        const int first = j0 + tid * V;
        if (j0 + kStep < hi) load(j0 + kStep, ahead);
        float most = v[0];
#pragma unroll
        for (int i = 1; i < kBatchValues; ++i) most = fmaxf(most, v[i]);
        const float top = fmaxf(mine.m, most);
        mine = about(mine, top);
        const float from = top == -INFINITY ? 0.f : top;
        float2 s2 = make_float2(0.f, 0.f), t2 = s2;
#pragma unroll
        for (int i = 0; i < kBatchValues; i += 2) {
            const float2 d = mul2(add2(make_float2(v[i], v[i + 1]), make_float2(-from, -from)),
                                  make_float2(kLog2e, kLog2e));
            const float2 e = make_float2(exp2_of(d.x), exp2_of(d.y));
            s2 = add2(s2, e);
            t2 = fma2(e, make_float2(fmaxf(d.x, kFar), fmaxf(d.y, kFar)), t2);
        }
        const float sum = s2.x + s2.y;
        mine.s += sum, mine.t += t2.x + t2.y;
        if (a.top == 0) continue;
        if (j0 == lo) {
            const uint32_t least = first_bound(sh.nth, most, a.top, w, lane);
            if (lane == 0) atomicMax(&sh.bar, least);
            __syncwarp();
        }
        // (a NaN is a candidate too, and shows in the sum)
        const float bar = ordered(*(volatile uint32_t *)&sh.bar);
        if (!__any_sync(~0u, !(most < bar) || sum != sum)) continue;
        // ---- candidates
        uint32_t left = 0;
#pragma unroll
        for (int i = 0; i < kBatchValues; ++i) {
            const int j = first + (i / V) * kScoreThreads * V + i % V;
            if (!(v[i] < bar) && j >= skew && j < hi) left |= 1u << i;
        }
        const int many = __reduce_add_sync(~0u, __popc(left));
        if (many <= kFew) {
            // one by one, of the lanes' next
            while (unsigned who = __ballot_sync(~0u, left != 0)) {
                const int i = __ffs(left) - 1;
                float next = v[0];
#pragma unroll
                for (int n = 1; n < kBatchValues; ++n) next = n == i ? v[n] : next;
                const Key key = key_of(next, first + (i / V) * kScoreThreads * V + i % V - skew);
                left &= left - 1;
#pragma unroll 1
                for (; who; who &= who - 1) {
                    const Key k = __shfl_sync(~0u, key, __ffs(who) - 1);
                    const Key up = __shfl_up_sync(~0u, list, 1);
                    const int place = __popc(__ballot_sync(~0u, list > k));
                    list = lane < place ? list : lane == place ? k : up;
                }
            }
        } else {
            // by turns each lane's largest that is not in yet
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
                if (!__any_sync(~0u, best != 0)) break;
                if (best) left &= ~(1u << at);
                list = merged(list, sorted(best, lane), lane);
                last = __shfl_sync(~0u, list, a.top - 1);
            }
        }
        const Key now = __shfl_sync(~0u, list, a.top - 1);
        if (now != last || many > kFew) {
            last = now;
            // (where the list ends with a NaN, no number passes)
            const float x = value_of(last);
            if (lane == 0 && last) atomicMax(&sh.bar, order_of(x != x ? INFINITY : x));
        }
    }
    // ---- joined over the warp, the CTA, the cluster
#pragma unroll
    for (int o = 16; o; o /= 2)
        mine = joined(mine, {__shfl_xor_sync(~0u, mine.m, o), __shfl_xor_sync(~0u, mine.s, o),
                             __shfl_xor_sync(~0u, mine.t, o)});
    if (lane == 0) sh.sums[w] = mine;
    sh.list[w][lane] = list;
    if (a.top) join_lists(sh, sh.list, kScoreWarps, a.top, w, lane);
    else __syncthreads();
    Sums all = {-INFINITY, 0.f, 0.f};
    if (w == 0) {
        if (lane < kScoreWarps) all = sh.sums[lane];
#pragma unroll
        for (int o = kScoreWarps / 2; o; o /= 2)
            all = joined(all, {__shfl_xor_sync(~0u, all.m, o), __shfl_xor_sync(~0u, all.s, o),
                               __shfl_xor_sync(~0u, all.t, o)});
    }
    if (ctas > 1) {
        cg::cluster_group cluster = cg::this_cluster();
        asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
        ScoreShared *to = cluster.map_shared_rank(&sh, 0);
        if (w == 0) {
            to->lists[rank][lane] = a.top ? sh.best[lane] : 0;
            if (lane == 0) to->parts[rank] = all;
        }
        cluster.sync();
        if (rank != 0) return;
        if (a.top) join_lists(sh, sh.lists, ctas, a.top, w, lane);
        if (w == 0) {
            all = lane < ctas ? sh.parts[lane] : Sums{-INFINITY, 0.f, 0.f};
#pragma unroll
            for (int o = kScoreCluster / 2; o; o /= 2)
                all = joined(all, {__shfl_xor_sync(~0u, all.m, o), __shfl_xor_sync(~0u, all.s, o),
                                   __shfl_xor_sync(~0u, all.t, o)});
        }
    }
    if (w != 0) return;
    list = sh.best[lane];
    all = {__shfl_sync(~0u, all.m, 0), __shfl_sync(~0u, all.s, 0), __shfl_sync(~0u, all.t, 0)};
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
    // CTAs of a row: up to 16, each with 4096 words or more, and two an SM in all.
    // 1, 9, 38, 100, 200 rows of 202048 f32 logits, 5 alternatives: 8.5, 10.8, 20.4,
    // 27.9, 40.2 us; one CTA a row 22.1, 23.4, 25.9, 27.2, 40.1; one an SM in all 8.6,
    // 10.8, 18.6, 26.9, 40.3; four an SM 8.4, 10.8, 26.0, 28.1, 40.8.
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
