// kq_verify.cu -- verification of drafted tokens (kq_verify_tree).
//
// A cluster of CTAs per sequence, each with a run of the vocabulary.  Every
// CTA walks the tree itself: whether a child is accepted depends on its
// token's entries in its parent's rows alone (and on the sums of what is left
// after rejections), so those are fetched for all nodes at once and the walk
// runs in shared memory.  Only a rejection and the final draw touch whole
// rows: r, the residual distribution, is kept in shared memory, a run each
// CTA, and sums go round the cluster through distributed shared memory, one
// barrier each.  Sums are over whole multiples of 2^-44, so any order gives
// the same.  Each warp has a run of the CTA's words, and the sums by warp that
// come with r's total are the draw's first two levels: only the warp whose run
// holds the goal looks at words again.
//
// Bound by latency: a sequence reads two rows (1.6 MB at 202048 words) over 16
// SMs, after one dependent fetch of the nodes' entries.  One chain of 5
// drafts, 202048 words, one rejection, rows not in L2, by clock64 in a copy:
// 15700 clocks, entries 3500, r 8100 (two batches of loads), the sum round the
// cluster 2700, the draw 1400.  Measured, rows in L2: 10.2 us (one CTA that
// forms r again from p and q for each pass: 134); 16 trees of up to 16 nodes:
// 21.3 us.  More loads in flight, with 1024 threads a CTA: 8% less for the
// chain, 28% more for the trees, whose clusters then have no room side by
// side.
#include <cooperative_groups.h>

#include <mutex>

#include "kq_decode.cuh"
#include "kq_decode_launch.h"

namespace kqd {

namespace cg = cooperative_groups;

constexpr int kVerifyThreads = 512;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kMostWords = KQ_MAX_VOCAB / kMaxCluster;  // of a CTA
constexpr int kMostCtas = 304;  // two an SM of this chip
// Loads of a thread in flight, of p and of q: what 64 registers hold, two CTAs
// an SM, and half of the 25 rounds of a warp's run at 202048 words in 16 CTAs.
constexpr int kBatch = 13;

// 0..1; NaN is 0.
__device__ __forceinline__ float unit(float x) { return fminf(fmaxf(x, 0.f), 1.f); }
// r (0..1) in whole multiples of 2^-44, rounded down: the significand, 24
// bits, moved to its place.  (The conversion to 64 bits, two or so a clock,
// took longer than all else of a pass over a row.)
__device__ __forceinline__ unsigned long long fixed(float r) {
    const uint32_t b = __float_as_uint(r);
    const int down = 127 - (int)(b >> 23 & 255);
    return (unsigned long long)(b & 0x7FFFFFu | 0x800000u) << 21 >> min(down, 63);
}

struct VerifyShared {
    unsigned long long warp[kVerifyWarps];  // sums of the warps' runs
    unsigned long long cta[2];  // the CTA's sum, by turns
    int32_t token[KQ_MAX_DRAFT], parent[KQ_MAX_DRAFT];
    float u[KQ_MAX_DRAFT];
    float pt[KQ_MAX_DRAFT], qt[KQ_MAX_DRAFT];  // parent's rows at the node's token
    float z[KQ_MAX_DRAFT];                     // sums before each rejected child ...
    int32_t out[KQ_MAX_DRAFT];                 // ... and its token
};

__global__ void __launch_bounds__(kVerifyThreads, 2)
    kq_verify_kernel(const __grid_constant__ VerifyArgs a, int chunk) {
    cg::cluster_group cluster = cg::this_cluster();
    const int nrank = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    __shared__ VerifyShared sh;
    extern __shared__ float r[];  // this CTA's run of the residual
    const int b = blockIdx.x / nrank, tid = threadIdx.x, V = a.vocab;
    const int lane = tid & 31, w = tid >> 5;
    const int lo = min(rank * chunk, V), n = min(lo + chunk, V) - lo;
    // each warp has a run of the CTA's, [w0, w1)
    const int seg = (chunk + kVerifyWarps - 1) / kVerifyWarps;
    const int w0 = min(w * seg, n), w1 = min(w0 + seg, n);
    const Seq s = seq_of(a.start, nullptr, a.ntok, a.max_new, b);
    if (s.n == 0) {  // the same for the whole cluster
        if (rank == 0 && tid == 0) a.count[b] = 0, a.next[b] = -1;
        return;
    }
    const unsigned long long u =
        min((unsigned long long)(unit(__ldg(a.u_next + b)) * 0x1p31f), 0x7FFFFFFFull);
    for (int j = tid; j < s.n; j += kVerifyThreads) {
        const int x = s.first + j, t = __ldg(a.token + x), p = __ldg(a.parent + x);
        const bool ok = j > 0 && p >= 0 && p < j && t >= 0 && t < V;
        sh.token[j] = t;
        sh.parent[j] = ok ? p : -1;
        sh.u[j] = unit(__ldg(a.u + x));
        const int64_t row = s.first + (ok ? p : 0);
        sh.pt[j] = ok ? unit(__ldg(a.p + row * a.p_stride + t)) : 0.f;
        sh.qt[j] = ok && a.q ? unit(__ldg(a.q + row * a.q_stride + t)) : 0.f;
    }
    __syncthreads();

    // The cluster's sum of one number a thread; `turn` counts the calls.
    // before: the sum over the CTAs of lower rank.
    int turn = 0;
    unsigned long long before = 0;
    auto cluster_sum = [&](unsigned long long v) {
#pragma unroll
        for (int o = 16; o; o /= 2) v += __shfl_xor_sync(~0u, v, o);
        if (lane == 0) sh.warp[w] = v;
        __syncthreads();
        if (tid < 32) {
            unsigned long long t = lane < kVerifyWarps ? sh.warp[lane] : 0;
#pragma unroll
            for (int o = 16; o; o /= 2) t += __shfl_xor_sync(~0u, t, o);
            if (tid == 0) sh.cta[turn & 1] = t;
        }
        // (the entry written two calls ago was read before the last barrier)
        cluster.sync();
        // every warp fetches all entries at once, a lane each
        unsigned long long t =
            lane < nrank ? *cluster.map_shared_rank(&sh.cta[turn & 1], lane) : 0;
        before = lane < rank ? t : 0;
#pragma unroll
        for (int o = 16; o; o /= 2) {
            t += __shfl_xor_sync(~0u, t, o);
            before += __shfl_xor_sync(~0u, before, o);
        }
        ++turn;
        return t;
    };
    // r at a token of the vocabulary from a row of p and the rejections so far
    int cur = 0, got = 1, rejected = 0;
    float zc = 1.f;
    auto left_of = [&](float p, float q, int t, int k) {
        for (int i = 0; i < k; ++i) {
            if (a.q) p = fmaxf(__fsub_rn(p, __fmul_rn(sh.z[i], q)), 0.f);
            else p = sh.out[i] == t ? 0.f : p;
        }
        return p;
    };
    // the warp's run of r after the first rej rejections; its sum's part
    auto form = [&](int rej) {
        const float *p = a.p + (int64_t)(s.first + cur) * a.p_stride + lo;
        const float *q = a.q ? a.q + (int64_t)(s.first + cur) * a.q_stride + lo : nullptr;
        unsigned long long sum = 0;
        for (int i0 = w0 + lane; i0 < w1; i0 += kBatch * 32) {
            float pv[kBatch], qv[kBatch];  // loads first, all in flight
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int i = i0 + k * 32;
                pv[k] = i < w1 ? __ldg(p + i) : 0.f;
                qv[k] = i < w1 && q && rej ? __ldg(q + i) : 0.f;
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) pv[k] = unit(pv[k]), qv[k] = unit(qv[k]);
            for (int j = 0; j < rej; ++j) {  // left_of, all at once
                const float z = sh.z[j];
                const int out = q ? -1 : sh.out[j] - lo - i0;
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                    if (q) pv[k] = fmaxf(__fsub_rn(pv[k], __fmul_rn(z, qv[k])), 0.f);
                    else pv[k] = out == k * 32 ? 0.f : pv[k];
                }
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {  // (past the run: 0)
                if (i0 + k * 32 < w1) r[i0 + k * 32] = pv[k];
                sum += fixed(pv[k]);
            }
        }
        return sum;
    };
    int held = -1;  // rejections that r in shared memory has seen (-1: not formed)
    unsigned long long total = 0;  // the sum of that r
    for (int j = 1; j < s.n; ++j) {
        if (sh.parent[j] != cur) continue;
        const int t = sh.token[j];
        const float have = left_of(sh.pt[j], sh.qt[j], t, rejected);
        const float d = a.q ? __fmul_rn(sh.qt[j], zc) : zc;
        if (__fmul_rn(sh.u[j], d) < have) {
            if (rank == 0 && tid == 0) a.path[s.first + got] = j;
            ++got;
            cur = j, rejected = 0, zc = 1.f, held = -1;
            continue;
        }
        // rejected: what is left without it
        __syncthreads();
        if (tid == 0) sh.z[rejected] = zc, sh.out[rejected] = t;
        __syncthreads();
        unsigned long long sum = 0;
        if (held == rejected && a.q) {  // one step on from the r at hand
            const float *q = a.q + (int64_t)(s.first + cur) * a.q_stride + lo;
            for (int i0 = w0 + lane; i0 < w1; i0 += kBatch * 32) {
                float qv[kBatch];
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                    const int i = i0 + k * 32;
                    qv[k] = i < w1 ? __ldg(q + i) : 0.f;
                }
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                    const int i = i0 + k * 32;
                    const float have = i < w1 ? r[i] : 0.f;
                    const float x = fmaxf(__fsub_rn(have, __fmul_rn(zc, unit(qv[k]))), 0.f);
                    if (i < w1) r[i] = x;
                    sum += fixed(x);
                }
            }
        } else {
            sum = form(rejected + 1);
        }
        sum = cluster_sum(sum);
        if (sum) {
            held = ++rejected, total = sum;
            zc = (float)((double)(long long)sum * 0x1p-44);
        } else {
            held = -1;  // r and z stay as they were
        }
    }
    if (held != rejected) total = cluster_sum(form(rejected));
    // The first token whose running sum passes the goal.  The warps' sums are
    // there with the total; the warp whose run holds the goal gives its lanes
    // a run each (an odd number of tokens, so that they fall on different
    // banks), and the lane that holds it walks its own.
    const unsigned long long goal = (total >> 31) * u + (((total & 0x7FFFFFFFull) * u) >> 31);
    unsigned long long from = before;
    for (int i = 0; i < w; ++i) from += sh.warp[i];
    if (goal >= from && goal < from + sh.warp[w]) {
        const int per = ((seg + 31) / 32) | 1;
        const int r0 = min(w0 + lane * per, w1), r1 = min(r0 + per, w1);
        unsigned long long mine = 0;
        __syncwarp();
        for (int i0 = r0; i0 < r1; i0 += kBatch) {
#pragma unroll
            for (int k = 0; k < kBatch; ++k) mine += i0 + k < r1 ? fixed(r[i0 + k]) : 0;
        }
        unsigned long long upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const unsigned long long v = __shfl_up_sync(~0u, upto, o);
            if (lane >= o) upto += v;
        }
        unsigned long long sum = from + upto - mine;
        if (goal >= sum && goal < sum + mine) {
            int i = r0;
            for (; i < r1 - 1; ++i) {
                sum += fixed(r[i]);
                if (sum > goal) break;
            }
            a.next[b] = lo + i;
        }
    }
    if (rank == 0) {
        for (int i = tid; i < s.n; i += kVerifyThreads)
            if (i == 0 || i >= got) a.path[s.first + i] = i ? -1 : 0;
        if (tid == 0) {
            a.count[b] = got;
            if (total == 0) a.next[b] = V - 1;
        }
    }
    cluster.sync();  // no CTA leaves while another may read its sums
}

cudaError_t verify(const VerifyArgs &a, cudaStream_t s) {
    // CTAs of a sequence: up to 16, each with 4096 words or more, and about two
    // an SM in all; a CTA's run is 32768 words (128 KB) at most.  (One chain of
    // 32000 words: 8 CTAs 6.6 us, 16 6.4, 2 11.0; 32 chains: 8 each 9.4, 16
    // 20.5, 2 12.1.  32 chains of 128256 words: 8 each 16.0 us, 16 28.0; 64 of
    // 32000: 4 each 11.7, 8 15.1.)
    int ctas = 1;
    while (ctas < kMaxCluster && ctas * 4096 < a.vocab &&
           (2 * ctas * a.nseq <= kMostCtas || ctas * kMostWords < a.vocab))
        ctas *= 2;
    const int chunk = (a.vocab + ctas - 1) / ctas;
    const int smem = 4 * chunk;
    static std::mutex mu;
    static bool configured[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (dev < 0 || dev >= 64 || !configured[dev]) {
            e = cudaFuncSetAttribute(kq_verify_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     4 * kMostWords);
            if (e == cudaSuccess)
                e = cudaFuncSetAttribute(kq_verify_kernel,
                                         cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e != cudaSuccess) return e;
            if (dev >= 0 && dev < 64) configured[dev] = true;
        }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.nseq * ctas));
    cfg.blockDim = dim3(kVerifyThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kq_verify_kernel, a, chunk);
}

}  // namespace kqd
