// kq_prompt_attn.cuh -- attention of whole prompts (kq_prompt_attention): what
// its kernels share, and the kernel of one block a CTA: f32 at every width, 16 bits
// at width 256 (kq_prompt_pairs.cuh has the others).
//
//   out_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = 2^(s_ij - m_i),  j <= limit of i
//
// Work: an item is up to 128 rows that share a key head, T tokens of a
// sequence by the query heads of the group (head fastest), so that few tokens
// fill a tile where heads are shared.  A sequence's last items come first, as
// they are the longest.  An item goes over its keys from the last to the first
// in tiles, with the running maximum m and sum of a softmax; where there are
// fewer items than SMs the keys are cut into parts, whose results are joined by
// a second kernel.
//
// The rows are the 128 lanes of an accumulator, a thread each.  Queries and
// probabilities are the first operand, in tensor memory, keys and values the
// second, in shared memory.  A warp issues S = Q K of each tile as soon as the
// softmax warps have taken an earlier one into registers, another O = P V.  In
// f32 O of a tile starts at zero and is added to the row's f32 sums in registers,
// by warps of their own, with the correction of the running maximum: the sums are
// rounded to nearest, whatever the tensor core's additions do over thousands of
// steps.
//
// f32 (two f16 terms hi + lo, after a scaling by a power of two):
//   S = Qlo Khi + Qhi Klo + Qhi Khi,  O = Plo Vhi + Phi Vlo + Phi Vhi
// the small products first, as the tensor core cuts its sums off at each step
// (4097 keys of width 128, off by 4.9e-7 in all; the other order 1.8e-6).
// Keys and values are split once, by a kernel before, into tiles as the
// products take them (a sequence's 64 or 32 tokens of a head, zeros past its
// end), with the tile's powers of two.  Where a tile's tokens lie further apart
// than 2^kApart, each has a power of its own, as rows before the larger ones do
// not attend them: a column of S is scaled by its token's, and of a row's P each
// by its token's, so that the largest product with a value's largest comes to
// 2^14; O of the tile then has the row's factor.  The query is multiplied by scale *
// log2(e) in f32 first, so that what follows only multiplies by powers of two,
// and the difference to the maximum is one rounding, however large both are.
//
// 16-bit types are copied as they are, by tensor copies, and O adds up in tensor
// memory, corrected when a maximum has grown by 2^8 or more; until then
// probabilities are held up to 2^8 times as large, in the sum too.  Those that
// become f16 are held times 2^7 besides, as f16 has few bits below 2^-14.
//
// Bound by the products and what stands between two of them.  f32, 4097 tokens,
// 32 / 2 heads of 128: 315 us, 437 TFLOP/s of the formula and three times that of
// products; the tensor core is at work 61% of the time, a tile takes about 2000
// clocks for 1536 of products.  bf16 at width 256, three prompts of up to 3001
// tokens behind 500, 16 / 4 heads: 239 us, 1014 TFLOP/s; a tile takes 1600 clocks
// for 1024 of products: S waits 340 for the one before to be taken, and then runs
// beside O.  (S and, two tiles later, O by one warp: 266 us; O not before the S of
// one or two tiles on is done: 247.  Clusters of two CTAs, each copying a half of
// a tile to both: 279, as a slot waits for both.)
//
// NaN and infinities must not reach rows that do not attend them (0 * inf):
// values that are not finite are zeros in the tile (f32: all tiles; 16 bits:
// those that some row sees in part), and rows that attend them add them in the
// end.
#pragma once

#include <cuda.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "kq_decode.cuh"
#include "kq_host.h"
#include "kq_prompt_launch.h"
#include "kq_tc5.cuh"
#include "kq_types.cuh"

namespace kqp {

using kqd::quiet_nan;

constexpr int kRows = 128;  // rows of an item
constexpr float kLazy = 8.f;  // 16 bits: log2 of the growth of a maximum that is not corrected
constexpr float kLog2E = 1.44269504088896340736f;

// f32: how far apart (log2 of their largest values) a tile's tokens may lie that
// have one power of two.  A token's values are held to 2^-39 of the tile's
// largest then, to 2^-27 of the token's.
constexpr int kApart = 12;

// Powers of two of a tile of an f32 call.
struct TileInfo {
    int ek;      // keys = stored * 2^ek
    int kstate;  // kKeysApart
    int vstate;  // kValuesApart; kSomeNotFinite: zeros in the tile
    float vf;    // values * 2^-15 = stored * vf
};
constexpr int kKeysApart = 1, kValuesApart = 2, kSomeNotFinite = 4;
// Each token's, where they are apart: keys = stored * 2^k, values * 2^15 = stored * 2^v.
struct alignas(16) TilePowers {
    int16_t k[64], v[64];
};

struct PromptArgs {
    CUtensorMap qmap, kmap, vmap;  // 16-bit types
    const int32_t *start, *kstart;
    const void *q, *v;
    int64_t q_stride, k_stride, v_stride;
    const void *k;
    void *out;
    uint8_t *tiles;  // f32: [slot][kv_heads][tile]
    TileInfo *info;  // f32: [slot][kv_heads]
    TilePowers *powers;  // the same
    float *part;     // splits > 1
    int32_t nseq, ntok, nkeys, q_heads, kv_heads;
    int32_t per;      // query heads of a key head
    int32_t hb;       // of them in an item
    int32_t hblocks;  // runs of hb heads
    int32_t tok;      // tokens of an item (equally many in each of its blocks of 128 rows)
    int32_t splits;
    int32_t items;    // items in all, at most
    float scale;      // with its sign
    float scale_m;    // f32: scale times log2(e) = scale_m * 2^scale_e, |scale_m| in 0.5..1,
    int32_t scale_e;  // or 0
    unsigned int *err;
    unsigned long long wait_ns;
    uint32_t suspend_ns;
};

// A run of rows and the keys they see, as all threads of a CTA read it.
struct Item {
    int seq, first, n, kfirst, m;  // the sequence, its tokens and keys
    int tok0, nt;                  // the item's tokens, of the sequence's
    int head, hq, nh;              // key head; first query head, how many
    int found;

    // Row r: its token (of the sequence) and head (of the item).
    __device__ __forceinline__ bool row(int hb, int r, int &t, int &h) const {
        t = r / hb, h = r - t * hb;
        t += tok0;
        return t < tok0 + nt && h < nh;
    }
    // The last key that token t attends; keys that the item attends.
    __device__ __forceinline__ int limit(int t) const { return m - n + t; }
    __device__ __forceinline__ int keys() const { return max(0, min(m, m - n + tok0 + nt)); }
};

__device__ __forceinline__ int scan_max(int x, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int v = __shfl_up_sync(~0u, x, o);
        if (lane >= o) x = max(x, v);
    }
    return x;
}

// Where a walk over the sequences is: at number b0, with the largest starts
// before it, and the blocks of rows before it.
struct Place {
    int b0 = 0, s = 0, k = 0, blocks = 0;
};
// N sequences: first token and end, first key and end.
template <int N>
struct Some {
    int b, lo[N], hi[N], klo[N], khi[N];
};

// Walks the sequences from `p` on, N a lane and 32 N at a time (empty ones past
// the last), until body(Some) returns true; p is then where it was.  A start
// counts as the largest so far, within what there is.  By one warp.
template <int N, class F>
__device__ __forceinline__ void walk(const PromptArgs &a, int lane, Place &p, F &&body) {
    while (p.b0 < a.nseq) {
        Some<N> q;
        q.b = p.b0 + N * lane;
        int x[N + 1], y[N + 1];
#pragma unroll
        for (int e = 0; e <= N; ++e) {  // (all loads at once)
            const int b = min(q.b + e, a.nseq);
            x[e] = __ldg(a.start + b), y[e] = a.kstart ? __ldg(a.kstart + b) : 0;
        }
        auto run = [&](int (&v)[N + 1], int all, int before, int (&lo)[N], int (&hi)[N]) {
            int most = 0;
#pragma unroll
            for (int e = 0; e <= N; ++e) {
                v[e] = min(max(v[e], 0), all);
                if (e < N) most = max(most, v[e]);
            }
            const int upto = scan_max(most, lane);
            const int prev = __shfl_up_sync(~0u, upto, 1);
            lo[0] = max(v[0], lane ? max(prev, before) : before);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                hi[e] = max(lo[e], v[e + 1]);
                if (e + 1 < N) lo[e + 1] = hi[e];
            }
        };
        run(x, a.ntok, p.s, q.lo, q.hi);
        if (a.kstart) {
            run(y, a.nkeys, p.k, q.klo, q.khi);
        } else {
#pragma unroll
            for (int e = 0; e < N; ++e) q.klo[e] = q.lo[e], q.khi[e] = q.hi[e];
        }
        if (body(q)) return;
        p.b0 += 32 * N;
        p.s = __shfl_sync(~0u, q.hi[N - 1], 31), p.k = __shfl_sync(~0u, q.khi[N - 1], 31);
    }
}

// Item `i` of the call into shared memory, by a warp; false (and found = 0) past
// the last.  p: where the walk for any other item ended, or the beginning.
template <int N>
__device__ __forceinline__ bool find_item(const PromptArgs &a, int i, Item &it, int lane, Place &p) {
    const int across = a.kv_heads * a.hblocks;
    const int blk = i / across, h = i - blk * across;
    if (blk < p.blocks) p = Place();  // (the walk is past it)
    if (lane == 0) it.found = 0;
    __syncwarp();
    walk<N>(a, lane, p, [&](const Some<N> &q) {
        int blocks[N], upto = 0;
#pragma unroll
        for (int e = 0; e < N; ++e) blocks[e] = (q.hi[e] - q.lo[e] + a.tok - 1) / a.tok, upto += blocks[e];
        const int mine = upto;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int v = __shfl_up_sync(~0u, upto, o);
            if (lane >= o) upto += v;
        }
        upto += p.blocks;
        const unsigned past = __ballot_sync(~0u, upto > blk);
        if (past == 0) {
            p.blocks = __shfl_sync(~0u, upto, 31);
            return false;
        }
        if (lane == __ffs(past) - 1) {
            int end = upto - mine;
            bool there = false;
#pragma unroll
            for (int e = 0; e < N; ++e) {
                end += blocks[e];
                if (there || end <= blk) continue;
                there = true;
                const int at = end - 1 - blk;  // the last block first
                it.seq = q.b + e, it.first = q.lo[e], it.n = q.hi[e] - q.lo[e];
                it.kfirst = q.klo[e], it.m = q.khi[e] - q.klo[e];
                it.tok0 = at * a.tok, it.nt = min(a.tok, it.n - it.tok0);
                it.head = h / a.hblocks;
                const int run = h - it.head * a.hblocks;
                it.hq = it.head * a.per + run * a.hb, it.nh = min(a.hb, a.per - run * a.hb);
                it.found = 1;
            }
        }
        return true;
    });
    __syncwarp();
    return it.found != 0;
}
__device__ __forceinline__ bool find_item(const PromptArgs &a, int i, Item &it, int lane, Place &p) {
    // (Four sequences a lane where there are many: 4096 prompts of 8 tokens, 16 / 4
    // heads of 256, f32, 6.0 ms with one, 3.6 with four.)
    return a.nseq > 32 ? find_item<4>(a, i, it, lane, p) : find_item<1>(a, i, it, lane, p);
}
// The first number of `given` (a CTA's; -1: no more) that find(number) finds
// something for; -1 if there is none.  Grids go by the most items that there may
// be, and numbers past the last need no CTA.  But no order of the numbers is
// promised: one after those may have an item.
template <class G, class F>
__device__ __forceinline__ int first_found(G &&given, F &&find) {
    int u = given();
    while (u >= 0 && !find(u)) u = given();
    return u;
}

// 32-bit words of two 16-bit values of which one is not finite.
template <class T>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
    constexpr uint32_t kExp = std::is_same<T, __half>::value ? 0x7C007C00u : 0x7F807F80u;
    constexpr uint32_t kOne = std::is_same<T, __half>::value ? 0x04000400u : 0x00800080u;
    return ((w & kExp) + kOne) & 0x80008000u;  // the exponent's carry
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Two f16 terms of two values, as pairs (what is not finite has no lo).
__device__ __forceinline__ void split2(float a, float b, uint32_t &hi, uint32_t &lo) {
    hi = pack2<__half>(a, b);
    const float2 f = unpack2<__half>(hi);
    lo = pack2<__half>(a - f.x, b - f.y);
}

// Another CTA of the grid that has not begun, whose work this one takes over
// instead: asked for, its number 16 bytes later at `to`.
__device__ __forceinline__ void ask_for_cta(uint32_t to, uint32_t bar) {
    asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(to),
        "r"(bar)
        : "memory");
}
// The answer: the CTA's number, or -1 where there is none (then none is asked
// for again).
__device__ __forceinline__ int cta_given(uint32_t at) {
    int x;
    asm volatile(
        "{\n .reg .b128 h;\n .reg .pred p;\n .reg .b32 a, b, c, d;\n"
        " ld.shared.b128 h, [%1];\n"
        " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n"
        " mov.b32 a, -1;\n"
        " @p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {a, b, c, d}, h;\n"
        " mov.b32 %0, a;\n}\n"
        : "=r"(x)
        : "r"(at)
        : "memory");
    return x;
}

// ------------------------------------------------------- splitting f32
// The largest finite magnitude's exponent e: it is below 2^e.
__device__ __forceinline__ int exponent_of(float top, int least) {
    return max((int)(__float_as_uint(top) >> 23 & 255) - 126, least);
}

// Bytes of a tile's keys, or values, of both terms.
__host__ __device__ constexpr int f32_tile_tokens(int d) { return d == 256 ? 32 : 64; }
constexpr int kSplitThreads = 256;

// One CTA per slot, head, and keys or values: 64 (32) tokens of a sequence into
// hi and lo tiles.  A sequence's slots begin at first key / tokens + its number.
// 4097 tokens of 2 heads of 128: 8 us (latency: a walk, one round of loads, one
// of stores).
template <int D>
__global__ void __launch_bounds__(kSplitThreads)
    kq_prompt_split(const __grid_constant__ PromptArgs a) {
    constexpr int TK = f32_tile_tokens(D), kPart = TK * D * 4;
    constexpr int kEach = TK * D / 4 / kSplitThreads;  // float4 of a thread
    constexpr int kLanes = D / 4 < 32 ? D / 4 : 32;  // of a warp, that share a token
    __shared__ int found[4];
    __shared__ uint32_t tops[TK];  // each token's largest finite magnitude
    __shared__ int bad;
    const int tid = threadIdx.x, lane = tid & 31;
    const int slot = blockIdx.x, head = blockIdx.y;
    const bool values = blockIdx.z != 0;
    kq::allow_dependents();
    if (tid == 0) found[0] = 0, bad = 0;
    if (tid < TK) tops[tid] = 0;
    if (tid < 32) {
        __syncwarp();
        Place p;
        walk<4>(a, lane, p, [&](const Some<4> &q) {
            bool here = false;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int base = q.klo[e] / TK + q.b + e, tiles = (q.khi[e] - q.klo[e] + TK - 1) / TK;
                if (q.b + e < a.nseq && slot >= base && slot < base + tiles) {
                    here = true;
                    found[1] = q.klo[e] + (slot - base) * TK, found[2] = min(TK, q.khi[e] - found[1]);
                    found[0] = 1;
                }
            }
            return __any_sync(~0u, here) != 0;
        });
    }
    __syncthreads();
    if (!found[0]) return;
    const int first = found[1], held = found[2];
    const float *x = static_cast<const float *>(values ? a.v : a.k);
    const int64_t stride = values ? a.v_stride : a.k_stride;
    float4 v[kEach];
    bool odd = false;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int at = tid + i * kSplitThreads, t = at / (D / 4), e = at % (D / 4);
        v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (t < held)
            v[i] = __ldg(reinterpret_cast<const float4 *>(x + (int64_t)(first + t) * stride +
                                                          (int64_t)head * D) + e);
        float *f = &v[i].x, top = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float m = fabsf(f[k]);
            if (m < INFINITY) {
                top = fmaxf(top, m);
            } else {
                odd = true;
                if (values) f[k] = 0.f;
            }
        }
        uint32_t its = __float_as_uint(top);
        if constexpr (kLanes == 32) {
            its = __reduce_max_sync(~0u, its);
        } else {
#pragma unroll
            for (int o = kLanes / 2; o; o /= 2) its = max(its, __shfl_xor_sync(~0u, its, o));
        }
        if (lane % kLanes == 0) atomicMax(&tops[t], its);
    }
    const bool any = __any_sync(~0u, odd);
    if (lane == 0 && any) atomicOr(&bad, 1);
    __syncthreads();
    // The tile's largest and its tokens' least (tokens of zeros have no say).
    const uint32_t one = tops[lane], two = TK > 32 ? tops[lane + TK - 32] : one;
    const uint32_t most = __reduce_max_sync(~0u, max(one, two));
    const uint32_t least = __reduce_min_sync(~0u, min(one ? one : ~0u, two ? two : ~0u));
    const bool apart = most && (int)(most >> 23) - (int)(least >> 23) > kApart;
    // (values' least: their factor is 2^-15 smaller)
    const int from = values ? -96 : -111;
    const int ex = exponent_of(__uint_as_float(most), from);
    uint8_t *to = a.tiles + ((int64_t)slot * a.kv_heads + head) * (2 * kPart) + (values ? kPart : 0);
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int at = tid + i * kSplitThreads, t = at / (D / 4), e = at % (D / 4);
        const int its = apart ? exponent_of(__uint_as_float(tops[t]), from) : ex;
        const float up = __uint_as_float((uint32_t)(127 + 15 - its) << 23);
        uint2 hi, lo;
        split2(v[i].x * up, v[i].y * up, hi.x, lo.x);
        split2(v[i].z * up, v[i].w * up, hi.y, lo.y);
        if (odd) {  // (inf - inf)
            lo.x = lo.x & (not_finite<__half>(hi.x) ? 0u : ~0u);
            lo.y = lo.y & (not_finite<__half>(hi.y) ? 0u : ~0u);
        }
        uint8_t *p = to + (e / 16) * (TK * 128) + tile_at(t, (e % 16) / 2) + (e & 1) * 8;
        *reinterpret_cast<uint2 *>(p) = hi;
        *reinterpret_cast<uint2 *>(p + kPart / 2) = lo;
    }
    TileInfo *info = a.info + (int64_t)slot * a.kv_heads + head;
    if (tid == 0) {
        if (values) {
            info->vf = __uint_as_float((uint32_t)(127 + ex - 30) << 23);
            info->vstate = (bad ? kSomeNotFinite : 0) | (apart ? kValuesApart : 0);
        } else {
            info->ek = ex - 15, info->kstate = apart ? kKeysApart : 0;
        }
    }
    if (apart && tid < TK) {
        const int its = exponent_of(__uint_as_float(tops[tid]), from);
        TilePowers *powers = a.powers + (int64_t)slot * a.kv_heads + head;
        if (values) powers->v[tid] = (int16_t)its;
        else powers->k[tid] = (int16_t)(its - 15);
    }
}

// --------------------------------------------------- any type and width
template <class T, int D>
struct Rows {
    static constexpr bool kTwo = std::is_same<T, float>::value;  // terms
    using H = typename std::conditional<kTwo, __half, T>::type;  // of the products
    static constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    static constexpr int TK = kTwo ? f32_tile_tokens(D) : 64;
    static constexpr int kTerm = TK * D * 2;                 // one term of a tile's keys or values
    static constexpr int kPart = kTerm * (kTwo ? 2 : 1);
    // columns of tensor memory: Q (lo in shared memory at width 256), S, P, O,
    // and how many of each it holds
    static constexpr bool kLoShared = kTwo && D == 256;
    static constexpr int kQCols = kTwo && !kLoShared ? D : D / 2;
    static constexpr int kPCols = kTwo ? TK : TK / 2;
    // (f32 at width 128: two of O and one of S and P; one of O, which is read
    // before it is formed again, and two of S and P measured the same)
    static constexpr int OB = kTwo && D <= 128 ? 2 : 1;
    static constexpr int PB = kTwo && D == 128 ? 1 : 2;
    static constexpr int SB = kQCols + 2 * TK + PB * kPCols + OB * D <= 512 ? 2 : 1;
    static constexpr int kS = kQCols, kP = kS + SB * TK, kO = kP + PB * kPCols;
    // Softmax warps: four, or four for each second tile, which hand each other
    // the rows' references (so that one tile's softmax is not what S waits for).
    static constexpr int SG = kTwo ? 1 : 2, kSoft = 4 * SG;
    static constexpr int OW = D == 256 ? 8 : 4;              // warps that write rows: f32 those that sum O
    static constexpr int OC = D * 4 / OW;                    // columns of each
    static constexpr int kFirst = kTwo ? 4 + OW : kSoft;     // S, copies, O, one that cleans
    static constexpr int kThreads = 32 * (kFirst + 4);
    static constexpr int kControl = 7168, kQLo = kLoShared ? kRows * D * 2 : 0;
    static constexpr int kRing = kControl + kQLo;
    static constexpr int kRoom = (227 * 1024 - 1024 - kRing) / kPart;
    static constexpr int kSlots = kRoom < 8 ? kRoom : 8;
    static constexpr int kBytes = kRing + kSlots * kPart + 1024;
    // Copies: tile i's keys are copy 2 i, its values 2 i + 1.  f32: slots by turns.
    // 16 bits: a half of the slots for each, as keys are used up to two tiles ahead
    // of the values (by turns: 255 us against 239 for three prompts).
    static constexpr int kEach = kSlots / 2;
    static __device__ __forceinline__ int slot(int k) {
        return kTwo ? k % kSlots : (k & 1) * kEach + (k >> 1) % kEach;
    }
    static __device__ __forceinline__ int turn(int k) { return kTwo ? k / kSlots : (k >> 1) / kEach; }
    // f32 up to width 128: an item's queries are copied to the ring's last two
    // slots first.  (Each thread its own row from memory: 318 against 314 us for
    // 4097 tokens.)
    static constexpr bool kQStaged = kTwo && D <= 128;
    static constexpr int kFree = kQStaged ? kSlots - 2 : kSlots;  // slots that are free meanwhile
    static constexpr int kQStage = kRing + (kSlots - 2) * kPart;
    static_assert(kO + OB * D <= 512 && kSlots >= 4 && (kTwo || (SB == 1 && PB == SG && OW == kSoft)), "layout");
    static_assert(!kQStaged || kRows * D * 4 <= 2 * kPart, "layout");
};

struct RowsShared {
    uint4 answer;  // of ask_for_cta
    Item item;
    uint64_t full[8], empty[8], sdone[2], sfree[2], pready[2], pfree[2], odone[2], ofree[2], cready[4],
        vraw[4], vclean[4], handed[8], ldone, given, qfull, drain[2];
    uint32_t tmem;
    int dead, bad;
    int unit;  // the number of the CTA whose work this is, where it is not its own
    // f32, of tile i & 3: the factor of what was summed before; 16 bits, of tile
    // i & 1: the rows' references after it
    float corr[4][kRows];
    float vf[4][kRows];  // f32: the row's factor of O of that tile, where its values are apart
    float m[2][kRows], l[2][kRows];  // of each softmax warps' tiles
};
static_assert(sizeof(RowsShared) <= 7168, "layout");

template <class T, int D>
__global__ void __launch_bounds__(Rows<T, D>::kThreads, 1)
    kq_prompt_rows(const __grid_constant__ PromptArgs a) {
    using M = Rows<T, D>;
    using H = typename M::H;
    constexpr bool kTwo = M::kTwo;
    constexpr int TK = M::TK, SB = M::SB, PB = M::PB, OB = M::OB;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024 - (kq::smem_addr(smem_raw) & 1023)) & 1023);
    RowsShared &cm = *reinterpret_cast<RowsShared *>(smem);
    const uint32_t base = kq::smem_addr(smem);
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    auto bar = [&](const uint64_t &b) { return kq::smem_addr(&b); };

    int unit = blockIdx.x;
    Place place;
    if (w == 0) {
        find_item(a, unit / a.splits, cm.item, lane, place);
    } else if (w == 1) {  // a lane a barrier, or a few
        if (lane < 8) {
            kq::mbar_init(bar(cm.full[lane]), 1), kq::mbar_init(bar(cm.empty[lane]), 1);
        } else if (lane < 10) {
            const int i = lane - 8;
            kq::mbar_init(bar(cm.sdone[i]), 1), kq::mbar_init(bar(cm.sfree[i]), 4);
            kq::mbar_init(bar(cm.pready[i]), 4), kq::mbar_init(bar(cm.pfree[i]), 1);
            kq::mbar_init(bar(cm.odone[i]), 1), kq::mbar_init(bar(cm.ofree[i]), M::OW);
            kq::mbar_init(bar(cm.drain[i]), 1);
        } else if (lane < 14) {
            const int i = lane - 10;
            kq::mbar_init(bar(cm.cready[i]), 4);
            kq::mbar_init(bar(cm.vraw[i]), 1), kq::mbar_init(bar(cm.vclean[i]), 1);
        } else if (lane == 14) {
            kq::mbar_init(bar(cm.ldone), kTwo ? 4 : M::kSoft + 1);
            kq::mbar_init(bar(cm.given), 1), kq::mbar_init(bar(cm.qfull), 1);
            cm.dead = cm.bad = 0;
        } else if (lane >= 16 && lane < 24) {
            kq::mbar_init(bar(cm.handed[lane - 16]), 1);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    } else if (w == M::kFirst) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                         kq::smem_addr(&cm.tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    } else if (!kTwo && w == M::kFirst + 1 && lane < 2) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(lane ? &a.vmap : &a.kmap) : "memory");
    }
    tc_before();
    __syncthreads();
    tc_after();
    if (!cm.item.found) {
        // Past the last item: CTAs that have not begun and have none either need
        // not begin.  (4096 prompts of 8 tokens, 16 / 4 heads of 256, f32: 4.0 ms if
        // they do, 3.6 so.)
        __syncthreads();  // (all have looked)
        if (w == 0) {
            int n = 0;
            unit = first_found(
                [&]() {
                    int u = -1;
                    if (lane == 0) {
                        kq::mbar_expect_tx(bar(cm.given), 16);
                        ask_for_cta(kq::smem_addr(&cm.answer), bar(cm.given));
                        bool there = kq::mbar_wait(bar(cm.given), n & 1, kq::kWaitLimitNs);
                        if (!there) {
                            atomicOr(a.err, 1u);
                            there = kq::mbar_wait(bar(cm.given), n & 1, kq::kWaitLimitNs);
                        }
                        if (there) u = cta_given(kq::smem_addr(&cm.answer));
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    }
                    ++n;
                    return __shfl_sync(~0u, u, 0);
                },
                [&](int u) { return find_item(a, u / a.splits, cm.item, lane, place); });
            if (lane == 0) cm.unit = unit;
        }
        __syncthreads();
        unit = cm.unit;
        if (unit < 0) {
            if (w == M::kFirst)
                asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(cm.tmem));
            if constexpr (kTwo) kq::wait_prerequisites();
            return;
        }
    }
    const Item it = cm.item;
    const int rank = unit % a.splits;
    const uint32_t tmem = cm.tmem;

    auto dead = [&]() { return *(volatile int *)&cm.dead != 0; };
    auto wait = [&](const uint64_t &b, int phase) {  // the completion of the barrier's phase
        if (kq::mbar_test(bar(b), phase & 1) || dead()) return;
        if (!kq::mbar_wait_awake(bar(b), phase & 1, a.wait_ns, a.suspend_ns)) {
            *(volatile int *)&cm.dead = 1;
            atomicOr(a.err, 1u);
        }
    };

    // The item's tiles, its last first: tile i of the walk is tile t1 - 1 - i
    // of the sequence.  The first `edges` of them some row sees in part.
    const int tiles = (it.keys() + TK - 1) / TK;
    const int t0 = (int)((int64_t)tiles * rank / a.splits);
    const int t1 = (int)((int64_t)tiles * (rank + 1) / a.splits);
    const int count = t1 - t0;
    const int whole = max(0, it.limit(it.tok0) + 1) / TK;  // tiles that every row sees
    const int edges = min(max(t1 - max(whole, t0), 0), count);
    const int64_t slot0 = kTwo ? (int64_t)(it.kfirst / TK + it.seq) * a.kv_heads + it.head : 0;

    // The tiles and their powers of two, which a kernel beside the beginning of this
    // one writes: plain loads, not those of memory that nobody writes meanwhile.
    if constexpr (kTwo) kq::wait_prerequisites();
    int copied = 0;  // copies that this warp has begun (16 bits: of keys, or of values)

    // f32: tile t's state, and whether some tile of the CTA's has tokens apart.
    // (The loops over tiles are there twice: with what such tiles take in the
    // only one, 4097 tokens of 32 / 2 heads of 128 took 326 us on the GPU against
    // 294 without and 301 so.)
    auto state_of = [&](int t) {
        const TileInfo *p = &a.info[slot0 + (int64_t)t * a.kv_heads];
        return p->kstate | p->vstate;
    };
    auto some_apart = [&]() {
        int all = 0;
        for (int t = t0 + lane; t < t1; t += 32) all |= state_of(t);
        return __any_sync(~0u, all & (kKeysApart | kValuesApart)) != 0;
    };

    // The rows' results, by warp n of those that write: its columns of O.
    auto write_rows = [&](float (&O)[M::OC], bool bad, int n) {
        const int r = 32 * (n & 3) + lane, c0 = n / 4 * M::OC;
        int tok, hq;
        const bool on = it.row(a.hb, r, tok, hq);
        wait(cm.ldone, 0);
        float l, m;
        if constexpr (kTwo) {
            l = cm.l[0][r], m = cm.m[0][r];
        } else {  // both halves' sums, of the last tile's reference
            const int last = count > 0 ? (count - 1) & 1 : 0;
            m = cm.m[last][r];
            const float other = cm.m[last ^ 1][r];
            const float f = other == m ? 1.f : other == -INFINITY ? 0.f
                                             : exp2_fast((other - m) * (fabsf(a.scale) * kLog2E));
            l = fmaf(cm.l[last ^ 1][r], f, cm.l[last][r]);
        }
        const int limit = on ? it.limit(tok) : -1;
        if constexpr (!kTwo) bad = *(volatile int *)&cm.bad != 0;
        if (bad && on) {
            // values that are not finite, of the tiles that left them out
            for (int t = kTwo ? t0 : t1 - edges; t < t1; ++t) {
                if (kTwo && !(a.info[slot0 + (int64_t)t * a.kv_heads].vstate & kSomeNotFinite)) continue;
                for (int j = t * TK; j < min((t + 1) * TK, limit + 1); ++j) {
                    const T *v = static_cast<const T *>(a.v) + (int64_t)(it.kfirst + j) * a.v_stride +
                                 (int64_t)it.head * D + c0;
#pragma unroll
                    for (int k = 0; k < M::OC; ++k) {
                        const float x = to_f32<T>(v[k]);
                        if (!(fabsf(x) < INFINITY)) O[k] += x;
                    }
                }
            }
        }
        const bool lost = __any_sync(~0u, dead());
        if (lost) l = quiet_nan();
        if (a.splits > 1) {
            float *part = a.part + (int64_t)unit * kRows * (D + 2);
            // by values, of 32 rows each: part[32 rows][D][32]
            float *to = part + (r - lane) * D + c0 * 32 + lane;
#pragma unroll
            for (int k = 0; k < M::OC; ++k) to[32 * k] = O[k];
            if (c0 == 0) part[kRows * D + r] = m, part[kRows * (D + 1) + r] = l;
        } else {
            // (a row that attends something and has no sum has scores of
            // -infinity only)
            float inv = limit < 0 ? 0.f : __fdiv_rn(kTwo ? 32768.f : 1.f, l);
            if (lost) inv = quiet_nan();
            T *to = static_cast<T *>(a.out) + ((int64_t)(it.first + it.tok0) * a.q_heads + it.hq) * D + c0;
            const uint32_t place = (tok - it.tok0) * a.q_heads + hq, rows = __ballot_sync(~0u, on);
            // Rows go out whole, through shared memory (every copy there was used
            // up by the last O): a lane's own row in pieces of 32 bytes took 3 us.
            constexpr int kRow = M::OC * sizeof(T), kLanes = kRow / 16;  // bytes; lanes of a row
            uint8_t *stage = smem + M::kRing + n * 32 * kRow;
            static_assert(M::OW * 32 * kRow <= M::kSlots * M::kPart && 32 % kLanes == 0, "layout");
            if (lost) {  // (copies may still come)
                for (int k = 0; k < M::OC && on; ++k) to[(int64_t)place * D + k] = from_f32<T>(inv);
            } else {
#pragma unroll
                for (int k = 0; k < kLanes; ++k) {
                    uint4 x;
                    uint32_t *q = &x.x;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if constexpr (kTwo) q[e] = __float_as_uint(O[4 * k + e] * inv);
                        else q[e] = pack2<H>(O[8 * k + 2 * e] * inv, O[8 * k + 2 * e + 1] * inv);
                    }
                    *reinterpret_cast<uint4 *>(stage + lane * kRow + ((k ^ (lane & 7)) << 4)) = x;
                }
                __syncwarp();
#pragma unroll 8
                for (int k = 0; k < kLanes; ++k) {
                    const int at = k * (32 / kLanes) + lane / kLanes, c = lane % kLanes;
                    const uint4 x = *reinterpret_cast<const uint4 *>(stage + at * kRow + ((c ^ (at & 7)) << 4));
                    const uint32_t far = __shfl_sync(~0u, place, at);
                    if (rows >> at & 1)
                        *reinterpret_cast<uint4 *>(to + (int64_t)far * D + c * (16 / sizeof(T))) = x;
                }
            }
        }
    };

    if (w < M::kSoft) {
        // ------------------------------------------------- softmax warps
        const int g = w >> 2, r = 32 * (w & 3) + lane;  // (g: of which tiles)
        int tok, hq;
        const bool on = it.row(a.hb, r, tok, hq);
        const uint32_t mine = tmem + ((uint32_t)(32 * (w & 3)) << 16);
        const bool apart = kTwo && some_apart();  // (while the queries come)
        int ex = 0;
        {   // ---- the row's query into tensor memory
            const T *x = static_cast<const T *>(a.q) + (int64_t)(it.first + tok) * a.q_stride +
                         (int64_t)(it.hq + hq) * D;
            if constexpr (kTwo) {
                // (up to width 128 the row is read once)
                constexpr int kHeld = D <= 128 ? D / 4 : 16;
                const float4 *x4 = reinterpret_cast<const float4 *>(x);
                const float sc = a.scale_m;
                float4 v[kHeld];
                if constexpr (M::kQStaged) wait(cm.qfull, 0);
                auto load = [&](int i0) {
#pragma unroll
                    for (int i = 0; i < kHeld; ++i) {
                        if (!on) {
                            v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                        } else if constexpr (M::kQStaged) {
                            v[i] = *reinterpret_cast<const float4 *>(smem + M::kQStage + (i / 8) * (kRows * 128) +
                                                                     tile_at(r, i & 7));
                        } else {
                            v[i] = __ldg(x4 + i0 + i);
                        }
                    }
                };
                float top = 0.f;
#pragma unroll 1
                for (int i0 = 0; i0 < D / 4; i0 += kHeld) {
                    load(i0);
#pragma unroll
                    for (int i = 0; i < kHeld; ++i)
                        top = fmaxf(top, fmaxf(fmaxf(fabsf(v[i].x * sc), fabsf(v[i].y * sc)),
                                               fmaxf(fabsf(v[i].z * sc), fabsf(v[i].w * sc))));
                }
                ex = exponent_of(top, -111);
                const float up = __uint_as_float((uint32_t)(127 + 15 - ex) << 23);
                ex += a.scale_e;
#pragma unroll 1
                for (int i0 = 0; i0 < D / 4; i0 += kHeld) {
                    if (kHeld < D / 4) load(i0);
#pragma unroll
                    for (int i = 0; i < kHeld / 8; ++i) {
                        uint32_t hi[16], lo[16];
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const float4 e = v[8 * i + k];
                            split2(e.x * sc * up, e.y * sc * up, hi[2 * k], lo[2 * k]);
                            split2(e.z * sc * up, e.w * sc * up, hi[2 * k + 1], lo[2 * k + 1]);
                        }
                        const int at = i0 / 8 + i;  // 32 values of the row
                        tc_store16(mine + 16 * at, hi);
                        if constexpr (M::kLoShared) {
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                *reinterpret_cast<uint4 *>(smem + M::kControl + (at / 2) * (kRows * 128) +
                                                           tile_at(r, (at & 1) * 4 + k)) =
                                    make_uint4(lo[4 * k], lo[4 * k + 1], lo[4 * k + 2], lo[4 * k + 3]);
                        } else {
                            tc_store16(mine + D / 2 + 16 * at, lo);
                        }
                    }
                }
                if constexpr (M::kLoShared || M::kQStaged)
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            } else {
                const uint4 *x8 = reinterpret_cast<const uint4 *>(x);
                const uint32_t sign = a.scale < 0.f ? 0x80008000u : 0u;
                // (half a row each)
                static_assert(D == 256, "halves of a row");
                {
                    const int i = 4 * g;
                    uint4 v[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) v[k] = on ? __ldg(x8 + 4 * i + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t q[16];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            q[4 * k] = v[4 * c + k].x ^ sign, q[4 * k + 1] = v[4 * c + k].y ^ sign;
                            q[4 * k + 2] = v[4 * c + k].z ^ sign, q[4 * k + 3] = v[4 * c + k].w ^ sign;
                        }
                        tc_store16(mine + 16 * (i + c), q);
                    }
                }
            }
            tc_stored();
            tc_before();
        }
        __syncthreads();
        const int limit = on ? it.limit(tok) : -1;
        const float factor = fabsf(a.scale) * kLog2E;  // (16-bit types)
        constexpr float kUp = M::kBf16 ? 0.f : 7.f;
        const TileInfo *info = nullptr;
        int ek = 0;
        if constexpr (kTwo) {
            info = a.info + slot0;
            if (count) ek = info[(int64_t)(t1 - 1) * a.kv_heads].ek;
        }
        float m = -INFINITY, l = 0.f;
        // body(k, its power) for a tile's tokens, eight powers a load
        auto each_power = [&](const int16_t *powers, auto &&body) {
#pragma unroll
            for (int k = 0; k < TK; k += 8) {
                const int4 x = *reinterpret_cast<const int4 *>(powers + k);
                const int w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) body(k + 2 * j, (int)(int16_t)w[j]), body(k + 2 * j + 1, w[j] >> 16);
            }
        };
        auto step = [&](int i, auto far) {
            constexpr bool kFar = decltype(far)::value;
            const int t = t1 - 1 - i;
            float f = 1.f;
            int state = 0;
            if constexpr (kTwo) {
                f = __uint_as_float((uint32_t)(127 + min(max(ex - 15 + ek, -126), 127)) << 23);
                if (i + 1 < count) ek = info[(int64_t)(t - 1) * a.kv_heads].ek;
                if (kFar) state = state_of(t);
            }
            float before = -INFINITY;  // the reference after the tile before
            if constexpr (!kTwo) {
                // (Who has handed it on has also seen the S before, and the O of
                // two tiles before that: no barrier is ever two phases behind.)
                if (i > 0) {
                    wait(cm.handed[4 * (g ^ 1) + (w & 3)], (i - 1) >> 1);
                    before = cm.corr[(i - 1) & 1][r];
                }
            }
            wait(cm.sdone[i % SB], i / SB);
            tc_after();
            uint32_t d[TK];
            const uint32_t sa = mine + M::kS + TK * (i % SB), pa = mine + M::kP + M::kPCols * (i % PB);
#pragma unroll
            for (int k = 0; k < TK / 32; ++k) tc_load32(d + 32 * k, sa + 32 * k);
            tc_loaded();
            tc_before();
            __syncwarp();
            if (lane == 0) kq::mbar_arrive(bar(cm.sfree[i % SB]));
            if (kFar && (state & kKeysApart)) {  // each key's own power of two
                each_power(a.powers[slot0 + (int64_t)t * a.kv_heads].k, [&](int k, int its) {
                    d[k] = __float_as_uint(__uint_as_float(d[k]) *
                                           __uint_as_float((uint32_t)(127 + min(max(ex - 15 + its, -126), 127)) << 23));
                });
                f = 1.f;
            }
            const int seen = i < edges ? limit + 1 - t * TK : TK;  // columns that the row attends
            if (i < edges) {
#pragma unroll
                for (int k = 0; k < TK; ++k)
                    if (k >= seen) d[k] = 0xFF800000u;
            }
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int k = 0; k < TK; ++k) mx[k & 3] = fmaxf(mx[k & 3], __uint_as_float(d[k]));
            mx[0] = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
            // The reference: f32, the maximum less 15, rounded up (it is in
            // units of log 2).  16 bits: a maximum of the scores themselves,
            // which is only moved when it has grown by 2^8 or more, as O has to
            // be corrected then.
            float corr = 1.f;
            if constexpr (kTwo) {
                const float now = fmaxf(m, mx[0] == -INFINITY ? mx[0] : __fsub_ru(mx[0] * f, 15.f));
                corr = exp2_fast(m - (now == -INFINITY ? 0.f : now));
                m = now;
            } else {
                if (i >= PB) {  // the O before has read P's place
                    wait(cm.pfree[i % PB], i / PB - 1);
                    tc_after();
                }
                const float now = fmaxf(before, mx[0]);
                const bool grown = now > before && !((now - before) * factor <= kLazy);
                const float ref = grown ? now : before;
                cm.corr[i & 1][r] = ref;
                __syncwarp();
                if (lane == 0) kq::mbar_arrive(bar(cm.handed[4 * g + (w & 3)]));
                if (__any_sync(~0u, ref != m))
                    corr = ref == m ? 1.f : m == -INFINITY ? 0.f : exp2_fast((m - ref) * factor);
                m = ref;
                if (__any_sync(~0u, grown) && i > 0) {
                    const float by = !grown ? 1.f : before == -INFINITY ? 0.f : exp2_fast((before - ref) * factor);
                    wait(cm.pfree[(i - 1) % PB], (i - 1) / PB);
                    tc_after();
                    const uint32_t oa = mine + M::kO;
                    if (!__any_sync(~0u, dead())) {
#pragma unroll 4
                        for (int k = 0; k < D; k += 16) {
                            uint32_t o[16];
                            tc_load16(o, oa + k);
                            tc_loaded();
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * by);
                            tc_store16(oa + k, o);
                        }
                    }
                }
            }
            const float from = m == -INFINITY ? 0.f : m;
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < TK; ++k) {
                const float s = __uint_as_float(d[k]);
                float p = exp2_fast(kTwo ? fmaf(s, f, -from) : fmaf(s - from, factor, kUp));
                if (i < edges && k >= seen) p = 0.f;
                sum[k & 3] += p;
                d[k] = __float_as_uint(p);
            }
            l = fmaf(l, corr, (sum[0] + sum[1]) + (sum[2] + sum[3]));
            if (kFar && (state & kValuesApart)) {
                // each value's own power of two, by the exponents' bits (what is
                // not a number stays one)
                const int16_t *powers = a.powers[slot0 + (int64_t)t * a.kv_heads].v;
                auto field = [](uint32_t x) { return (int)(x >> 23); };
                int most = -1000;
                each_power(powers, [&](int k, int its) {
                    if (d[k] != 0 && field(d[k]) < 255) most = max(most, field(d[k]) + its);
                });
                const int ev = max(most - (127 + 14), -96);
                f = __uint_as_float((uint32_t)(127 + ev - 30) << 23);
                each_power(powers, [&](int k, int its) {
                    const int by = its - ev;
                    if (field(d[k]) < 255) d[k] = d[k] != 0 && field(d[k]) + by > 0 ? d[k] + ((uint32_t)by << 23) : 0u;
                });
            }
            if (kTwo && i >= PB) {  // the O before has read P's place
                wait(cm.pfree[i % PB], i / PB - 1);
                tc_after();
            }
            if constexpr (kTwo) cm.corr[i & 3][r] = corr;
            if (kFar && (state & kValuesApart)) cm.vf[i & 3][r] = f;
#pragma unroll
            for (int k = 0; k < TK / 32; ++k) {
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float p0 = __uint_as_float(d[32 * k + 2 * j]), p1 = __uint_as_float(d[32 * k + 2 * j + 1]);
                    if constexpr (kTwo) split2(p0, p1, hi[j], lo[j]);
                    else hi[j] = pack2<H>(p0, p1);
                }
                tc_store16(pa + 16 * k, hi);
                if constexpr (kTwo) tc_store16(pa + TK / 2 + 16 * k, lo);
            }
            tc_stored();
            tc_before();
            __syncwarp();
            if (lane == 0) {
                kq::mbar_arrive(bar(cm.pready[i % PB]));
                if constexpr (kTwo) kq::mbar_arrive(bar(cm.cready[i & 3]));
            }
        };
        if (apart) {
            for (int i = g; i < count; i += M::SG) step(i, std::bool_constant<kTwo>());
        } else {
            for (int i = g; i < count; i += M::SG) step(i, std::false_type());
        }
        cm.m[g][r] = m;
        cm.l[g][r] = l;
        __syncwarp();
        if (lane == 0) kq::mbar_arrive(bar(cm.ldone));
        if constexpr (!kTwo) {
            float O[M::OC];
#pragma unroll
            for (int k = 0; k < M::OC; ++k) O[k] = 0.f;
            if (count) {  // the sums are in tensor memory
                wait(cm.odone[0], 0);
                tc_after();
                if (!__any_sync(~0u, dead())) {
#pragma unroll
                    for (int k = 0; k < M::OC; k += 32)
                        tc_load32(reinterpret_cast<uint32_t *>(O) + k, mine + M::kO + g * M::OC + k);
                    tc_loaded();
                    tc_before();
                }
            }
            write_rows(O, false, w);
        }
    } else if (kTwo && w < M::kFirst) {
        // ------------------------------------------- the sums of O, and out
        if constexpr (kTwo && D == 256) asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
        const bool apart = kTwo && some_apart();
        __syncthreads();
        const int r = 32 * (w & 3) + lane, c0 = (w - 4) / 4 * M::OC;
        const uint32_t mine = tmem + ((uint32_t)(32 * (w & 3)) << 16) + M::kO + c0;
        int tok, hq;
        const bool on = it.row(a.hb, r, tok, hq);
        float O[M::OC];
#pragma unroll
        for (int k = 0; k < M::OC; ++k) O[k] = 0.f;
        bool bad = false;
        auto sums = [&](auto far) {
            constexpr bool kFar = decltype(far)::value;
            const TileInfo *info = a.info + slot0;
            float vf = 1.f;
            int state = 0;
            auto look = [&](int i) {
                const TileInfo *p = info + (int64_t)(t1 - 1 - i) * a.kv_heads;
                vf = p->vf, state = p->vstate;
            };
            if (count) look(0);
            for (int i = 0; i < count; ++i) {
                float f = vf;
                const bool own = kFar && (state & kValuesApart);
                bad |= (state & kSomeNotFinite) != 0;
                if (i + 1 < count) look(i + 1);
                wait(cm.cready[i & 3], i >> 2);
                const float corr = cm.corr[i & 3][r];
                if (own) f = cm.vf[i & 3][r];
                wait(cm.odone[i % OB], i / OB);
                tc_after();
                const uint32_t at = mine + (i % OB) * D;
#pragma unroll
                for (int k = 0; k < M::OC; k += 32) {
                    uint32_t d[32];
                    tc_load32(d, at + k);
                    tc_loaded();
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        O[k + j] = fmaf(__uint_as_float(d[j]), f, O[k + j] * corr);
                }
                tc_before();
                __syncwarp();
                if (lane == 0) kq::mbar_arrive(bar(cm.ofree[i % OB]));
            }
        };
        if constexpr (kTwo) {
            if (apart) sums(std::true_type());
            else sums(std::false_type());
        }
        write_rows(O, bad, w - 4);
    } else {
        if constexpr (kTwo && D == 256) asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        // ------------------------------------------------- copies
        auto copy = [&](int k) {
            const int s = M::slot(k), t = t1 - 1 - (k >> 1);
            const uint32_t to = base + M::kRing + s * M::kPart;
            uint32_t done = bar(cm.full[s]);
            // Values that are cleaned have barriers of their own: who waits
            // for some tiles only could be two phases ahead of a slot's.
            if (!kTwo && (k & 1) && (k >> 1) < edges) {
                kq::mbar_arrive(done);
                done = bar(cm.vraw[(k >> 1) & 3]);
            }
            kq::mbar_expect_tx(done, M::kPart);
            if constexpr (kTwo) {
                kq::bulk_g2s(to, a.tiles + (slot0 + (int64_t)t * a.kv_heads) * (2 * M::kPart) +
                                     (k & 1) * M::kPart, M::kPart, done);
            } else {
#pragma unroll
                for (int c = 0; c < D / 64; ++c)
                    tensor2d_g2s(to + c * TK * 128, k & 1 ? &a.vmap : &a.kmap, it.head * D + 64 * c,
                                 it.kfirst + t * TK, done);
            }
        };
        // by the producer: all copies, or the values'
        constexpr int kStep = kTwo ? 1 : 2;
        auto copy_until = [&](int until) {
            for (; copied < until; ++copied) {
                const int k = kStep * copied + (kStep - 1);
                if (M::turn(k) > 0) wait(cm.empty[M::slot(k)], M::turn(k) - 1);
                if (dead()) break;
                copy(k);
            }
        };
        const bool producer = w == M::kFirst + 1 && lane == 0;
        if (M::kQStaged && producer) {  // hb heads of tok tokens
            kq::mbar_expect_tx(bar(cm.qfull), (uint32_t)a.tok * a.hb * (D * 4));
            for (int c = 0; c < D / 32; ++c)
                tensor3d_g2s(base + M::kQStage + c * (kRows * 128), &a.qmap, 32 * c, it.hq, it.first + it.tok0,
                             bar(cm.qfull));
        }
        // (while the queries are fetched)
        if (producer) copy_until(kTwo ? min(2 * count, M::kFree) : min(count, M::kEach));
        if (!kTwo && w == M::kFirst) {
            for (; copied < min(count, M::kEach); ++copied)
                if (lane == 0) copy(2 * copied);
        }
        __syncthreads();
        // terms' products, the small ones first
        constexpr int kTerms = kTwo ? 3 : 1;
        auto lo_first = [](int term) { return kTwo && term == 0; };
        auto lo_second = [](int term) { return kTwo && term == 1; };
        if (producer) {
            copy_until(kTwo ? 2 * count : count);
        } else if (w == M::kFirst) {
            // --------------------------------------------- S of each tile
            // (One warp for both, O first: f32 370 against 328 us, as it issues
            // a product in about the time that the tensor core takes for one.)
            tc_after();
            const uint32_t tm = uniform(tmem);
            const uint64_t qd = desc_k(uniform(base + M::kControl));  // (the queries' lo terms)
            constexpr uint32_t is = mma_idesc(TK, M::kBf16, false);
            for (int i = 0; i < count; ++i) {
                const int k = 2 * i;
                wait(cm.full[M::slot(k)], M::turn(k));
                if (i >= SB) wait(cm.sfree[i % SB], i / SB - 1);
                if (__any_sync(~0u, dead())) break;
                tc_after();
                const uint32_t s = uniform(M::slot(k)), b = uniform(i % SB);
                const uint32_t d = tm + M::kS + TK * b;
                const uint64_t kd = desc_k(uniform(base + M::kRing) + s * M::kPart);
                if (elected()) {
#pragma unroll
                    for (int term = 0; term < kTerms; ++term)
#pragma unroll
                        for (int j = 0; j < D / 16; ++j) {
                            const uint64_t kj = kd + (((lo_second(term) ? M::kTerm : 0) +
                                                       (j >> 2) * (TK * 128) + (j & 3) * 32) >> 4);
                            const uint64_t qj = qd + (((j >> 2) * (kRows * 128) + (j & 3) * 32) >> 4);
                            const uint32_t qt = tm + (lo_first(term) ? D / 2 : 0) + 8 * j;
                            if (M::kLoShared && lo_first(term)) {
                                if (term + j) tc_add_ss(d, qj, kj, is);
                                else tc_mma_ss(d, qj, kj, is, false);
                            } else {
                                if (term + j) tc_add_ts(d, qt, kj, is);
                                else tc_mma_ts(d, qt, kj, is, false);
                            }
                        }
                    tc_commit(bar(cm.sdone[0]) + 8 * b);
                    if (kTwo) tc_commit(bar(cm.empty[0]) + 8 * s);
                }
                // 16 bits: the S before has been read, so its keys' slot is free
                if (!kTwo && i > 0 && copied < count) {
                    if (lane == 0) copy(2 * copied);
                    ++copied;
                }
                __syncwarp();
            }
        } else if (w == M::kFirst + 2) {
            // --------------------------------------------- O of each tile
            tc_after();
            const uint32_t tm = uniform(tmem);
            constexpr uint32_t io = mma_idesc(D, M::kBf16, true);
            for (int i = 0; i < count; ++i) {
                const int k = 2 * i + 1;
                wait(cm.full[M::slot(k)], M::turn(k));
                if (!kTwo && i < edges) wait(cm.vclean[i & 3], i >> 2);
                if (kTwo && i >= OB) wait(cm.ofree[i % OB], i / OB - 1);
                wait(cm.pready[i % PB], i / PB);
                if (__any_sync(~0u, dead())) break;
                tc_after();
                const uint32_t s = uniform(M::slot(k)), b = uniform(i % PB);
                const uint32_t o = kTwo ? uniform(i % OB) : 0, more = uniform(!kTwo && i > 0);
                const uint64_t vd = desc_n(uniform(base + M::kRing) + s * M::kPart, TK * 128);
                const uint32_t d = tm + M::kO + D * o, p = tm + M::kP + M::kPCols * b;
                if (elected()) {
#pragma unroll
                    for (int term = 0; term < kTerms; ++term)
#pragma unroll
                        for (int j = 0; j < TK / 16; ++j) {
                            const uint32_t pj = p + (lo_first(term) ? TK / 2 : 0) + 8 * j;
                            const uint64_t vj = vd + (((lo_second(term) ? M::kTerm : 0) + j * 2048) >> 4);
                            if (term + j) tc_add_ts(d, pj, vj, io);
                            else tc_mma_ts(d, pj, vj, io, more);
                        }
                    if (kTwo || i == count - 1) tc_commit(bar(cm.odone[0]) + 8 * o);
                    tc_commit(bar(cm.pfree[0]) + 8 * b);
                    tc_commit(bar(cm.empty[0]) + 8 * s);
                }
                __syncwarp();
            }
        } else if (!kTwo && w == M::kFirst + 3) {
            // ------------- values that are not finite, of tiles seen in part
            for (int i = 0; i < edges; ++i) {
                const int k = 2 * i + 1, s = M::slot(k);
                wait(cm.vraw[i & 3], i >> 2);
                uint4 *v = reinterpret_cast<uint4 *>(smem + M::kRing + s * M::kPart);
                bool found = false;
                if (!dead())
                    for (int c = lane; c < M::kPart / 16; c += 32) {
                        uint4 x = v[c];
                        if (not_finite<H>(x.x) | not_finite<H>(x.y) | not_finite<H>(x.z) | not_finite<H>(x.w)) {
                            found = true;
                            uint32_t *e = &x.x;
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const uint32_t n = not_finite<H>(e[j]);
                                if (n & 0x8000u) e[j] &= 0xFFFF0000u;
                                if (n & 0x80000000u) e[j] &= 0x0000FFFFu;
                            }
                            v[c] = x;
                        }
                    }
                if (found) *(volatile int *)&cm.bad = 1;
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) kq::mbar_arrive(bar(cm.vclean[i & 3]));
            }
            __syncwarp();
            if (lane == 0) kq::mbar_arrive(bar(cm.ldone));
        }
        __syncwarp();
    }
    tc_before();
    __syncthreads();
    // After an expired wait no copy and no product may run on past this.
    if (dead()) {
        if ((w == M::kFirst + 1 || (!kTwo && w == M::kFirst)) && lane == 0) {
            const bool values = !kTwo && w == M::kFirst + 1;
            for (int n = max(0, copied - (kTwo ? M::kSlots : M::kEach)); n < copied; ++n) {
                const int k = kTwo ? n : 2 * n + values;
                kq::mbar_wait(bar(cm.full[M::slot(k)]), M::turn(k) & 1, kq::kWaitLimitNs);
                if (values && n < edges) kq::mbar_wait(bar(cm.vraw[n & 3]), (n >> 2) & 1, kq::kWaitLimitNs);
            }
            if (M::kQStaged) kq::mbar_wait(bar(cm.qfull), 0, kq::kWaitLimitNs);
        }
        if (w == M::kFirst || w == M::kFirst + 2) {
            const uint64_t &drain = cm.drain[w == M::kFirst ? 0 : 1];
            tc_after();
            if (elected()) tc_commit(bar(drain));
            __syncwarp();
            kq::mbar_wait(bar(drain), 0, kq::kWaitLimitNs);
            __syncwarp();
        }
        __syncthreads();
    }
    if (w == M::kFirst) {
        tc_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    }
}

// ------------------------------------------------------------------ host
// Slots of an f32 call's tiles.
inline int64_t f32_slots(const PromptArgs &a, int d) { return a.nkeys / f32_tile_tokens(d) + a.nseq; }

// Workspace: tiles, their powers of two, their tokens', partial results; in all.
struct Space {
    int64_t info, powers, part, bytes;
};
inline Space space_of(const PromptArgs &a, int blocks, bool f32, int d) {
    Space s{};
    const int64_t tiles = f32 ? f32_slots(a, d) * a.kv_heads : 0;
    s.info = tiles * (f32_tile_tokens(d) * d * 8);
    s.powers = s.info + tiles * (int64_t)sizeof(TileInfo);
    s.part = (s.powers + tiles * (int64_t)sizeof(TilePowers) + 255) / 256 * 256;
    s.bytes = s.part + (a.splits > 1 ? 4ll * a.items * a.splits * blocks * kRows * (d + 2) : 0);
    s.bytes = (s.bytes + 255) / 256 * 256;
    return s;
}

template <auto KERNEL>
cudaError_t allow_shared(int bytes) {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && (done.load() >> dev & 1))) return e;
    e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < 64) done.fetch_or(1ull << dev);
    return e;
}

// A launch that may begin before the one before it ends (it waits itself).
template <class F, class... A>
cudaError_t launch_early(F *kernel, dim3 grid, int threads, int smem, cudaStream_t s, const A &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Keys or values as a tensor map of tokens by all heads' values.
template <class T>
cudaError_t keys_map(const void *p, int64_t stride, const PromptArgs &a, int d, int tokens, CUtensorMap *m) {
    const uint64_t dims[2] = {(uint64_t)a.kv_heads * d, (uint64_t)a.nkeys}, strides[1] = {2ull * stride};
    const uint32_t box[2] = {64, (uint32_t)tokens};
    return kqhost::values_map(p, type_of<T>(), 2, dims, strides, box, m);
}

// Queries as (value, head, token): boxes of hb heads of `tokens` tokens.
template <class T>
cudaError_t queries_map(const PromptArgs &a, int d, int tokens, CUtensorMap *m) {
    constexpr uint64_t kSize = sizeof(T);
    const uint64_t dims[3] = {(uint64_t)d, (uint64_t)a.q_heads, (uint64_t)a.ntok};
    const uint64_t strides[2] = {kSize * d, kSize * a.q_stride};
    const uint32_t box[3] = {128 / sizeof(T), (uint32_t)a.hb, (uint32_t)tokens};
    return kqhost::values_map(a.q, type_of<T>(), 3, dims, strides, box, m);
}

template <class T, int D>
cudaError_t launch_rows(PromptArgs &a, cudaStream_t s) {
    using M = Rows<T, D>;
    cudaError_t e = allow_shared<kq_prompt_rows<T, D>>(M::kBytes);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)(a.items * a.splits));
    if constexpr (M::kTwo) {
        if (M::kQStaged) {
            e = queries_map<T>(a, D, a.tok, &a.qmap);
            if (e != cudaSuccess) return e;
        }
        const dim3 tiles((unsigned)f32_slots(a, D), a.kv_heads, 2);
        kq_prompt_split<D><<<tiles, kSplitThreads, 0, s>>>(a);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        return launch_early(kq_prompt_rows<T, D>, grid, M::kThreads, M::kBytes, s, a);
    } else {
        if (a.nkeys > 0) {
            e = keys_map<T>(a.k, a.k_stride, a, D, M::TK, &a.kmap);
            if (e == cudaSuccess) e = keys_map<T>(a.v, a.v_stride, a, D, M::TK, &a.vmap);
            if (e != cudaSuccess) return e;
        }
        kq_prompt_rows<T, D><<<grid, M::kThreads, M::kBytes, s>>>(a);
        return cudaGetLastError();
    }
}

}  // namespace kqp
