// kq_attn.cuh -- attention of new tokens over the paged cache
// (kq_tree_attention): the kernel, compiled per cache format in
// kq_attn_<format>.cu.
//
// Work.  An item is a key head of a sequence with a block of its rows (a row
// is a new token and one of the query heads that share the key head); its
// units are the sequence's pages.  All units in order are cut into as many
// equal runs as there are CTAs, so ragged lengths balance; an item that
// falls into several runs leaves a partial result (row maxima, sums,
// weighted values) in each, joined by kq_attn_join.
//
// A page.  A CTA has groups of four warps; a group takes whole pages, two
// bulk copies each (keys, values) into a ring of its own, and works on one
// page at a time:
//   1. each warp forms the logits of 16 of the page's 64 tokens,
//   2. the warps exchange row maxima, form the probabilities and leave them
//      in shared memory,
//   3. each warp adds its quarter of the values' width, over all 64 tokens.
//
// Arithmetic.  The tensor cores take f16 operands, and codes are exact in
// f16.  Queries and probabilities are f32, held as two f16 terms hi + lo (22
// bits): an 8-row tile of them fills the 16 rows of an m16n8k16 operand, hi
// above lo, so that one MMA forms both products and the two halves of its
// result are added in f32.  A query row is scaled by a power of two first
// (its largest magnitude below 2^15), probabilities times the values' scale
// likewise by page and group.  Scales of quantised keys multiply the f32 sums
// of their group.  Each page's sums start at zero and are added to the
// running ones in f32, with the running maximum's correction.
//
// The k index inside an MMA is any order that both operands share.  A lane
// takes eight consecutive values of a key (an octet) or 16 tokens of a value
// from one or two wide loads, and queries and probabilities are laid out to
// match; the cache layout (kq_decode.h) makes those loads free of bank
// conflicts.
//
// Bound by: memory (the cache is read once) for few rows; the issue of the
// conversions and MMAs for many.
#pragma once

#include <mutex>

#include "kq_async.cuh"
#include "kq_decode.cuh"
#include "kq_decode_launch.h"

namespace kqd {

constexpr int kMaxGroups = 4;
constexpr int kMaxSlots = 8;  // of a group's ring; a slot holds a page's keys or values

struct AttnArgs {
    Seqs q;
    const float *x;
    int64_t x_stride;
    const uint64_t *mask;
    float *out;
    float *part;    // partial results, two slots a CTA
    int4 *meta;     // two entries a CTA: the item that begins in it and goes on
    unsigned int *err;
    unsigned long long wait_ns;
    int32_t q_heads, per;  // query heads; of them to a key head
    float scale;           // times log2 e
    int32_t ng, nslot;     // groups a CTA, slots of a group's ring
};

// Rows of a CTA's block, floats of a partial result.
__host__ __device__ constexpr int part_floats(int rb, int d) { return rb * (d + 2); }

// ------------------------------------------------------------ shared memory
// common | queries | per group: ring, probabilities, maxima
struct AttnCommon {
    uint64_t rowmask[32];
    uint64_t bars[kMaxGroups * kMaxSlots];
    long long scan[16];
    long long start_unit;
    int start_seq;
    int dead;                              // a wait has expired
    int badpage[kMaxGroups * kMaxSlots];   // the slot's page is not valid
    float rowfactor[32];
    float ml[kMaxGroups][5][32];           // group's row maxima, warps' row sums
};
template <int FMT, int D, int MT>
struct AttnSmem {
    static constexpr int kRows = 8 * MT;
    static constexpr int kWg = 4;             // warps of a group
    static constexpr int kGroups = 16 / kWg;  // groups of an SM
    static constexpr int kHalf = Kv<FMT, D>::kV;  // bytes of a slot
    static constexpr int kCommon = (sizeof(AttnCommon) + 127) / 128 * 128;
    static constexpr int kQ = kRows * D * 4;
    static constexpr int kP = kRows * kPage * 4;
    static constexpr int kMax = kWg * kRows * 4;
    static __host__ __device__ int group(int nslot) { return nslot * kHalf + kP + kMax; }
    static __host__ __device__ int total(int ng, int nslot) {
        return kCommon + kQ + ng * group(nslot);
    }
};

// -------------------------------------------------------------- operations
__device__ __forceinline__ void mma(float (&d)[4], const uint4 &a, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float exp2_of(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t bits_of(__half2 h) {
    uint32_t w;
    memcpy(&w, &h, 4);
    return w;
}
__device__ __forceinline__ __half2 half2_of(uint32_t w) {
    __half2 h;
    memcpy(&h, &w, 4);
    return h;
}

// hi and lo terms of a pair.
__device__ __forceinline__ void split(float a, float b, uint32_t &hi, uint32_t &lo) {
    const __half2 h = __floats2half2_rn(a, b);
    const float2 f = __half22float2(h);
    hi = bits_of(h);
    lo = bits_of(__floats2half2_rn(a - f.x, b - f.y));
}

// f16 pairs of codes.  The f16 with bits 0x6400 | n is 1024 + n for n < 1024,
// so a code shifted to be positive is put in place and the offset taken off,
// both exactly.
__device__ __forceinline__ void codes8(uint32_t w, uint32_t &b0, uint32_t &b1) {
    w ^= 0x80808080u;
    const __half2 off = half2_of(0x64806480u);  // 1024 + 128
    b0 = bits_of(__hsub2(half2_of(__byte_perm(w, 0x64646464u, 0x4140)), off));
    b1 = bits_of(__hsub2(half2_of(__byte_perm(w, 0x64646464u, 0x4342)), off));
}
// Eight 4-bit codes: pairs (0, 4), (1, 5), (2, 6), (3, 7).
__device__ __forceinline__ uint32_t nibble(uint32_t w, uint32_t mask, uint32_t with) {
    uint32_t r;  // (w & mask) ^ with
    asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(r) : "r"(w), "r"(mask), "r"(with));
    return r;
}
__device__ __forceinline__ void codes4(uint32_t w, uint32_t (&b)[4]) {
    const __half2 off = half2_of(0x64086408u);    // 1024 + 8
    const __half2 div = half2_of(0x2C002C00u);    // 1 / 16
    const __half2 off16 = half2_of(0xD480D480u);  // -(64 + 8)
    const uint32_t v = w >> 8;
    b[0] = bits_of(__hsub2(half2_of(nibble(w, 0x000F000Fu, 0x64086408u)), off));
    b[1] = bits_of(__hfma2(half2_of(nibble(w, 0x00F000F0u, 0x64806480u)), div, off16));
    b[2] = bits_of(__hsub2(half2_of(nibble(v, 0x000F000Fu, 0x64086408u)), off));
    b[3] = bits_of(__hfma2(half2_of(nibble(v, 0x00F000F0u, 0x64806480u)), div, off16));
}
// Element pairs of the two k-steps of eight: pair h of step s.
template <int FMT>
__device__ __forceinline__ constexpr int pair_first(int s, int h) {
    return FMT == KQ_KV_Q4 ? 2 * s + h : 4 * s + 2 * h;
}
template <int FMT>
__device__ __forceinline__ constexpr int pair_second(int s, int h) {
    return FMT == KQ_KV_Q4 ? 2 * s + h + 4 : 4 * s + 2 * h + 1;
}

template <int THREADS>
__device__ __forceinline__ void group_sync(int g) {
    asm volatile("bar.sync %0, %1;" ::"r"(g + 1), "n"(THREADS) : "memory");
}

// Probabilities in shared memory, [row][16 chunks of 4 tokens]: lane c's
// tokens of a value (Kv order) are chunks 4 i + c, i = 0..3; odd rows are
// turned by half a line.
template <int FMT>
__device__ __forceinline__ int p_at(int row, int tok) {
    int c, i;
    if (FMT == KQ_KV_F16) {
        c = (tok >> 3) & 3, i = 2 * (tok >> 5) + ((tok >> 2) & 1);
    } else {
        c = tok >> 4, i = (tok >> 2) & 3;
    }
    return row * kPage + (((4 * i + c) ^ ((row & 1) << 2)) << 2) + (tok & 3);
}

// ------------------------------------------------------------------- units
// Pages of a sequence that are looked at: up to the last new token, but no
// more than one page past the table (a committed place without a page makes
// every row NaN already).
__device__ __forceinline__ int64_t pages_of(const Seqs &q, const Seq &s) {
    const int64_t n = ((int64_t)s.ctx + s.n + kPage - 1) / kPage;
    return s.ctx / kPage > q.max_pages ? q.max_pages + 1 : n;
}
template <int RB>
__device__ __forceinline__ int64_t units_of(const AttnArgs &a, const Seq &s, int &blocks) {
    blocks = (s.n * a.per + RB - 1) / RB;
    return s.n ? pages_of(a.q, s) * blocks * a.q.heads : 0;
}
// CTA that works on unit u, of `total` cut into n runs.
__device__ __forceinline__ int cta_of(long long u, long long total, int n) {
    const long long base = total / n, rem = total % n;
    return (int)(u < rem * (base + 1) ? u / (base + 1) : rem + (u - rem * (base + 1)) / base);
}

// ------------------------------------------------------------------ kernel
template <int FMT, int D, int MT>
__global__ void __launch_bounds__(AttnSmem<FMT, D, MT>::kGroups * AttnSmem<FMT, D, MT>::kWg * 32, 1)
    kq_attn_kernel(const __grid_constant__ AttnArgs a) {
    using L = Kv<FMT, D>;
    using M = AttnSmem<FMT, D, MT>;
    constexpr int RB = M::kRows;
    constexpr int kSteps = D / 16;          // k-steps of a logit
    constexpr int kWg = M::kWg, kGroupThreads = 32 * kWg;
    constexpr int kTok = kPage / kWg, J = kTok / 8;  // tokens of a warp in part 1, in tiles
    constexpr int kSlice = D / kWg;         // values of a warp in part 3
    constexpr int kTiles = kSlice / 8;      // its n-tiles
    constexpr int kSliceGroups = kSlice > kGroup ? kSlice / kGroup : 1;
    constexpr int kTilesG = kTiles / kSliceGroups;

    extern __shared__ __align__(128) uint8_t smem[];
    AttnCommon &cm = *reinterpret_cast<AttnCommon *>(smem);
    uint4 *qs = reinterpret_cast<uint4 *>(smem + M::kCommon);  // [tile][k-step][lane]
    const int tid = threadIdx.x, lane = tid & 31;
    const int g = tid / kGroupThreads, w = (tid >> 5) % kWg;
    const int n8 = lane >> 2, c = lane & 3;  // row (or column) of an operand, and its quarter
    const int nthreads = a.ng * kGroupThreads;
    uint8_t *gbase = smem + M::kCommon + M::kQ + g * M::group(a.nslot);
    float *ps = reinterpret_cast<float *>(gbase + a.nslot * M::kHalf);
    float *smax = ps + RB * kPage;  // [warp][row]
    const uint32_t ring = kq::smem_addr(gbase);
    const uint32_t bars = kq::smem_addr(&cm.bars[g * kMaxSlots]);

    if (tid < a.ng * kMaxSlots && (tid % kMaxSlots) < a.nslot) {
        kq::mbar_init(kq::smem_addr(&cm.bars[tid]), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (tid == 0) cm.dead = 0;
    kq::allow_dependents();  // kq_attn_join waits for this kernel's end

    // ---- this CTA's run of units
    long long u0, u1, total;
    {
        const int each = (a.q.nseq + nthreads - 1) / nthreads;
        const int b0 = min(tid * each, a.q.nseq), b1 = min(b0 + each, a.q.nseq);
        long long mine = 0;
        int blocks;
        for (int b = b0; b < b1; ++b) mine += units_of<RB>(a, seq_of(a.q, b), blocks);
        long long upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const long long v = __shfl_up_sync(~0u, upto, o);
            if (lane >= o) upto += v;
        }
        if (lane == 31) cm.scan[tid >> 5] = upto;
        __syncthreads();
        total = 0;
        for (int i = 0; i < nthreads / 32; ++i) {
            if (i == (tid >> 5)) upto += total;
            total += cm.scan[i];
        }
        const long long base = total / gridDim.x, rem = total % gridDim.x, k = blockIdx.x;
        u0 = k * base + min(k, rem);
        u1 = u0 + base + (k < rem ? 1 : 0);
        if (u0 < u1 && u0 >= upto - mine && u0 < upto) {
            long long at = upto - mine;
            int b = b0;
            for (;; ++b) {
                const long long n = units_of<RB>(a, seq_of(a.q, b), blocks);
                if (u0 < at + n) break;
                at += n;
            }
            cm.start_seq = b;
            cm.start_unit = u0 - at;
        }
        if (tid == 0) a.meta[2 * blockIdx.x] = make_int4(-1, 0, 0, 0);
        __syncthreads();
    }
    if (u0 >= u1) return;

    // the group's ring: next slot to fill and to use, and the use's parity
    int fill = 0, use = 0;
    uint32_t parity = 0, op0 = 0;  // op0: copies before this segment
    int b = cm.start_seq;
    long long off = cm.start_unit;
    for (long long u = u0; u < u1 && b < a.q.nseq;) {
        // ---- the segment: pages [pg0, pg0 + npg) of one item
        int blocks;
        Seq s = seq_of(a.q, b);
        const long long units = units_of<RB>(a, s, blocks);
        if (off >= units) {
            ++b, off = 0;
            continue;
        }
        const int pages = (int)pages_of(a.q, s);
        const int item = (int)(off / pages);
        const int pg0 = (int)(off - (long long)item * pages);
        const int npg = (int)min((long long)(pages - pg0), u1 - u);
        const int head = item / blocks, row0 = (item - head * blocks) * RB;
        const int nrows = min(RB, s.n * a.per - row0);
        const int count = npg > g ? (npg - g + a.ng - 1) / a.ng : 0;  // the group's pages

        // ---- copies: warp 0 of the group looks up 32 pages at a time and
        // one lane issues
        int64_t found = -1;
        int live = 0;  // copies issued (lane 0 of warp 0)
        auto copy = [&](int i) {  // copy i of the segment: keys, then values, page by page
            const int k = i >> 1;
            if ((i & 1) == 0 && (k & 31) == 0)
                found = k + lane < count ? page_of(a.q, b, pg0 + g + (int64_t)(k + lane) * a.ng) : -1;
            const int64_t page = __shfl_sync(~0u, found, k & 31);
            // (once a wait has expired nothing more is issued or waited for)
            if (lane == 0 && !*(volatile int *)&cm.dead) {
                live = i + 1;
                const uint32_t bar = bars + 8 * fill;
                cm.badpage[g * kMaxSlots + fill] = page < 0;
                kq::mbar_expect_tx(bar, M::kHalf);
                kq::bulk_g2s(ring + fill * M::kHalf,
                             a.q.data + (max(page, (int64_t)0) * a.q.heads + head) * L::kBlock +
                                 (i & 1) * M::kHalf,
                             M::kHalf, bar);
            }
            if (++fill == a.nslot) fill = 0;
            __syncwarp();
        };
        int issued = 0;
        if (w == 0)
            for (; issued < min(2 * count, a.nslot); ++issued) copy(issued);

        // ---- queries: rows scaled by a power of two, hi and lo terms, laid
        // out as the operands of part 1
        for (int r = tid >> 5; r < RB; r += nthreads / 32) {
            const bool on = r < nrows;
            const int tok = on ? (row0 + r) / a.per : 0, hq = on ? (row0 + r) % a.per : 0;
            const float *row = a.x + (s.first + tok) * a.x_stride + (head * a.per + hq) * D;
            constexpr int kLoads = D > 128 ? D / 128 : 1;
            float4 v[kLoads];
            float top = 0.f;
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int e = 4 * lane + 128 * i;
                v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (on && e < D) v[i] = *reinterpret_cast<const float4 *>(row + e);
                top = fmaxf(top, fmaxf(fmaxf(fabsf(v[i].x), fabsf(v[i].y)),
                                       fmaxf(fabsf(v[i].z), fabsf(v[i].w))));
            }
#pragma unroll
            for (int o = 16; o; o /= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
            // top < 2^ex; the row times 2^(15 - ex)
            const int ex = max((int)((__float_as_uint(top) >> 23) & 255) - 126, -111);
            const float up = __uint_as_float((uint32_t)(127 + 15 - ex) << 23);
            if (lane == 0) {
                // (2^(ex - 15) in two steps: it may be below the normal range)
                cm.rowfactor[r] = a.scale * __uint_as_float((uint32_t)(127 + (ex >> 1)) << 23) *
                                  __uint_as_float((uint32_t)(127 + (ex - (ex >> 1)) - 15) << 23);
                cm.rowmask[r] = !on ? 0
                                : a.mask ? __ldg(a.mask + s.first + tok)
                                         : ~0ull >> (63 - tok);
            }
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                float x[4] = {v[i].x * up, v[i].y * up, v[i].z * up, v[i].w * up};
                const int e = 4 * lane + 128 * i;
                if (FMT == KQ_KV_Q4) {
                    // pairs are (j, j + 4) of an octet: the even lane of two
                    // takes j = 0, 1 (step 0), the odd one j = 2, 3 (step 1)
                    const bool odd = lane & 1;
                    const float s0 = odd ? x[0] : x[2], s1 = odd ? x[1] : x[3];
                    const float r0 = __shfl_xor_sync(~0u, s0, 1), r1 = __shfl_xor_sync(~0u, s1, 1);
                    const float m0 = odd ? x[2] : x[0], m1 = odd ? x[3] : x[1];
                    x[0] = odd ? r0 : m0, x[1] = odd ? m0 : r0;
                    x[2] = odd ? r1 : m1, x[3] = odd ? m1 : r1;
                }
                if (e < D) {
                    uint4 o;
                    split(x[0], x[1], o.x, o.y);
                    split(x[2], x[3], o.z, o.w);
                    const int octet = e >> 3;
                    const int step = 2 * (octet >> 2) + ((e >> 2) & 1);
                    qs[((r >> 3) * kSteps + step) * 32 + 4 * (r & 7) + (octet & 3)] = o;
                }
            }
        }
        __syncthreads();

        float m[MT], l[MT], O[MT][kTiles][2];
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            m[t] = -INFINITY, l[t] = 0.f;
#pragma unroll
            for (int i = 0; i < kTiles; ++i) O[t][i][0] = O[t][i][1] = 0.f;
        }

        // the next slot, once its copy has arrived
        auto arrived = [&]() {
            if (!*(volatile int *)&cm.dead && !kq::mbar_wait(bars + 8 * use, parity, a.wait_ns)) {
                *(volatile int *)&cm.dead = 1;
                atomicOr(a.err, 1u);
            }
            const int slot = use;
            if (++use == a.nslot) use = 0, parity ^= 1;
            return slot;
        };
        for (int k = 0; k < count; ++k) {
            const int pg = pg0 + g + k * a.ng;
            const int left = s.ctx - pg * kPage;      // committed tokens of the page and after
            const bool edge = left < kPage;           // new tokens, or the end
            // bit t: token t may be attended by row r (edge pages)
            auto allowed = [&](int r) -> uint64_t {
                const uint64_t nw = cm.rowmask[r] & (~0ull >> (64 - s.n));
                if (left <= 0) return -left < 64 ? nw >> -left : 0;
                return (nw << left) | ~(~0ull << left);
            };
            // ---- 1. logits of tokens 16 w .. 16 w + 15
            const int ks = arrived();
            const uint8_t *kb = gbase + ks * M::kHalf;
            const bool badpage = cm.badpage[g * kMaxSlots + ks];
            float S[MT][J][2];
            {
                float acc[MT][J][4];
                constexpr int kLane = L::kSlabBytes / 4;  // bytes of a lane in a slab
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int j = 0; j < J; ++j) {
                        S[t][j][0] = S[t][j][1] = 0.f;
                        if (!L::kQuant) acc[t][j][0] = acc[t][j][1] = acc[t][j][2] = acc[t][j][3] = 0.f;
                    }
#pragma unroll
                for (int sl = 0; sl < L::kSlabs; ++sl) {
                    uint32_t raw[J][kLane / 4];
                    uint32_t skw[J][2][(L::kSlabGroups + 1) / 2];  // scales, two groups a word
#pragma unroll
                    for (int j = 0; j < J; ++j) {
                        const uint8_t *p = kb + sl * kPage * L::kSlabBytes +
                                           (kTok * w + 8 * j + n8) * L::kSlabBytes + c * kLane;
                        if constexpr (kLane == 16) {
                            const uint4 v = *reinterpret_cast<const uint4 *>(p);
                            raw[j][0] = v.x, raw[j][1] = v.y, raw[j][2] = v.z, raw[j][3] = v.w;
                        } else {
                            const uint2 v = *reinterpret_cast<const uint2 *>(p);
                            raw[j][0] = v.x, raw[j][1] = v.y;
                        }
                        if constexpr (L::kQuant) {
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const uint8_t *sp = kb + L::k_scale(kTok * w + 8 * j + 2 * c + i,
                                                                    sl * L::kSlabGroups);
                                if constexpr (L::kSlabGroups == 4) {
                                    const uint2 v = *reinterpret_cast<const uint2 *>(sp);
                                    skw[j][i][0] = v.x, skw[j][i][1] = v.y;
                                } else {
                                    skw[j][i][0] = *reinterpret_cast<const uint32_t *>(sp);
                                }
                            }
                        }
                    }
#pragma unroll
                    for (int gl = 0; gl < L::kSlabGroups; ++gl) {
                        const int gg = sl * L::kSlabGroups + gl;
                        uint32_t bb[J][4];
                        float sk[J][2];
#pragma unroll
                        for (int j = 0; j < J; ++j) {
                            if constexpr (FMT == KQ_KV_F16) {
#pragma unroll
                                for (int i = 0; i < 4; ++i) bb[j][i] = raw[j][i];
                            } else if constexpr (FMT == KQ_KV_Q8) {
                                codes8(raw[j][2 * gl], bb[j][0], bb[j][1]);
                                codes8(raw[j][2 * gl + 1], bb[j][2], bb[j][3]);
                            } else {
                                codes4(raw[j][gl], bb[j]);
                            }
                            if constexpr (L::kQuant) {
#pragma unroll
                                for (int i = 0; i < 2; ++i) {
                                    const __half2 h = half2_of(skw[j][i][gl / 2]);
                                    sk[j][i] = gl & 1 ? __high2float(h) : __low2float(h);
                                }
                            }
                        }
#pragma unroll
                        for (int t = 0; t < MT; ++t) {
                            const uint4 q0 = qs[(t * kSteps + 2 * gg) * 32 + lane];
                            const uint4 q1 = qs[(t * kSteps + 2 * gg + 1) * 32 + lane];
#pragma unroll
                            for (int j = 0; j < J; ++j) {
                                if constexpr (L::kQuant) {
                                    float d[4] = {0.f, 0.f, 0.f, 0.f};
                                    mma(d, q0, bb[j][0], bb[j][1]);
                                    mma(d, q1, bb[j][2], bb[j][3]);
                                    S[t][j][0] = fmaf(sk[j][0], d[0] + d[2], S[t][j][0]);
                                    S[t][j][1] = fmaf(sk[j][1], d[1] + d[3], S[t][j][1]);
                                } else {
                                    mma(acc[t][j], q0, bb[j][0], bb[j][1]);
                                    mma(acc[t][j], q1, bb[j][2], bb[j][3]);
                                }
                            }
                        }
                    }
                }
                if constexpr (!L::kQuant) {
#pragma unroll
                    for (int t = 0; t < MT; ++t)
#pragma unroll
                        for (int j = 0; j < J; ++j) {
                            S[t][j][0] = acc[t][j][0] + acc[t][j][2];
                            S[t][j][1] = acc[t][j][1] + acc[t][j][3];
                        }
                }
            }
            // ---- 2. row maxima, probabilities
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                const float f = badpage ? quiet_nan() : cm.rowfactor[8 * t + n8];
#pragma unroll
                for (int j = 0; j < J; ++j)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        S[t][j][i] *= f;
                if (edge) {
                    const uint32_t ok = (uint32_t)(allowed(8 * t + n8) >> (kTok * w + 2 * c));
#pragma unroll
                    for (int j = 0; j < J; ++j)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            if (!((ok >> (8 * j + i)) & 1)) S[t][j][i] = -INFINITY;
                }
                float v = fmaxf(S[t][0][0], S[t][0][1]);
#pragma unroll
                for (int j = 1; j < J; ++j) v = fmaxf(v, fmaxf(S[t][j][0], S[t][j][1]));
                v = fmaxf(v, __shfl_xor_sync(~0u, v, 1));
                v = fmaxf(v, __shfl_xor_sync(~0u, v, 2));
                if (c == 0) smax[w * RB + 8 * t + n8] = v;
            }
            group_sync<kGroupThreads>(g);
            // every warp is done with these keys and the values before them
            if (w == 0)
                for (; issued < min(2 * count, 2 * k + 1 + a.nslot); ++issued) copy(issued);
            float alpha[MT];
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                const int r = 8 * t + n8;
                float now = m[t];
#pragma unroll
                for (int i = 0; i < kWg; ++i) now = fmaxf(now, smax[i * RB + r]);
                const float base = now == -INFINITY ? 0.f : now;
                alpha[t] = exp2_of(m[t] - base);
                m[t] = now;
                const float high = base - 15.f;  // probabilities (and l, O) times 2^15
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    const float p0 = exp2_of(S[t][j][0] - high), p1 = exp2_of(S[t][j][1] - high);
                    sum += p0 + p1;
                    *reinterpret_cast<float2 *>(ps + p_at<FMT>(r, kTok * w + 8 * j + 2 * c)) =
                        make_float2(p0, p1);
                }
                l[t] = fmaf(l[t], alpha[t], sum);
            }
            // ---- 3. values kSlice w .. of all 64 tokens
            const int vs = arrived();
            group_sync<kGroupThreads>(g);
            // (offsets of Kv count from the block's start; the slot starts at
            // the values)
            const uint8_t *vb = gbase + vs * M::kHalf - L::kV;
            auto token = [&](int i) {  // lane's token i of 16
                return FMT == KQ_KV_F16 ? 32 * (i >> 3) + 8 * c + (i & 7) : 16 * c + i;
            };
            // tokens that no row may attend (past the end), or whose values
            // are not finite: left out of the MMAs; the latter are added row
            // by row below
            uint64_t bad = 0;
            const uint64_t held = !edge ? ~0ull
                                  : left + s.n >= kPage ? ~0ull
                                  : left + s.n <= 0 ? 0ull : ~(~0ull << (left + s.n));
#pragma unroll
            for (int sg = 0; sg < kSliceGroups; ++sg) {
                const int group = w * kSlice / kGroup + sg;
                float fac = 1.f;
                __half2 sn[8];     // scales of the lane's tokens, normalised
                uint32_t keep[8];  // f16: pairs of tokens that stay
                if constexpr (L::kQuant) {
                    const uint4 *sp = reinterpret_cast<const uint4 *>(vb + L::v_scale(16 * c, group));
                    uint32_t raw[8];
                    const uint4 s0 = sp[0], s1 = sp[1];
                    raw[0] = s0.x, raw[1] = s0.y, raw[2] = s0.z, raw[3] = s0.w;
                    raw[4] = s1.x, raw[5] = s1.y, raw[6] = s1.z, raw[7] = s1.w;
                    if (edge) {
                        uint32_t b16 = 0;
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const uint32_t h = (raw[i / 2] >> (16 * (i & 1))) & 0xFFFFu;
                            const bool in = (held >> (16 * c + i)) & 1;
                            const bool nf = (h & 0x7C00u) == 0x7C00u;
                            if (in && nf) b16 |= 1u << i;
                            if (!in || nf) raw[i / 2] &= i & 1 ? 0x0000FFFFu : 0xFFFF0000u;
                        }
                        bad = (uint64_t)b16 << (16 * c);
                        bad |= __shfl_xor_sync(~0u, bad, 1);
                        bad |= __shfl_xor_sync(~0u, bad, 2);
                    }
                    // |scales| of the page and group are below 2^ex: times
                    // 2^-ex, they and a probability make less than 2^15
                    __half2 big = __habs2(half2_of(raw[0]));
#pragma unroll
                    for (int i = 1; i < 8; ++i) big = __hmax2(big, __habs2(half2_of(raw[i])));
                    big = __hmax2(big, half2_of(__shfl_xor_sync(~0u, bits_of(big), 1)));
                    big = __hmax2(big, half2_of(__shfl_xor_sync(~0u, bits_of(big), 2)));
                    const uint32_t top = bits_of(__hmax2(big, __lowhigh2highlow(big))) & 0xFFFFu;
                    const int ex = max((int)(top >> 10) - 14, -15);
                    const uint32_t up = ex <= 14 ? (uint32_t)(15 - ex) << 10 : 0x400u >> (ex - 14);
                    fac = __uint_as_float((uint32_t)(127 + ex) << 23);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        sn[i] = __hmul2(half2_of(raw[i]), half2_of(up | up << 16));
                } else if (edge) {
                    // (one pass over the slice's values, on edge pages only)
                    uint32_t b16 = 0;
#pragma unroll 1
                    for (int nt = 0; nt < kTiles; ++nt) {
                        const int e = w * kSlice + 8 * nt + n8;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const uint32_t v = *reinterpret_cast<const uint32_t *>(
                                vb + L::v_word(e, token(2 * i) / 2));
                            if ((v & 0x7C00u) == 0x7C00u) b16 |= 1u << (2 * i);
                            if ((v & 0x7C000000u) == 0x7C000000u) b16 |= 2u << (2 * i);
                        }
                    }
                    b16 |= __shfl_xor_sync(~0u, b16, 4);
                    b16 |= __shfl_xor_sync(~0u, b16, 8);
                    b16 |= __shfl_xor_sync(~0u, b16, 16);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const bool in = (held >> token(i)) & 1;
                        if (((b16 >> i) & 1) && in) bad |= 1ull << token(i);
                        if (!in) b16 |= 1u << i;
                    }
                    bad |= __shfl_xor_sync(~0u, bad, 1);
                    bad |= __shfl_xor_sync(~0u, bad, 2);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        keep[i] = (b16 >> (2 * i) & 1 ? 0u : 0xFFFFu) |
                                  (b16 >> (2 * i) & 2 ? 0u : 0xFFFF0000u);
                }
                uint4 pa[MT][4];  // operands of the four k-steps
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    const int r = 8 * t + n8;
                    float p[16];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 v = *reinterpret_cast<const float4 *>(
                            ps + r * kPage + (((4 * i + c) ^ ((r & 1) << 2)) << 2));
                        p[4 * i] = v.x, p[4 * i + 1] = v.y, p[4 * i + 2] = v.z, p[4 * i + 3] = v.w;
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int o = 8 * (i >> 1), st = i & 1;
                        auto pair = [&](int h, uint32_t &hi, uint32_t &lo) {
                            const int x = o + pair_first<FMT>(st, h), y = o + pair_second<FMT>(st, h);
                            split(p[x], p[y], hi, lo);
                            if constexpr (L::kQuant) {
                                // (hi + lo) s as two terms: hi s is rounded,
                                // what that loses (exact in f16) joins lo s
                                const __half2 sc =
                                    __halves2half2(x & 1 ? __high2half(sn[x / 2]) : __low2half(sn[x / 2]),
                                                   y & 1 ? __high2half(sn[y / 2]) : __low2half(sn[y / 2]));
                                const __half2 h2 = half2_of(hi), hs = __hmul2(h2, sc);
                                lo = bits_of(__hfma2(half2_of(lo), sc, __hfma2(h2, sc, __hneg2(hs))));
                                hi = bits_of(hs);
                            }
                        };
                        pair(0, pa[t][i].x, pa[t][i].y);
                        pair(1, pa[t][i].z, pa[t][i].w);
                    }
                }
#pragma unroll
                for (int nt = 0; nt < kTilesG; ++nt) {
                    const int e = w * kSlice + 8 * (sg * kTilesG + nt) + n8;
                    uint32_t vv[8];
                    if constexpr (FMT == KQ_KV_F16) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint4 v = *reinterpret_cast<const uint4 *>(
                                vb + L::v_word(e, token(8 * h) / 2));
                            vv[4 * h] = v.x, vv[4 * h + 1] = v.y;
                            vv[4 * h + 2] = v.z, vv[4 * h + 3] = v.w;
                        }
                        if (edge) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) vv[i] &= keep[i];
                        }
                    } else if constexpr (FMT == KQ_KV_Q8) {
                        const uint4 v = *reinterpret_cast<const uint4 *>(vb + L::v_word(e, 4 * c));
                        codes8(v.x, vv[0], vv[1]);
                        codes8(v.y, vv[2], vv[3]);
                        codes8(v.z, vv[4], vv[5]);
                        codes8(v.w, vv[6], vv[7]);
                    } else {
                        const uint2 v = *reinterpret_cast<const uint2 *>(vb + L::v_word(e, 2 * c));
                        uint32_t x[4];
                        codes4(v.x, x);
#pragma unroll
                        for (int i = 0; i < 4; ++i) vv[i] = x[i];
                        codes4(v.y, x);
#pragma unroll
                        for (int i = 0; i < 4; ++i) vv[4 + i] = x[i];
                    }
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int i = 0; i < 4; ++i) mma(d, pa[t][i], vv[2 * i], vv[2 * i + 1]);
                        float *o = O[t][sg * kTilesG + nt];
                        if constexpr (L::kQuant) {
                            o[0] = fmaf(d[0] + d[2], fac, o[0] * alpha[t]);
                            o[1] = fmaf(d[1] + d[3], fac, o[1] * alpha[t]);
                        } else {
                            o[0] = fmaf(o[0], alpha[t], d[0] + d[2]);
                            o[1] = fmaf(o[1], alpha[t], d[1] + d[3]);
                        }
                    }
                }
                // values that are not finite reach the rows that attend them
                while (bad) {
                    const int tok = __ffsll((long long)bad) - 1;
                    bad &= bad - 1;
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        const int r = 8 * t + n8;
                        if (!((allowed(r) >> tok) & 1)) continue;
                        const float pv = ps[p_at<FMT>(r, tok)];
#pragma unroll
                        for (int nt = 0; nt < kTilesG; ++nt)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const int e = w * kSlice + 8 * (sg * kTilesG + nt) + 2 * c + i;
                                const uint32_t v = *reinterpret_cast<const uint32_t *>(
                                    vb + L::v_word(e, tok / L::kVPerWord));
                                const int bit = tok % L::kVPerWord * L::kBits;
                                float x;
                                if constexpr (L::kQuant)
                                    x = (float)((int)(v << (32 - L::kBits - bit)) >> (32 - L::kBits)) *
                                        __half2float(*reinterpret_cast<const __half *>(
                                            vb + L::v_scale(tok, group)));
                                else
                                    x = __half2float(__ushort_as_half((uint16_t)(v >> bit)));
                                float &o = O[t][sg * kTilesG + nt][i];
                                o = fmaf(pv, x, o);
                            }
                    }
                }
            }
        }

        // ---- the segment's rows: groups joined, then out or to a partial
        // result (the ring is idle now and holds the groups' values)
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            float v = l[t];
            v += __shfl_xor_sync(~0u, v, 1);
            v += __shfl_xor_sync(~0u, v, 2);
            if (c == 0) {
                cm.ml[g][1 + w][8 * t + n8] = v;
                if (w == 0) cm.ml[g][0][8 * t + n8] = m[t];
            }
        }
        // after an expired wait: no copy may land later than this
        if (w == 0 && lane == 0 && *(volatile int *)&cm.dead)
            for (int i = max(0, live - a.nslot); i < live; ++i)
                kq::mbar_wait(bars + 8 * ((op0 + i) % a.nslot), ((op0 + i) / a.nslot) & 1,
                              kq::kWaitLimitNs);
        op0 += 2 * count;
        group_sync<kGroupThreads>(g);
        float *os = reinterpret_cast<float *>(gbase);
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int nt = 0; nt < kTiles; ++nt)
                *reinterpret_cast<float2 *>(os + (8 * t + n8) * D + w * kSlice + 8 * nt + 2 * c) =
                    make_float2(O[t][nt][0], O[t][nt][1]);
        __syncthreads();
        const bool whole = npg == pages;
        const int slot = u == u0 ? 0 : 1;
        float *part = a.part + (2 * (int64_t)blockIdx.x + slot) * part_floats(RB, D);
        for (int i = tid; i < nrows * (D / 4); i += nthreads) {
            const int r = i / (D / 4), e = 4 * (i % (D / 4));
            float top = -INFINITY;
            for (int k = 0; k < a.ng; ++k) top = fmaxf(top, cm.ml[k][0][r]);
            const float base = top == -INFINITY ? 0.f : top;
            float sum = 0.f;
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int k = 0; k < a.ng; ++k) {
                const float f = exp2_of(cm.ml[k][0][r] - base);
                const float *lk = &cm.ml[k][1][r];
                float lsum = lk[0];
#pragma unroll
                for (int i = 1; i < kWg; ++i) lsum += lk[32 * i];
                sum = fmaf(f, lsum, sum);
                const float4 v = *reinterpret_cast<const float4 *>(
                    smem + M::kCommon + M::kQ + k * M::group(a.nslot) + 4 * (r * D + e));
                y.x = fmaf(f, v.x, y.x), y.y = fmaf(f, v.y, y.y);
                y.z = fmaf(f, v.z, y.z), y.w = fmaf(f, v.w, y.w);
            }
            if (cm.dead) sum = quiet_nan();
            if (whole) {
                const float inv = sum == 0.f ? 0.f : __fdiv_rn(1.f, sum);
                const int tok = (row0 + r) / a.per, hq = (row0 + r) % a.per;
                *reinterpret_cast<float4 *>(
                    a.out + ((int64_t)(s.first + tok) * a.q_heads + head * a.per + hq) * D + e) =
                    make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv);
            } else {
                *reinterpret_cast<float4 *>(part + r * D + e) = y;
                if (e == 0) part[RB * D + r] = top, part[RB * D + RB + r] = sum;
            }
        }
        if (tid == 0 && !whole && pg0 == 0) {
            a.meta[2 * blockIdx.x] =
                make_int4(cta_of(u + pages - 1, total, gridDim.x), slot, nrows, head);
            a.meta[2 * blockIdx.x + 1] = make_int4(s.first, row0, 0, 0);
        }
        // what was written to the ring comes before the next copies into it
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncthreads();
        u += npg;
        off += npg;
    }
}

// Joins the partial results of the item that begins in CTA blockIdx.x and
// goes on: one row a block, four runs of parts at a time.
template <int D, int RB>
__global__ void __launch_bounds__(4 * D)
    kq_attn_join(const __grid_constant__ AttnArgs a) {
    __shared__ float acc[4][D], sums[4];
    kq::wait_prerequisites();
    const int4 m0 = a.meta[2 * blockIdx.x];
    const int r = blockIdx.y, e = threadIdx.x % D, run = threadIdx.x / D;
    if (m0.x < 0 || r >= m0.z) return;
    const int4 m1 = a.meta[2 * blockIdx.x + 1];
    const int first = blockIdx.x, n = m0.x - first + 1;
    // part i: slot m0.y of the first CTA, slot 0 of those after it
    auto part = [&](int i) {
        return a.part + (2 * (int64_t)(first + i) + (i ? 0 : m0.y)) * part_floats(RB, D);
    };
    float top = -INFINITY;
    for (int i = threadIdx.x; i < n; i += 4 * D) top = fmaxf(top, part(i)[RB * D + r]);
#pragma unroll
    for (int o = 16; o; o /= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    __shared__ float wt[4 * D / 32];
    if ((threadIdx.x & 31) == 0) wt[threadIdx.x / 32] = top;
    __syncthreads();
    for (int i = 0; i < 4 * D / 32; ++i) top = fmaxf(top, wt[i]);
    const float base = top == -INFINITY ? 0.f : top;
    float y = 0.f, sum = 0.f;
#pragma unroll 4
    for (int i = run; i < n; i += 4) {
        const float *p = part(i);
        const float f = exp2_of(p[RB * D + r] - base);
        sum = fmaf(f, p[RB * D + RB + r], sum);
        y = fmaf(f, p[r * D + e], y);
    }
    acc[run][e] = y;
    if (e == 0) sums[run] = sum;
    __syncthreads();
    if (run) return;
    sum = (sums[0] + sums[1]) + (sums[2] + sums[3]);
    y = (acc[0][e] + acc[1][e]) + (acc[2][e] + acc[3][e]);
    const int tok = (m1.y + r) / a.per, hq = (m1.y + r) % a.per;
    a.out[((int64_t)(m1.x + tok) * a.q_heads + m0.w * a.per + hq) * D + e] =
        sum == 0.f ? 0.f : __fdiv_rn(y, sum);
}

// ------------------------------------------------------------------ launch
// CTAs of a launch, groups and slots of each.
struct AttnShape {
    int ctas, ng, nslot;
};

template <int FMT, int D, int MT>
cudaError_t launch_attn(AttnArgs a, int sms, cudaStream_t s, int64_t *floats) {
    using M = AttnSmem<FMT, D, MT>;
    // 16 warps of an SM in all: in one CTA that joins them where there are few
    // items, else in four, so that a CTA's warps have fewer items to join.
    // Fewer where a slot is too large for three a group.
    const int kSm = 227 * 1024;
    const int64_t items = (int64_t)a.q.nseq * a.q.heads *
                          (((int64_t)a.q.max_new * a.per + M::kRows - 1) / M::kRows);
    AttnShape sh;
    auto fit = [&](int ctas) {  // CTAs of an SM
        const int room = kSm / ctas - 1024 - M::kCommon - M::kQ;
        sh.ctas = ctas * sms;
        sh.ng = M::kGroups / ctas;
        while (sh.ng > 1 && room / sh.ng - M::kP - M::kMax < 3 * M::kHalf) --sh.ng;
        sh.nslot = (room / sh.ng - M::kP - M::kMax) / M::kHalf;
    };
    fit(4);
    if (items < 4 * (int64_t)sms || sh.nslot < 3) fit(1);
    if (sh.nslot > kMaxSlots) sh.nslot = kMaxSlots;
    *floats = 2 * (int64_t)sh.ctas * part_floats(M::kRows, D);
    if (!a.part) return cudaSuccess;
    a.ng = sh.ng, a.nslot = sh.nslot;
    a.meta = reinterpret_cast<int4 *>(a.part);  // meta first, 16-byte aligned
    a.part += 8 * (int64_t)sh.ctas;
    const int smem = M::total(sh.ng, sh.nslot);
    static std::mutex mu;
    static int configured[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (dev < 0 || dev >= 64 || configured[dev] < smem) {
            e = cudaFuncSetAttribute(kq_attn_kernel<FMT, D, MT>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (e != cudaSuccess) return e;
            if (dev >= 0 && dev < 64) configured[dev] = smem;
        }
    }
    kq_attn_kernel<FMT, D, MT><<<sh.ctas, 32 * M::kWg * sh.ng, smem, s>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(sh.ctas, M::kRows);
    cfg.blockDim = dim3(4 * D);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kq_attn_join<D, M::kRows>, a);
}

// The launch for a format and width: tiles of a row block by the rows that a
// key head has.
template <int FMT>
cudaError_t attn_format(int dim, const AttnArgs &a, int sms, cudaStream_t s, int64_t *floats) {
    const int64_t rows = (int64_t)a.q.max_new * a.per;
    switch (dim) {
    case 64:
        return rows <= 8    ? launch_attn<FMT, 64, 1>(a, sms, s, floats)
               : rows <= 16 ? launch_attn<FMT, 64, 2>(a, sms, s, floats)
                            : launch_attn<FMT, 64, 4>(a, sms, s, floats);
    case 128:
        return rows <= 8    ? launch_attn<FMT, 128, 1>(a, sms, s, floats)
               : rows <= 16 ? launch_attn<FMT, 128, 2>(a, sms, s, floats)
                            : launch_attn<FMT, 128, 4>(a, sms, s, floats);
    default:
        return rows <= 8 ? launch_attn<FMT, 256, 1>(a, sms, s, floats)
                         : launch_attn<FMT, 256, 2>(a, sms, s, floats);
    }
}

}  // namespace kqd
