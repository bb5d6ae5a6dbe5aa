// kq_attn.cuh -- attention of new tokens over the paged cache
// (kq_tree_attention): the kernel, compiled per cache format in
// kq_attn_<format>.cu.
//
// Work.  An item is a key head of a sequence with a block of its rows (a row
// is a new token and one of the query heads that share the key head); its
// units are the sequence's pages.  All units in order are cut into as many
// equal runs as there are CTAs, so ragged lengths balance (each item by itself
// where CTAs have few units); an item that falls into several runs leaves a
// partial result (row maxima, sums, weighted values) in each, joined by
// kq_attn_join.
//
// A page.  A CTA has groups of two or four warps; a group takes whole pages, two
// bulk copies each (keys, values) into a ring of its own, and works on one
// page at a time:
//   1. each warp forms the logits of its share of the page's 64 tokens,
//   2. the warps exchange row maxima, form the probabilities and leave them
//      in shared memory,
//   3. each warp adds its share of the values' width, over all 64 tokens.
//
// Arithmetic.  The tensor cores take f16 operands, and codes are exact in
// f16.  Keys and values are the operand of 16 rows (tokens, or places of the
// values' width), four rows of queries or probabilities that of eight
// columns: they are f32, held as two f16 terms hi + lo (22 bits) side by
// side, so that one m16n8k16 MMA forms both products and a lane adds the two
// in f32.  (Eight rows as the operand of 16, hi above lo, gave half the useful
// work to an MMA where a key head has four rows, and the rate of these MMAs,
// one in eight clocks an SM, was what bounded the kernel.)  A query row is
// scaled by a power of two first (its largest magnitude below 2^15), the
// values' scales by page and group, probabilities by 2^15.  Scales of
// quantised keys multiply the f32 sums of their group; those of values
// multiply the probabilities' terms, whose rounding joins the lower term.
// Each page's sums start at zero and are added to the running ones in f32,
// with the correction of the row's running reference, its maximum less 15.
// (The maximum and the 15 together, taken off each logit, lost the 15 to
// rounding past 2^24.)
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

#include <atomic>

#include "kq_async.cuh"
#include "kq_decode.cuh"
#include "kq_decode_launch.h"

namespace kqd {

constexpr int kMaxGroups = 8;
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
    uint32_t suspend_ns;  // the lesser of it and kq::kSuspendNs
    int32_t q_heads, per;  // query heads; of them to a key head
    float scale_m;         // scale times log2 e = scale_m * 2^scale_e,
    int32_t scale_e;       // |scale_m| in 0.5..1, or 0
    int32_t ng, nslot;     // groups a CTA, slots of a group's ring
};

// Rows of a CTA's block, floats of a partial result.
__host__ __device__ constexpr int part_floats(int rb, int d) { return rb * (d + 2); }

// ------------------------------------------------------------ shared memory
// common | queries | per group: ring, probabilities, maxima
struct RunShared {
    long long scan[32];
    uint32_t items[32], runs[32];
    long long off;
    int seq, pages, parts;
};
struct AttnCommon {
    uint64_t rowmask[32];
    uint64_t bars[kMaxGroups * kMaxSlots];   // a slot's copy has arrived
    uint64_t empty[kMaxGroups * kMaxSlots];  // and has been used
    RunShared run;
    int dead;                              // a wait has expired
    int badpage[kMaxGroups * kMaxSlots];   // the slot's page is not valid
    float rowfactor[32];
    float ml[kMaxGroups][5][32];           // group's row maxima, warps' row sums
};
template <int FMT, int D, int NT>
struct AttnSmem {
    static constexpr int kRows = 4 * NT;
    // Warps of a group: two, so that less is waited for at its barrier and
    // counted for a page; four for f16, of whose pages shared memory holds
    // fewer, and for width 256 (registers).
    static constexpr int kWg = FMT != KQ_KV_F16 && D <= 128 ? 2 : 4;
    static constexpr int kHalf = Kv<FMT, D>::kV;  // bytes of a slot
    static constexpr int kCommon = (sizeof(AttnCommon) + 127) / 128 * 128;
    static constexpr int kQ = kRows * D * 4;
    static constexpr int kP = 2 * 2 * kRows * kPage * 2;  // hi and lo columns, two pages
    static constexpr int kMax = 2 * kWg * kRows * 4;
    // Groups of an SM, by tiles: what registers hold (96 a thread for 20 warps,
    // 128 for 16, 168 for 12), less where shared memory holds fewer with three
    // slots each; of four warps one less for f16, whose slots are twice as
    // large.  Four warps (5, 4, 3, 3 groups) / two warps (8, 7, 5, 5), 8-bit,
    // 1..4 tiles: 153 / 139 us (32 sequences of 16384 tokens at most, 32 / 8
    // heads), 62.8 / 59.7 (16 sequences, 32 / 4), 50.9 / 47.9 (24 / 2), 65.2 /
    // 56.7 (32 / 2); 4-bit 165 / 145, 64.7 / 59.8, 49.7 / 51.2, 60.4 / 59.2.
    // Two warps, one tile, 10 / 8 / 7 groups, 4-bit: 155 / 145 / 145, and 107 /
    // 97 / 114 for 128 sequences of 2000; two tiles, 8 / 7 / 6: 64.9 / 59.8 /
    // 60.3; four tiles, 6 / 5 / 4: 69.9 / 59.2 / 60.8.  Four warps, f16, two
    // tiles, 4 / 3: 76.9 / 66.1; three tiles, 4 / 3 / 2: 64.9 / 50.6 / 51.9.
    static constexpr int kSm = 227 * 1024;
    static constexpr int kMost = kWg == 2 ? (NT == 1 ? 8 : NT == 2 ? 7 : 5)
                                 : (NT == 1 ? 5 : NT == 2 ? 4 : 3) - (FMT == KQ_KV_F16 && NT < 3);
    // of each of `ctas` CTAs of an SM
    static constexpr int groups(int ctas) {
        const int fit = (kSm / ctas - 1024 - kCommon - kQ) / (3 * kHalf + kP + kMax);
        return fit < kMost / ctas ? fit : kMost / ctas;
    }
    static constexpr int kGroups = groups(1);
    // CTAs of an SM that hold the most groups, more than one if that can be
    static constexpr int apart() {
        int best = 1, most = 0;
        for (int c = 4; c > 1; --c)
            if (c * groups(c) > most) best = c, most = c * groups(c);
        return best;
    }
    static_assert(kGroups >= 1, "a group");
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
// The exponent of 2 in a row's factor, for queries below 2^ex that were brought
// below 2^15: past either end the scaled query is not finite, or the logits
// vanish.
__device__ __forceinline__ int factor_exponent(int ex, int scale_e) {
    return min(max(ex - 15 + scale_e, -126), 127);
}
template <int THREADS>
__device__ __forceinline__ void group_sync(int g) {
    asm volatile("bar.sync %0, %1;" ::"r"(g + 1), "n"(THREADS) : "memory");
}

// Probabilities in shared memory: columns (row hi, row lo, next row hi, ...)
// of 64 f16 in the order in which the values' operand takes the tokens: a
// lane quarter's 16 are two chunks of eight; odd columns are turned by one.
template <int FMT>
__device__ __forceinline__ int p_at(int col, int tok) {
    int chunk = tok >> 3, k = tok & 7;
    if (FMT == KQ_KV_F16) chunk = 2 * (chunk & 3) + (chunk >> 2);
    if (FMT == KQ_KV_Q4) k = 2 * (k & 3) + (k >> 2);  // pairs (0, 4), (1, 5) ...
    return col * kPage + ((chunk ^ (col & 1)) << 3) + k;
}

// ------------------------------------------------------------------- units
// Pages of a sequence that are looked at: up to the last new token, but no
// more than one page past the table (a committed place without a page makes
// every row NaN already).
__device__ __forceinline__ int64_t pages_of(const Seqs &q, const Seq &s) {
    const int64_t n = ((int64_t)s.ctx + s.n + kPage - 1) / kPage;
    return s.ctx / kPage > q.max_pages ? q.max_pages + 1 : n;
}
// (rb: rows of a block)
__device__ __forceinline__ int64_t units_of(const AttnArgs &a, const Seq &s, int rb, int &blocks) {
    blocks = (s.n * a.per + rb - 1) / rb;
    return s.n ? pages_of(a.q, s) * blocks * a.q.heads : 0;
}
// CTA that works on unit u, of `total` cut into n runs.
__device__ __forceinline__ int cta_of(long long u, long long total, int n) {
    const long long base = total / n, rem = total % n;
    return (int)(u < rem * (base + 1) ? u / (base + 1) : rem + (u - rem * (base + 1)) / base);
}

// This CTA's run [u0, u1) of units; it begins at unit `off` of sequence `seq`.
// Every thread of the block takes part (nthreads, a multiple of 32).
//
// All units are cut evenly where CTAs have many.  Where they have few, a CTA
// that ends one item and begins another would take the longer: then each item
// is cut by itself into `parts` runs, none longer than `most` pages
// (sum of ceil(pages / most) <= units / most + items <= CTAs).  A second item
// costs a CTA 4 to 6 us or more, kApartPages pages' time: one sequence of 4000
// tokens, 32 / 8 heads, 8-bit, 17.5 us cut evenly and 13.0 by items.
struct Run {
    long long u0, u1, total, off;
    int seq;
    int parts;  // runs of the item (0: cut evenly over all units)
};
constexpr int kApartPages = 8;
__device__ __forceinline__ Run run_of(const AttnArgs &a, int rb, int nthreads, RunShared &sh) {
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, nw = nthreads / 32;
    const int each = (a.q.nseq + nthreads - 1) / nthreads;
    const int b0 = min(tid * each, a.q.nseq), b1 = min(b0 + each, a.q.nseq);
    if (tid == 0) a.meta[2 * blockIdx.x] = make_int4(-1, 0, 0, 0);
    // the last sequence looked at stays, as a thread mostly has one
    int known = -1, pages = 0;
    long long items = 0;
    auto look = [&](int b) {
        if (b == known) return;
        const Seq s = seq_of(a.q, b);
        known = b;
        pages = s.n ? (int)pages_of(a.q, s) : 0;
        items = s.n ? (int64_t)((s.n * a.per + rb - 1) / rb) * a.q.heads : 0;
    };
    long long mine = 0, count = 0;
    for (int b = b0; b < b1; ++b) look(b), mine += pages * items, count += items;
    long long upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const long long v = __shfl_up_sync(~0u, upto, o);
        if (lane >= o) upto += v;
    }
    const uint32_t some = __reduce_add_sync(~0u, (uint32_t)min(count, 1ll << 20));
    if (lane == 31) sh.scan[w] = upto, sh.items[w] = some;
    __syncthreads();
    Run r;
    r.total = 0;
    uint32_t nitems = 0;
    for (int i = 0; i < nw; ++i) {
        if (i == w) upto += r.total;
        r.total += sh.scan[i];
        nitems += sh.items[i];
    }
    const uint32_t grid = gridDim.x, k = blockIdx.x;
    uint32_t most = 0;
    if (nitems < grid && r.total > grid && r.total < 1 << 30) {
        const uint32_t n = (uint32_t)r.total, room = grid - nitems;
        most = (n + room - 1) / room;
        if (most > (n + grid - 1) / grid + kApartPages) most = 0;
    }
    r.parts = 0;
    if (most) {
        uint32_t runs = 0;
        for (int b = b0; b < b1; ++b) look(b), runs += (uint32_t)items * ((pages + most - 1) / most);
        uint32_t to = runs;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const uint32_t v = __shfl_up_sync(~0u, to, o);
            if (lane >= o) to += v;
        }
        if (lane == 31) sh.runs[w] = to;
        __syncthreads();
        uint32_t all = 0;
        for (int i = 0; i < nw; ++i) {
            if (i == w) to += all;
            all += sh.runs[i];
        }
        if (k >= to - runs && k < to) {
            uint32_t at = to - runs;
            for (int b = b0;; ++b) {
                look(b);
                const uint32_t parts = (pages + most - 1) / most, n = (uint32_t)items * parts;
                if (k < at + n) {
                    const uint32_t item = (k - at) / parts, j = (k - at) - item * parts;
                    const uint32_t base = pages / parts, rem = pages - base * parts;
                    sh.seq = b, sh.parts = (int)parts;
                    sh.off = (long long)item * pages + j * base + min(j, rem);
                    sh.pages = (int)(base + (j < rem));
                    break;
                }
                at += n;
            }
        }
        __syncthreads();
        r.u0 = 0, r.u1 = k < all ? sh.pages : 0;
        r.parts = sh.parts;
    } else {
        const long long base = r.total / grid, rem = r.total - base * grid;
        r.u0 = k * base + min((long long)k, rem);
        r.u1 = r.u0 + base + (k < rem ? 1 : 0);
        if (r.u0 < r.u1 && r.u0 >= upto - mine && r.u0 < upto) {
            long long at = upto - mine;
            int b = b0;
            for (;; ++b) {
                look(b);
                if (r.u0 < at + pages * items) break;
                at += pages * items;
            }
            sh.seq = b;
            sh.off = r.u0 - at;
        }
        __syncthreads();
    }
    r.seq = sh.seq;
    r.off = sh.off;
    return r;
}
// The last CTA of an item that begins in this one, at unit u.
__device__ __forceinline__ int last_cta(const Run &run, long long u, int pages) {
    return run.parts ? blockIdx.x + run.parts - 1 : cta_of(u + pages - 1, run.total, gridDim.x);
}

// ------------------------------------------------------------------ kernel
template <int FMT, int D, int NT>
__global__ void __launch_bounds__(AttnSmem<FMT, D, NT>::kGroups * AttnSmem<FMT, D, NT>::kWg * 32 + 32, 1)
    kq_attn_kernel(const __grid_constant__ AttnArgs a) {
    using L = Kv<FMT, D>;
    using M = AttnSmem<FMT, D, NT>;
    constexpr int RB = M::kRows;
    constexpr int kWg = M::kWg, kGroupThreads = 32 * kWg;
    constexpr int kTok = kPage / 16 / kWg;  // tiles of 16 tokens of a warp in part 1
    constexpr int kSlice = D / kWg;         // values of a warp in part 3
    constexpr int kTiles = kSlice / 16;     // its tiles
    constexpr int kSliceGroups = kSlice > kGroup ? kSlice / kGroup : 1;
    constexpr int kTilesG = kTiles / kSliceGroups;

    extern __shared__ __align__(128) uint8_t smem[];
    AttnCommon &cm = *reinterpret_cast<AttnCommon *>(smem);
    uint4 *qs = reinterpret_cast<uint4 *>(smem + M::kCommon);  // [tile][group][lane]
    const int tid = threadIdx.x, lane = tid & 31;
    const int ntail = a.ng * kGroupThreads;   // threads of the groups
    const bool producer = tid >= ntail;       // the last warp issues the copies
    // (in the producer warp lane g serves group g)
    const int g = producer ? min(tid - ntail, a.ng - 1) : tid / kGroupThreads;
    const int w = (tid >> 5) % kWg;
    const int n8 = lane >> 2, c = lane & 3;  // row or column of an operand, and its quarter;
                                             // in results: token or place n8 (+ 8), row c of four
    const int nthreads = ntail + 32;
    uint8_t *gbase = smem + M::kCommon + M::kQ + g * M::group(a.nslot);
    __half *ps = reinterpret_cast<__half *>(gbase + a.nslot * M::kHalf);
    float *smax = reinterpret_cast<float *>(gbase + a.nslot * M::kHalf + M::kP);  // [warp][row]
    const uint32_t ring = kq::smem_addr(gbase);
    const uint32_t bars = kq::smem_addr(&cm.bars[g * kMaxSlots]);

    if (tid < a.ng * kMaxSlots && (tid % kMaxSlots) < a.nslot) {
        kq::mbar_init(kq::smem_addr(&cm.bars[tid]), 1);
        kq::mbar_init(kq::smem_addr(&cm.empty[tid]), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (tid == 0) cm.dead = 0;
    kq::allow_dependents();  // kq_attn_join waits for this kernel's end

    const Run run = run_of(a, RB, nthreads, cm.run);
    if (run.u0 >= run.u1) return;

    // the group's ring: next slot to fill or to use, its turn's parity, and
    // the first slot that is in use and not yet handed back
    int use = 0, back = 0;
    uint32_t parity = 0;
    int primed = 0;  // (producer) slots of the ring that have been filled once
    int b = run.seq;
    long long off = run.off;
    for (long long u = run.u0; u < run.u1 && b < a.q.nseq;) {
        // ---- the segment: pages [pg0, pg0 + npg) of one item
        int blocks;
        Seq s = seq_of(a.q, b);
        const long long units = units_of(a, s, RB, blocks);
        if (off >= units) {
            ++b, off = 0;
            continue;
        }
        const int pages = (int)pages_of(a.q, s);
        const int item = (int)(off / pages);
        const int pg0 = (int)(off - (long long)item * pages);
        const int npg = (int)min((long long)(pages - pg0), run.u1 - u);
        const int head = item / blocks, row0 = (item - head * blocks) * RB;
        const int nrows = min(RB, s.n * a.per - row0);
        const int count = npg > g ? (npg - g + a.ng - 1) / a.ng : 0;  // the group's pages

        // ---- the producer warp: lane g copies group g's keys and values into
        // its ring, in the order of their use: the first keys, then the next
        // page's keys and a page's values by turns, the last values
        const int mine = producer && tid - ntail < a.ng ? 2 * count : 0;
        int issued = 0;
        int64_t kpage = -1, vpage = -1, next = mine ? page_of(a.q, b, pg0 + g) : -1;
        auto pump = [&](int until) {  // (the whole warp)
            unsigned long long since = 0;  // the lane waits for its slot (0: it does not)
            while (__any_sync(~0u, issued < until)) {
                if (__any_sync(~0u, *(volatile int *)&cm.dead)) break;
                // (a slot's first filling waits for nothing)
                bool room = issued < until &&
                            (primed < a.nslot ||
                             kq::mbar_test(kq::smem_addr(&cm.empty[g * kMaxSlots + use]), parity ^ 1));
                // (a group whose wait ran out hands back slots whose copies may be
                // on their way: it sets `dead` first, so this look comes after
                // the one at the slot)
                room = room && !*(volatile int *)&cm.dead;
                if (room) {
                    const int i = issued++;
                    const bool values = i == mine - 1 || (i > 0 && (i & 1) == 0);
                    if (!values) {
                        vpage = kpage, kpage = next;
                        const int k = (i + 1) / 2 + 1;  // the next page, looked up ahead
                        if (k < count) next = page_of(a.q, b, pg0 + g + (int64_t)k * a.ng);
                    }
                    const int64_t page = !values || i == mine - 1 ? kpage : vpage;
                    const uint32_t bar = bars + 8 * use;
                    cm.badpage[g * kMaxSlots + use] = page < 0;
                    kq::mbar_expect_tx(bar, M::kHalf);
                    kq::bulk_g2s(ring + use * M::kHalf,
                                 a.q.data + (max(page, (int64_t)0) * a.q.heads + head) * L::kBlock +
                                     (values ? M::kHalf : 0),
                                 M::kHalf, bar);
                    if (primed < a.nslot) ++primed;
                    if (++use == a.nslot) use = 0, parity ^= 1;
                    since = 0;
                } else if (issued < until) {
                    const unsigned long long now = kq::global_ns();
                    if (!since) since = now;
                    if (now - since > a.wait_ns) {
                        *(volatile int *)&cm.dead = 1;
                        atomicOr(a.err, 1u);
                    }
                }
            }
        };
        if (producer) pump(min(mine, a.nslot));

        // ---- queries: rows scaled by a power of two, hi and lo terms, laid
        // out as the operands of part 1
        for (int r = tid >> 5; !producer && r < RB; r += ntail / 32) {
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
                cm.rowfactor[r] = a.scale_m *
                                  __uint_as_float((uint32_t)(127 + factor_exponent(ex, a.scale_e)) << 23);
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
                    uint2 hi, lo;
                    split(x[0], x[1], hi.x, lo.x);
                    split(x[2], x[3], hi.y, lo.y);
                    const int octet = e >> 3;
                    uint2 *o = reinterpret_cast<uint2 *>(
                        qs + ((r >> 2) * L::kGroups + (octet >> 2)) * 32 + 8 * (r & 3) + (octet & 3));
                    o[(e >> 2) & 1] = hi;      // column 2 r
                    o[8 + ((e >> 2) & 1)] = lo;  // column 2 r + 1: four lanes on
                }
            }
        }
        __syncthreads();
        if (producer) {
            pump(mine);
            __syncwarp();
        }

        float m[NT], l[NT], O[NT][kTiles][2];  // rows 4 t + c
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            m[t] = -INFINITY, l[t] = 0.f;
#pragma unroll
            for (int i = 0; i < kTiles; ++i) O[t][i][0] = O[t][i][1] = 0.f;
        }

        // the next slot, once its copy has arrived
        auto arrived = [&]() {
            if (!*(volatile int *)&cm.dead &&
                !kq::mbar_wait_for(bars + 8 * use, parity, a.wait_ns, a.suspend_ns)) {
                *(volatile int *)&cm.dead = 1;
                atomicOr(a.err, 1u);
            }
            const int slot = use;
            if (++use == a.nslot) use = 0, parity ^= 1;
            return slot;
        };
        // A turn forms page k's logits, adds page k - 1's values and forms page
        // k's probabilities, with one barrier: maxima and probabilities are
        // kept for two pages by turns.
        float alpha[NT];
        // bit t: row r may attend token t of a page with `left` committed
        // tokens in it and after
        auto allowed = [&](int left, int r) -> uint64_t {
            const uint64_t nw = cm.rowmask[r] & (~0ull >> (64 - s.n));
            if (left <= 0) return -left < 64 ? nw >> -left : 0;
            return left >= kPage ? ~0ull : (nw << left) | ~(~0ull << left);
        };
        for (int k = 0; k <= (count && !producer ? count : -1); ++k) {
            float S[NT][kTok][2];
            float *sm = smax + (k & 1) * kWg * RB;
            if (k < count) {
                const int left = s.ctx - (pg0 + g + k * a.ng) * kPage;
                const bool edge = left < kPage;  // new tokens, or the end
                // ---- 1. logits of tokens 16 w + n8 (+ 8)
                const int ks = arrived();
                const uint8_t *kb = gbase + ks * M::kHalf;
                const bool badpage = cm.badpage[g * kMaxSlots + ks];
#pragma unroll
                for (int tt = 0; tt < kTok; ++tt) {
                    float acc[NT][4];
                    constexpr int kLane = L::kSlabBytes / 4;  // bytes of a lane in a slab
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        S[t][tt][0] = S[t][tt][1] = 0.f;
                        acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0.f;
                    }
#pragma unroll
                    for (int sl = 0; sl < L::kSlabs; ++sl) {
                        uint32_t raw[2][kLane / 4];
                        uint32_t skw[2][(L::kSlabGroups + 1) / 2];  // scales, two groups a word
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const int tok = 16 * (kTok * w + tt) + 8 * j + n8;
                            const uint8_t *p =
                                kb + sl * kPage * L::kSlabBytes + tok * L::kSlabBytes + c * kLane;
                            if constexpr (kLane == 16) {
                                const uint4 v = *reinterpret_cast<const uint4 *>(p);
                                raw[j][0] = v.x, raw[j][1] = v.y, raw[j][2] = v.z, raw[j][3] = v.w;
                            } else {
                                const uint2 v = *reinterpret_cast<const uint2 *>(p);
                                raw[j][0] = v.x, raw[j][1] = v.y;
                            }
                            if constexpr (L::kQuant) {
                                const uint8_t *sp = kb + L::k_scale(tok, sl * L::kSlabGroups);
                                if constexpr (L::kSlabGroups == 4) {
                                    const uint2 v = *reinterpret_cast<const uint2 *>(sp);
                                    skw[j][0] = v.x, skw[j][1] = v.y;
                                } else {
                                    skw[j][0] = *reinterpret_cast<const uint32_t *>(sp);
                                }
                            }
                        }
#pragma unroll
                        for (int gl = 0; gl < L::kSlabGroups; ++gl) {
                            uint32_t bb[2][4];
                            float sk[2];
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
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
                                    const __half2 h = half2_of(skw[j][gl / 2]);
                                    sk[j] = gl & 1 ? __high2float(h) : __low2float(h);
                                }
                            }
                            const uint4 k0 = make_uint4(bb[0][0], bb[1][0], bb[0][1], bb[1][1]);
                            const uint4 k1 = make_uint4(bb[0][2], bb[1][2], bb[0][3], bb[1][3]);
#pragma unroll
                            for (int t = 0; t < NT; ++t) {
                                const uint4 q = qs[(t * L::kGroups + sl * L::kSlabGroups + gl) * 32 + lane];
                                if constexpr (L::kQuant) {
                                    float d[4] = {0.f, 0.f, 0.f, 0.f};
                                    mma(d, k0, q.x, q.y);
                                    mma(d, k1, q.z, q.w);
                                    S[t][tt][0] = fmaf(sk[0], d[0] + d[1], S[t][tt][0]);
                                    S[t][tt][1] = fmaf(sk[1], d[2] + d[3], S[t][tt][1]);
                                } else {
                                    mma(acc[t], k0, q.x, q.y);
                                    mma(acc[t], k1, q.z, q.w);
                                }
                            }
                        }
                    }
                    if constexpr (!L::kQuant) {
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            S[t][tt][0] = acc[t][0] + acc[t][1];
                            S[t][tt][1] = acc[t][2] + acc[t][3];
                        }
                    }
                }
                // ---- 2. row maxima
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const float f = badpage ? quiet_nan() : cm.rowfactor[4 * t + c];
                    float v = -INFINITY;
#pragma unroll
                    for (int tt = 0; tt < kTok; ++tt) {
                        S[t][tt][0] *= f, S[t][tt][1] *= f;
                        if (edge) {
                            const uint64_t ok = allowed(left, 4 * t + c) >> (16 * (kTok * w + tt) + n8);
                            if (!(ok & 1)) S[t][tt][0] = -INFINITY;
                            if (!(ok & 256)) S[t][tt][1] = -INFINITY;
                        }
                        v = fmaxf(v, fmaxf(S[t][tt][0], S[t][tt][1]));
                    }
                    v = fmaxf(v, __shfl_xor_sync(~0u, v, 4));
                    v = fmaxf(v, __shfl_xor_sync(~0u, v, 8));
                    v = fmaxf(v, __shfl_xor_sync(~0u, v, 16));
                    if (n8 == 0) sm[w * RB + 4 * t + c] = v;
                }
            }
            group_sync<kGroupThreads>(g);
            // every warp is done with page k's keys and page k - 2's values
            if (w == 0 && lane == 0) {
                const int n = (k < count) + (k > 1);
                for (int i = 0; i < n; ++i) {
                    kq::mbar_arrive(kq::smem_addr(&cm.empty[g * kMaxSlots + back]));
                    if (++back == a.nslot) back = 0;
                }
            }
            if (k > 0) {
                const int left = s.ctx - (pg0 + g + (k - 1) * a.ng) * kPage;
                const bool edge = left < kPage;
                const __half *pv = ps + ((k - 1) & 1) * 2 * RB * kPage;
                // ---- 3. values kSlice w .. of all 64 tokens
                const int vs = arrived();
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
                        for (int nt = 0; nt < 2 * kTiles; ++nt) {
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
                    // the slice's values, as operands of the four k-steps
                    uint4 vv[kTilesG][4];
#pragma unroll
                    for (int mt = 0; mt < kTilesG; ++mt) {
                        uint32_t x[2][8];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int e = w * kSlice + 16 * (sg * kTilesG + mt) + 8 * h + n8;
                            if constexpr (FMT == KQ_KV_F16) {
#pragma unroll
                                for (int i = 0; i < 2; ++i) {
                                    const uint4 v = *reinterpret_cast<const uint4 *>(
                                        vb + L::v_word(e, token(8 * i) / 2));
                                    x[h][4 * i] = v.x, x[h][4 * i + 1] = v.y;
                                    x[h][4 * i + 2] = v.z, x[h][4 * i + 3] = v.w;
                                }
                                if (edge) {
#pragma unroll
                                    for (int i = 0; i < 8; ++i) x[h][i] &= keep[i];
                                }
                            } else if constexpr (FMT == KQ_KV_Q8) {
                                const uint4 v = *reinterpret_cast<const uint4 *>(vb + L::v_word(e, 4 * c));
                                codes8(v.x, x[h][0], x[h][1]);
                                codes8(v.y, x[h][2], x[h][3]);
                                codes8(v.z, x[h][4], x[h][5]);
                                codes8(v.w, x[h][6], x[h][7]);
                            } else {
                                const uint2 v = *reinterpret_cast<const uint2 *>(vb + L::v_word(e, 2 * c));
                                uint32_t y[4];
                                codes4(v.x, y);
#pragma unroll
                                for (int i = 0; i < 4; ++i) x[h][i] = y[i];
                                codes4(v.y, y);
#pragma unroll
                                for (int i = 0; i < 4; ++i) x[h][4 + i] = y[i];
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            vv[mt][i] =
                            make_uint4(x[0][2 * i], x[1][2 * i], x[0][2 * i + 1], x[1][2 * i + 1]);
                    }
                    // scales in the order of the probabilities' pairs
                    if constexpr (FMT == KQ_KV_Q4) {
#pragma unroll
                        for (int i = 0; i < 8; i += 4) {
                            const __half2 s01 = sn[i], s23 = sn[i + 1], s45 = sn[i + 2], s67 = sn[i + 3];
                            sn[i] = __lows2half2(s01, s45), sn[i + 1] = __highs2half2(s01, s45);
                            sn[i + 2] = __lows2half2(s23, s67), sn[i + 3] = __highs2half2(s23, s67);
                        }
                    }
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        // column n8: the hi or lo terms of row n8 / 2
                        uint32_t pb[8];
                        const int col = 8 * t + n8;
                        auto load = [&](int of, uint32_t (&x)[8]) {
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const uint4 v = *reinterpret_cast<const uint4 *>(
                                    pv + of * kPage + (((2 * c + i) ^ (of & 1)) << 3));
                                x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
                            }
                        };
                        if constexpr (L::kQuant) {
                            // (hi + lo) s as two terms: hi s is rounded, and what
                            // that loses (exact in f16) joins lo s
                            uint32_t hi[8], lo[8];
                            load(col & ~1, hi);
                            load(col | 1, lo);
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const __half2 h = half2_of(hi[i]), hs = __hmul2(h, sn[i]);
                                const __half2 off = __hfma2(h, sn[i], __hneg2(hs));
                                const __half2 ls = __hfma2(half2_of(lo[i]), sn[i], off);
                                pb[i] = n8 & 1 ? bits_of(ls) : bits_of(hs);
                            }
                        } else {
                            load(col, pb);
                        }
#pragma unroll
                        for (int mt = 0; mt < kTilesG; ++mt) {
                            float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                            for (int i = 0; i < 4; ++i) mma(d, vv[mt][i], pb[2 * i], pb[2 * i + 1]);
                            float *o = O[t][sg * kTilesG + mt];
                            if constexpr (L::kQuant) {
                                o[0] = fmaf(d[0] + d[1], fac, o[0] * alpha[t]);
                                o[1] = fmaf(d[2] + d[3], fac, o[1] * alpha[t]);
                            } else {
                                o[0] = fmaf(o[0], alpha[t], d[0] + d[1]);
                                o[1] = fmaf(o[1], alpha[t], d[2] + d[3]);
                            }
                        }
                    }
                    // values that are not finite reach the rows that attend them
                    while (bad) {
                        const int tok = __ffsll((long long)bad) - 1;
                        bad &= bad - 1;
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            const int r = 4 * t + c;
                            if (!((allowed(left, r) >> tok) & 1)) continue;
                            const float prob = __half2float(pv[p_at<FMT>(2 * r, tok)]) +
                                               __half2float(pv[p_at<FMT>(2 * r + 1, tok)]);
#pragma unroll
                            for (int mt = 0; mt < kTilesG; ++mt)
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    const int e = w * kSlice + 16 * (sg * kTilesG + mt) + 8 * h + n8;
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
                                    float &o = O[t][sg * kTilesG + mt][h];
                                    o = fmaf(prob, x, o);
                                }
                        }
                    }
                }
            }
            // ---- 2. probabilities
            if (k < count) {
                __half *pw = ps + (k & 1) * 2 * RB * kPage;
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const int r = 4 * t + c;
                    // Probabilities (and l, O) are held times 2^15.  The row's reference
                    // is its maximum less 15, rounded up, and all that follows goes by
                    // the reference: however large the logits are, and the steps in
                    // which f32 holds them, none passes 2^15.
                    float top = sm[r];
#pragma unroll
                    for (int i = 1; i < kWg; ++i) top = fmaxf(top, sm[i * RB + r]);
                    const float now = fmaxf(m[t], __fsub_ru(top, 15.f));
                    const float base = now == -INFINITY ? 0.f : now;
                    alpha[t] = exp2_of(m[t] - base);
                    m[t] = now;
                    l[t] *= alpha[t];
#pragma unroll
                    for (int tt = 0; tt < kTok; ++tt) {
                        const float p0 = exp2_of(S[t][tt][0] - base), p1 = exp2_of(S[t][tt][1] - base);
                        l[t] += p0 + p1;
                        const __half h0 = __float2half_rn(p0), h1 = __float2half_rn(p1);
                        const int tok = 16 * (kTok * w + tt) + n8;
                        pw[p_at<FMT>(2 * r, tok)] = h0;
                        pw[p_at<FMT>(2 * r, tok + 8)] = h1;
                        pw[p_at<FMT>(2 * r + 1, tok)] = __float2half_rn(p0 - __half2float(h0));
                        pw[p_at<FMT>(2 * r + 1, tok + 8)] = __float2half_rn(p1 - __half2float(h1));
                    }
                }
            }
        }

        // ---- the segment's rows: groups joined, then out or to a partial
        // result (the ring is idle now and holds the groups' values)
        if (!producer) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                float v = l[t];
                v += __shfl_xor_sync(~0u, v, 4);
                v += __shfl_xor_sync(~0u, v, 8);
                v += __shfl_xor_sync(~0u, v, 16);
                if (n8 == 0) {
                    cm.ml[g][1 + w][4 * t + c] = v;
                    if (w == 0) cm.ml[g][0][4 * t + c] = m[t];
                }
            }
            // (all copies have been used; the last page's values are handed back)
            group_sync<kGroupThreads>(g);
            if (count && w == 0 && lane == 0) {
                kq::mbar_arrive(kq::smem_addr(&cm.empty[g * kMaxSlots + back]));
                if (++back == a.nslot) back = 0;
            }
            float *os = reinterpret_cast<float *>(gbase);
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int mt = 0; mt < kTiles; ++mt)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        os[(4 * t + c) * D + w * kSlice + 16 * mt + 8 * h + n8] = O[t][mt][h];
        }
        __syncthreads();
        // After an expired wait no copy may land later than this.  (Not before
        // the barrier: a group's wait may expire when the producer is done, with
        // copies on their way.  The last one of a slot is this lap's before `use`,
        // else the lap's before.)
        if (producer && tid - ntail < a.ng && *(volatile int *)&cm.dead) {
            for (int k = 0; k < primed; ++k)
                kq::mbar_wait(bars + 8 * k, parity ^ (k >= use), kq::kWaitLimitNs);
        }
        const bool whole = npg == pages;
        const int slot = u == run.u0 ? 0 : 1;
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
                make_int4(last_cta(run, u, pages), slot, nrows, head);
            a.meta[2 * blockIdx.x + 1] = make_int4(s.first, row0, 0, 0);
        }
        // what was written to the ring comes before the next copies into it
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncthreads();
        u += npg;
        off += npg;
    }
}

// Joins partial results: a job is a row of an item that begins in one CTA and
// goes on in others.  Every block counts the jobs of all CTAs and takes its
// share; a row's parts are added in four runs side by side, in their order.
// (A block per CTA and row, most of them with nothing to do, took 36 us for
// 128 rows.)
constexpr int kJoinRuns = 4;
template <int D>
__global__ void __launch_bounds__(kJoinRuns *D)
    kq_attn_join(const __grid_constant__ AttnArgs a, int rb, int ctas) {
    constexpr int kThreads = kJoinRuns * D, kWarps = kThreads / 32;
    __shared__ float acc[kJoinRuns][D], sums[kJoinRuns], wt[kWarps];
    __shared__ int scan[kWarps], job[2];
    kq::wait_prerequisites();
    const int tid = threadIdx.x, lane = tid & 31, e = tid % D, run = tid / D;
    // this thread's CTAs, and the jobs before them
    const int each = (ctas + kThreads - 1) / kThreads;
    const int c0 = min(tid * each, ctas), c1 = min(c0 + each, ctas);
    int mine = 0;
    for (int i = c0; i < c1; ++i) mine += a.meta[2 * i].x < 0 ? 0 : a.meta[2 * i].z;
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int v = __shfl_up_sync(~0u, upto, o);
        if (lane >= o) upto += v;
    }
    if (lane == 31) scan[tid >> 5] = upto;
    __syncthreads();
    int total = 0;
    for (int i = 0; i < kWarps; ++i) {
        if (i == (tid >> 5)) upto += total;
        total += scan[i];
    }
    for (int j = blockIdx.x; j < total; j += gridDim.x) {
        if (j >= upto - mine && j < upto) {
            int at = upto - mine;
            for (int i = c0; i < c1; ++i) {
                const int n = a.meta[2 * i].x < 0 ? 0 : a.meta[2 * i].z;
                if (j < at + n) {
                    job[0] = i, job[1] = j - at;
                    break;
                }
                at += n;
            }
        }
        __syncthreads();
        const int first = job[0], r = job[1];
        const int4 m0 = a.meta[2 * first], m1 = a.meta[2 * first + 1];
        const int n = m0.x - first + 1;
        // part i: slot m0.y of the first CTA, slot 0 of those after it
        auto part = [&](int i) {
            return a.part + (2 * (int64_t)(first + i) + (i ? 0 : m0.y)) * part_floats(rb, D);
        };
        float top = -INFINITY;
        for (int i = tid; i < n; i += kThreads) top = fmaxf(top, part(i)[rb * D + r]);
#pragma unroll
        for (int o = 16; o; o /= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
        if (lane == 0) wt[tid >> 5] = top;
        __syncthreads();
        for (int i = 0; i < kWarps; ++i) top = fmaxf(top, wt[i]);
        const float base = top == -INFINITY ? 0.f : top;
        float y = 0.f, sum = 0.f;
#pragma unroll 8
        for (int i = run; i < n; i += kJoinRuns) {
            const float *p = part(i);
            const float f = exp2_of(p[rb * D + r] - base);
            sum = fmaf(f, p[rb * D + rb + r], sum);
            y = fmaf(f, p[r * D + e], y);
        }
        acc[run][e] = y;
        if (e == 0) sums[run] = sum;
        __syncthreads();
        if (run == 0) {
            sum = (sums[0] + sums[1]) + (sums[2] + sums[3]);
            y = (acc[0][e] + acc[1][e]) + (acc[2][e] + acc[3][e]);
            const int tok = (m1.y + r) / a.per, hq = (m1.y + r) % a.per;
            a.out[((int64_t)(m1.x + tok) * a.q_heads + m0.w * a.per + hq) * D + e] =
                sum == 0.f ? 0.f : __fdiv_rn(y, sum);
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------------ launch
// CTAs of a launch, groups and slots of each.
struct AttnShape {
    int ctas, ng, nslot;
};

// Once per kernel and device: all of an SM's shared memory may be asked for.
// (Two threads may both do it.)
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

// The kernel and, after it, the join.
template <int D, auto KERNEL, class ARGS>
cudaError_t launch_pair(const ARGS &a, int sms, int ctas, int threads,
                        int smem, int rb, cudaStream_t s) {
    // rows that may have parts to join: all there are, at most
    const int64_t jobs = (int64_t)a.q.nseq * a.q.heads * a.q.max_new * a.per;
    cudaError_t e = allow_shared<KERNEL>(227 * 1024);
    if (e != cudaSuccess) return e;
    KERNEL<<<ctas, threads, smem, s>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(jobs < 2 * sms ? jobs : 2 * sms));
    cfg.blockDim = dim3(kJoinRuns * D);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kq_attn_join<D>, static_cast<const AttnArgs &>(a), rb, ctas);
}

template <int FMT, int D, int NT>
cudaError_t launch_attn(AttnArgs a, int sms, cudaStream_t s, int64_t *floats) {
    using M = AttnSmem<FMT, D, NT>;
    // The groups of an SM stand in one CTA that joins them where there are few
    // items, else in two to four CTAs, so that fewer wait for another at an
    // item's end.  One / apart, 8-bit, 32 / 8 heads: 256 items 152 / 158 us (of
    // 16384 tokens at most), 512 items 33.0 / 22.3 (200), 1024 items 140 / 95.9
    // (2000).  Four / three / two CTAs: 8-bit 109 / 95.9 / 105 us (4, 6, 6
    // groups), 4-bit 96.3 / 102 / 102 (8, 6, 8), f16 - / 77.0 / 75.2 (1024 items
    // of 1000, 3 and 4 groups).  (The rule counts items and not their pages: where
    // CTAs apart hold fewer groups in all, as with 8 bits and width 128, 6 for
    // 7, many long items lose some.)
    const int64_t items = (int64_t)a.q.nseq * a.q.heads *
                          (((int64_t)a.q.max_new * a.per + M::kRows - 1) / M::kRows);
    AttnShape sh;
    auto fit = [&](int ctas) {  // CTAs of an SM
        const int room = M::kSm / ctas - 1024 - M::kCommon - M::kQ;
        sh.ctas = ctas * sms;
        sh.ng = M::groups(ctas);
        sh.nslot = (room / sh.ng - M::kP - M::kMax) / M::kHalf;
    };
    fit(items < 3 * (int64_t)sms ? 1 : M::apart());
    if (sh.nslot > kMaxSlots) sh.nslot = kMaxSlots;
    *floats = 2 * (int64_t)sh.ctas * part_floats(M::kRows, D);
    if (!a.part) return cudaSuccess;
    a.ng = sh.ng, a.nslot = sh.nslot;
    a.meta = reinterpret_cast<int4 *>(a.part);  // meta first, 16-byte aligned
    a.part += 8 * (int64_t)sh.ctas;
    return launch_pair<D, kq_attn_kernel<FMT, D, NT>>(a, sms, sh.ctas, 32 * M::kWg * sh.ng + 32,
                                                      M::total(sh.ng, sh.nslot), M::kRows, s);
}

// The launch for a format and width: tiles of four rows by the rows that a
// key head has.
template <int FMT, int D>
cudaError_t attn_tiles(int64_t rows, const AttnArgs &a, int sms, cudaStream_t s, int64_t *floats) {
    // Up to four tiles to a block, blocks alike.  (Width 256 has no other
    // kernel for more rows; a block of 32 spilled, 83 us against 59 for 8
    // sequences of 4100 tokens with 20 rows a key head.)
    const int64_t tiles = (rows + 3) / 4, blocks = (tiles + 3) / 4;
    switch ((int)((tiles + blocks - 1) / blocks)) {
    case 1: return launch_attn<FMT, D, 1>(a, sms, s, floats);
    case 2: return launch_attn<FMT, D, 2>(a, sms, s, floats);
    case 3: return launch_attn<FMT, D, 3>(a, sms, s, floats);
    default: return launch_attn<FMT, D, 4>(a, sms, s, floats);
    }
}

template <int FMT>
cudaError_t attn_format(int dim, const AttnArgs &a, int sms, cudaStream_t s, int64_t *floats) {
    const int64_t rows = (int64_t)a.q.max_new * a.per;
    switch (dim) {
    case 64: return attn_tiles<FMT, 64>(rows, a, sms, s, floats);
    case 128: return attn_tiles<FMT, 128>(rows, a, sms, s, floats);
    default: return attn_tiles<FMT, 256>(rows, a, sms, s, floats);
    }
}

}  // namespace kqd
