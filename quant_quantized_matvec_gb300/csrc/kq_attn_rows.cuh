// kq_attn_rows.cuh -- attention where a key head has many rows (drafted
// tokens times the query heads that share it): the products on the
// fifth-generation tensor cores.  Formula, work division and partial results
// are those of kq_attn.cuh; a tile is one page.
//
// The rows are the 128 lanes of an accumulator.  Queries and probabilities
// are the first operand, in tensor memory, as two f16 terms hi + lo; keys and
// values the second, in shared memory, a quantised page converted once for
// all rows by a group of warps:
//   S [row][token]  = Qhi K + Qlo K        (f16 cache)
//                   = Qhi Khi + Qhi Klo + Qlo Khi
//   O [row][value]  = Phi V + Plo V,  Phi Vhi + Phi Vlo + Plo Vhi
// where a quantised cache's code * scale is formed as two f16 terms, exactly
// (scales after a power of two a page; what is dropped is below 2^-22).  A
// thread of the four softmax warps has a row: no reduction across lanes.
// Each page's O starts at zero and is added to the row's f32 sums in
// registers, with the correction of the running reference, the row's maximum
// less 15.  Queries are multiplied by the fraction of the scale as they are
// brought in (one f32 rounding), so that scores are multiplied by powers of
// two alone, exactly: fma(score, factor, -reference) is at most 15 whatever the
// size of both.  (A rounded product, the maximum taken off and the result
// multiplied by 2^15: 480 us against 418 in the 8-bit case below.)
//
// Blocks of up to 32 rows stand in all four quarters of the lanes, and the
// four warps take pages by turns, each with its own maxima and sums (32..64
// rows: two pairs of warps); they are joined at the end of an item's pages.
//
// A page goes through: producer warp (copies of the raw page) -> conversion
// warps -> S -> softmax warps -> P -> O -> softmax warps; each stage has two
// buffers or more but O, so that S of the next pages is formed while a page's
// probabilities are, and its O while the next page's are.  An f16 page is not
// converted: tensor copies lay its rows of 64 bytes out as the MMAs take them,
// and only the values of pages with new tokens, or that end, are gone over in
// place (converted by a copy within shared memory: 365 us against 276 for 4
// sequences of 131071 at most, 8 drafts, 32 / 8 heads).
//
// The softmax warps' code is kept short (loops over half a page, scores read
// twice from tensor memory), and the number of sets is fixed per instance:
// four roles run side by side, and with the page unrolled, or the sets counted
// at run time, the warps waited for instructions (32 sequences of 16384 at
// most, 4 drafts, 64 / 8 heads, 8-bit: 427 us, 509 with sets at run time).
//
// Bound by: the MMAs of a page, 3 * 8 * 32 + 3 * 4 * 64 = 1536 clocks for a
// quantised page of width 128 (1024 for f16) whatever the rows up to 128, and
// the shared memory that they and the conversion read and write (195 KB a
// page, 1520 clocks; f16 96 KB); f16 with 32 rows by memory: 84% of the copy
// rate in the case above.
#pragma once

#include <cuda.h>

#include <type_traits>

#include "kq_attn.cuh"
#include "kq_host.h"

namespace kqd {

constexpr int kRowSlots = 8;    // most raw slots
constexpr int kConvWarps = 16;
constexpr int kConvThreads = 32 * kConvWarps;
constexpr int kFirstOther = 4 + kConvWarps;  // first warp of the last four: S, copies, O
constexpr int kRowsThreads = 32 * (kFirstOther + 4);
// Registers of a thread after the split: softmax, conversion, the others.
// 128 threads * 216 + 512 * 56 + 128 * 32 = 60416 of the 768 * 80 at launch.
constexpr int kSoftRegs = 216, kConvRegs = 56, kOtherRegs = 32;

struct RowsCommon {
    RunShared run;
    uint64_t rawfull[kRowSlots], rawempty[kRowSlots], scaled[kRowSlots];
    uint64_t kready[2], kfree[2], vready[4], vfree[2], edge[4];
    // sdone: by tile & 3.  (A phase's parity tells it from the next only, so no
    // barrier may complete twice before its waiter has looked, nor be waited for
    // two phases ahead: S of tile t + 4 needs the buffer of tile t, or of a later
    // one, back.)
    uint64_t sfree[4], sdone[4], pready[4], pvdone[4], ofree, drain[2];
    uint32_t tmem;
    int dead, drained[2];
    int badpage[8];          // of tile t & 7: the page is not valid
    uint32_t badtok[4][2];   // values of these tokens are not finite (edge pages)
    float kf[8], vf[8];      // powers of two of the page's scales
    uint32_t up[kRowSlots];  // their inverse, as f16 pairs, by raw slot
    float m[128], l[128];
};

template <int FMT, int D>
struct RowsSmem {
    using L = Kv<FMT, D>;
    static constexpr int kTile = kPage * D * 2;         // one f16 tile
    static constexpr int kBuf = L::kQuant ? 2 * kTile : 0;  // hi and lo (f16: the raw slots)
    static constexpr int kTiles0 = 4096;                        // after RowsCommon
    static constexpr int kRaw = kTiles0 + 4 * kBuf;             // K 0, K 1, V 0, V 1
    static constexpr int kHalf = L::kV;
    static constexpr int kRoom = (227 * 1024 - 2048 - kRaw) / kHalf;
    static constexpr int kSlots = kRoom < kRowSlots ? kRoom : kRowSlots;
    static constexpr int kTotal = kRaw + kSlots * kHalf + 1024;  // (1024: alignment)
    // columns of tensor memory
    static constexpr int kQ = 0, kP = D, kO = D + 64, kS = 2 * D + 64;
    static constexpr int kSBufs = D == 64 ? 4 : 3;
    static_assert(sizeof(RowsCommon) <= kTiles0 && kSlots >= 3 && kS + 64 * kSBufs <= 512, "layout");
    static_assert(128 * (D + 4) * 4 <= 4 * kBuf + kSlots * kHalf, "the join's rows");
};

// ------------------------------------------------------ tcgen05 operations
__device__ __forceinline__ void tc_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// One lane of a converged warp, and a value that all its lanes share, so that
// the MMAs' descriptors stay in uniform registers (issued from a branch of lane
// 0, an MMA took about 90 clocks).
__device__ __forceinline__ bool elected() {
    uint32_t is;
    asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}\n" : "=r"(is));
    return is != 0;
}
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(~0u, x, 0); }
__device__ __forceinline__ void tc_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
                 : "memory");
}
// D (+)= A B, f16, f32 sums; A in tensor memory, B in shared memory.
template <bool ADD>
__device__ __forceinline__ void tc_mma(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "n"(ADD ? 1 : 0)
        : "memory");
}
// 32 columns of the warp's lanes, a column a register.
__device__ __forceinline__ void tc_load32(uint32_t (&r)[32], uint32_t addr) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
        "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
          "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
          "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tc_store16(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15,%16};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tc_stored() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// A tile of rows of 128 bytes, 16-byte chunks swizzled over 8 rows (K-major).
__device__ __forceinline__ uint64_t tile_desc(uint32_t addr) {
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// f16 operands, f32 sums, 128 x n.
__host__ __device__ constexpr uint32_t tile_idesc(int n) {
    return 1u << 4 | (uint32_t)(n >> 3) << 17 | (128u >> 4) << 24;
}
__device__ __forceinline__ uint32_t tile_at(int row, int chunk) {
    return row * 128 + ((chunk ^ (row & 7)) << 4);
}
// The same with rows of 64 bytes, as an f16 page is copied.
__device__ __forceinline__ uint64_t raw_desc(uint32_t addr) {
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)1 << 16 | (uint64_t)(512 >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)4 << 61;
}
__device__ __forceinline__ uint32_t raw_at(int row, int chunk) {
    return row * 64 + ((chunk ^ (row >> 1 & 3)) << 4);
}
// Box of half a block (keys or values), rows `y` on of block z.
__device__ __forceinline__ void tensor3d_g2s(uint32_t dst, const CUtensorMap *map, int y, int z,
                                             uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cta.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(map), "r"(0), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

// The cache as rows of 64 bytes, for f16.
struct RowsArgs : AttnArgs {
    CUtensorMap map;
};

// Element pair h (0..3) of an octet as the converted tiles hold it.
template <int FMT>
__device__ __forceinline__ constexpr int oct_a(int h) {
    return FMT == KQ_KV_Q4 ? h : 2 * h;
}
template <int FMT>
__device__ __forceinline__ constexpr int oct_b(int h) {
    return FMT == KQ_KV_Q4 ? h + 4 : 2 * h + 1;
}

// Eight codes as they lie in a quantised cache, and as f16 pairs.
template <int FMT>
struct Octet {
    using T = typename std::conditional<FMT == KQ_KV_Q8, uint2, uint32_t>::type;
};
template <int FMT>
__device__ __forceinline__ void octet_codes(typename Octet<FMT>::T v, uint32_t (&c)[4]) {
    if constexpr (FMT == KQ_KV_Q8) {
        codes8(v.x, c[0], c[1]);
        codes8(v.y, c[2], c[3]);
    } else {
        codes4(v, c);
    }
}

// o + p v for a stored value v that is not finite, else o (rare: not inlined).
template <int FMT, int D>
__device__ __noinline__ float add_not_finite(const uint8_t *block, int tok, int e, float p, float o) {
    using L = Kv<FMT, D>;
    float x;
    const uint32_t v =
        *reinterpret_cast<const uint32_t *>(block + L::v_word(e, tok / L::kVPerWord));
    const int bit = tok % L::kVPerWord * L::kBits;
    if constexpr (L::kQuant)
        x = (float)((int)(v << (32 - L::kBits - bit)) >> (32 - L::kBits)) *
            __half2float(*reinterpret_cast<const __half *>(block + L::v_scale(tok, e / kGroup)));
    else
        x = __half2float(__ushort_as_half((uint16_t)(v >> bit)));
    return fabsf(x) <= 3.4e38f ? o : fmaf(p, x, o);
}

// (QW: warps of a set, rows of a block / 32)
template <int FMT, int D, int QW>
__global__ void __launch_bounds__(kRowsThreads, 1)
    kq_attn_rows_kernel(const __grid_constant__ RowsArgs a) {
    using L = Kv<FMT, D>;
    using M = RowsSmem<FMT, D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024 - (kq::smem_addr(smem_raw) & 1023)) & 1023);
    RowsCommon &cm = *reinterpret_cast<RowsCommon *>(smem);
    const uint32_t base = kq::smem_addr(smem);
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    constexpr int qw = QW, rb = 32 * QW;            // rows of a block
    constexpr int ns = 4 / QW;                      // sets
    constexpr int nsl = ns == 4 ? 2 : ns == 2 ? 1 : 0;  // log2
    // Sets take turns, so that a page's O is formed while others form P.  A
    // single set has two buffers of P for that, one of them a buffer of S
    // (8-bit, 128 rows: 45.8 us against 51.1 for a tree of 16 over 32001 tokens;
    // with two sets 158.8 against 153.5 for 16 sequences of 16384 at most, 64
    // rows; not for f16, whose edge pages are gone over only after the O before
    // them).
    constexpr bool kTwoP = L::kQuant && ns == 1;
    constexpr int kSB = kTwoP ? 2 : M::kSBufs;
    auto pcol = [](int t) { return kTwoP && (t >> nsl & 1) ? M::kS + 128 : M::kP; };
    auto bar = [&](const uint64_t &b) { return kq::smem_addr(&b); };

    if (tid == 0) {
        for (int i = 0; i < kRowSlots; ++i) {
            kq::mbar_init(bar(cm.rawfull[i]), 1);
            kq::mbar_init(bar(cm.rawempty[i]), L::kQuant ? kConvWarps : 1);
            kq::mbar_init(bar(cm.scaled[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            kq::mbar_init(bar(cm.kready[i]), kConvWarps);
            kq::mbar_init(bar(cm.kfree[i]), 1);
            kq::mbar_init(bar(cm.vfree[i]), 1);
        }
        for (int i = 0; i < 4; ++i) {
            kq::mbar_init(bar(cm.sfree[i]), qw);
            kq::mbar_init(bar(cm.sdone[i]), 1);
            kq::mbar_init(bar(cm.edge[i]), 1);
            kq::mbar_init(bar(cm.vready[i]), kConvWarps);
            kq::mbar_init(bar(cm.pvdone[i]), 1);
            kq::mbar_init(bar(cm.pready[i]), qw);
            cm.badtok[i][0] = cm.badtok[i][1] = 0;
        }
        kq::mbar_init(bar(cm.ofree), qw);
        kq::mbar_init(bar(cm.drain[0]), 1);
        kq::mbar_init(bar(cm.drain[1]), 1);
        cm.dead = cm.drained[0] = cm.drained[1] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    kq::allow_dependents();
    const Run run = run_of(a, rb, kRowsThreads, cm.run);
    if (run.u0 >= run.u1) return;
    if (w == kFirstOther) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                         kq::smem_addr(&cm.tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = cm.tmem;

    auto dead = [&]() { return *(volatile int *)&cm.dead != 0; };
    auto wait = [&](const uint64_t &b, int phase) {  // the completion of the barrier's phase
        if (kq::mbar_test(bar(b), phase & 1) || dead()) return;
        if (!kq::mbar_wait_for(bar(b), phase & 1, a.wait_ns, a.suspend_ns)) {
            *(volatile int *)&cm.dead = 1;
            atomicOr(a.err, 1u);
        }
    };

    // The CTA's segments, as every role walks them: tile t0 is the first of
    // the segment, counted since the launch.
    struct Seg {
        Seq s;
        int b, pages, pg0, npg, head, row0, nrows;
        long long u;
        int t0;
        int pe, e0;  // first edge page, and edge tiles before the segment's
    };
    auto segments = [&](auto &&body) {
        int b = run.seq, t0 = 0, e0 = 0;
        long long off = run.off;
        for (long long u = run.u0; u < run.u1 && b < a.q.nseq;) {
            int blocks;
            Seg g;
            g.s = seq_of(a.q, b);
            const long long units = units_of(a, g.s, rb, blocks);
            if (off >= units) {
                ++b, off = 0;
                continue;
            }
            g.b = b, g.u = u, g.t0 = t0;
            g.pages = (int)pages_of(a.q, g.s);
            const int item = (int)(off / g.pages);
            g.pg0 = (int)(off - (long long)item * g.pages);
            g.npg = (int)min((long long)(g.pages - g.pg0), run.u1 - u);
            g.head = item / blocks, g.row0 = (item - g.head * blocks) * rb;
            g.nrows = min(rb, g.s.n * a.per - g.row0);
            g.pe = max(g.pg0, g.s.ctx / kPage), g.e0 = e0;
            body(g);
            e0 += max(0, g.pg0 + g.npg - g.pe);
            u += g.npg, off += g.npg, t0 += g.npg;
        }
    };
    // The number of tile t's turn at the barriers of its converted values
    // (f16: edge pages only have one; two a segment at most).
    auto turn_of = [](const Seg &g, int t) {
        return L::kQuant ? t : g.e0 + (g.pg0 + (t - g.t0) - g.pe);
    };
    // The end of a segment, for all threads: the softmax warps have left
    // their rows in shared memory (the tiles are idle now).
    float *rows = reinterpret_cast<float *>(smem + M::kTiles0);
    auto finish = [&](const Seg &g) {
        __syncthreads();
        const bool whole = g.npg == g.pages;
        const int slot = g.u == run.u0 ? 0 : 1;
        float *part = a.part + (2 * (int64_t)blockIdx.x + slot) * part_floats(rb, D);
        for (int i = tid; i < g.nrows * (D / 4); i += kRowsThreads) {
            const int r = i / (D / 4), e = 4 * (i % (D / 4));
            float top = -INFINITY;
            for (int k = 0; k < ns; ++k) top = fmaxf(top, cm.m[k * rb + r]);
            const float from = top == -INFINITY ? 0.f : top;
            float sum = 0.f;
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int k = 0; k < ns; ++k) {
                const float f = exp2_of(cm.m[k * rb + r] - from);
                sum = fmaf(f, cm.l[k * rb + r], sum);
                const float4 v =
                    *reinterpret_cast<const float4 *>(rows + (k * rb + r) * (D + 4) + e);
                y.x = fmaf(f, v.x, y.x), y.y = fmaf(f, v.y, y.y);
                y.z = fmaf(f, v.z, y.z), y.w = fmaf(f, v.w, y.w);
            }
            if (dead()) sum = quiet_nan();
            if (whole) {
                const float inv = sum == 0.f ? 0.f : __fdiv_rn(1.f, sum);
                const int tok = (g.row0 + r) / a.per, hq = (g.row0 + r) % a.per;
                *reinterpret_cast<float4 *>(
                    a.out + ((int64_t)(g.s.first + tok) * a.q_heads + g.head * a.per + hq) * D + e) =
                    make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv);
            } else {
                *reinterpret_cast<float4 *>(part + r * D + e) = y;
                if (e == 0) part[rb * D + r] = top, part[rb * D + rb + r] = sum;
            }
        }
        if (tid == 0 && !whole && g.pg0 == 0) {
            a.meta[2 * blockIdx.x] =
                make_int4(last_cta(run, g.u, g.pages), slot, g.nrows, g.head);
            a.meta[2 * blockIdx.x + 1] = make_int4(g.s.first, g.row0, 0, 0);
        }
        // what was written comes before the next copies and MMAs there
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncthreads();
    };

    if (w < 4) {
        // ------------------------------------------------- softmax warps
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
        const int set = w / qw;
        const uint32_t mine = tmem + ((uint32_t)(32 * w) << 16);
        segments([&](const Seg &g) {
            const int r = (w % qw) * 32 + lane;
            const bool on = r < g.nrows;
            const int tok = on ? (g.row0 + r) / a.per : 0, hq = on ? (g.row0 + r) % a.per : 0;
            // ---- the row's query: its power of two, then both terms
            const float4 *x = reinterpret_cast<const float4 *>(
                a.x + (int64_t)(g.s.first + tok) * a.x_stride + (int64_t)(g.head * a.per + hq) * D);
            float4 v[D / 4];  // all loads in flight at once
#pragma unroll
            for (int i = 0; i < D / 4; ++i) v[i] = on ? __ldg(x + i) : make_float4(0.f, 0.f, 0.f, 0.f);
            float top = 0.f;
#pragma unroll
            for (int i = 0; i < D / 4; ++i)
                top = fmaxf(top, fmaxf(fmaxf(fabsf(v[i].x), fabsf(v[i].y)),
                                       fmaxf(fabsf(v[i].z), fabsf(v[i].w))));
            const int ex = max((int)((__float_as_uint(top) >> 23) & 255) - 126, -111);
            // The query is multiplied by the fraction of the scale (which has its
            // sign) as well, so that the factor of the scores is a power of two
            // and their product with it exact.
            const float up = a.scale_m * __uint_as_float((uint32_t)(127 + 15 - ex) << 23);
            const float rowf =
                __uint_as_float((uint32_t)(127 + factor_exponent(ex, a.scale_e)) << 23);
            const uint64_t nw = (!on      ? 0
                                 : a.mask ? __ldg(a.mask + g.s.first + tok)
                                          : ~0ull >> (63 - tok)) &
                                (~0ull >> (64 - g.s.n));
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int o = 0; o < 4; ++o) {
                    const float4 v0 = v[8 * i + 2 * o], v1 = v[8 * i + 2 * o + 1];
                    const float e[8] = {v0.x * up, v0.y * up, v0.z * up, v0.w * up,
                                        v1.x * up, v1.y * up, v1.z * up, v1.w * up};
#pragma unroll
                    for (int h = 0; h < 4; ++h)
                        split(e[oct_a<FMT>(h)], e[oct_b<FMT>(h)], hi[4 * o + h], lo[4 * o + h]);
                }
                tc_store16(mine + M::kQ + 16 * i, hi);
                tc_store16(mine + M::kQ + D / 2 + 16 * i, lo);
            }
            tc_stored();
            tc_before();
            __syncthreads();

            float O[D], m = -INFINITY, l = 0.f;
#pragma unroll
            for (int i = 0; i < D; ++i) O[i] = 0.f;
            // O of tile t, whose page moved the maximum by `alpha`
            auto take = [&](int t, float alpha) {
                const float f = L::kQuant ? *(volatile float *)&cm.vf[t & 7] : 1.f;
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    uint32_t d[32];
                    tc_load32(d, mine + M::kO + 32 * i);
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        O[32 * i + k] = fmaf(__uint_as_float(d[k]), f, O[32 * i + k] * alpha);
                }
                tc_before();
                __syncwarp();
                if (lane == 0) kq::mbar_arrive(bar(cm.ofree));
            };
            int before = -1;       // a tile whose O is still to come
            float factor = 1.f;    // and its alpha
            auto flush = [&]() {
                if (before < 0) return;
                wait(cm.pvdone[before & 3], before >> 2);
                tc_after();
                take(before, factor);
                before = -1;
            };
            auto page = [&](int t, auto is_edge) {
                constexpr bool kEdge = decltype(is_edge)::value;
                const int pg = g.pg0 + (t - g.t0);
                uint64_t ok = ~0ull;
                if constexpr (kEdge) {
                    const int left = g.s.ctx - pg * kPage;
                    ok = left <= 0 ? (-left < 64 ? nw >> -left : 0) : (nw << left) | ~(~0ull << left);
                }
                // ---- S, maxima, probabilities times 2^15
                const int sb = t % kSB;
                wait(cm.sdone[t & 3], t >> 2);
                tc_after();
                float f = rowf * (L::kQuant ? *(volatile float *)&cm.kf[t & 7] : 1.f);
                if (*(volatile int *)&cm.badpage[t & 7]) f = quiet_nan();
                const uint32_t sa = mine + M::kS + 64 * sb;
                // the half page's scores, those not attended as -infinity
                auto scores = [&](int half, uint32_t (&d)[32]) {
                    tc_load32(d, sa + 32 * half);
                    if constexpr (kEdge) {
                        const uint32_t in = (uint32_t)(ok >> (32 * half));
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (!((in >> i) & 1)) d[i] = 0xFF800000u;
                    }
                };
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    uint32_t d[32];
                    scores(half, d);
#pragma unroll
                    for (int i = 0; i < 32; ++i) mx[i & 3] = fmaxf(mx[i & 3], __uint_as_float(d[i]));
                }
                mx[0] = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                // Probabilities are held times 2^15.  The row's reference is its
                // maximum less 15, rounded up, and all that follows goes by the
                // reference: however large the logits are, and the steps in which
                // f32 holds them, none passes 2^15.
                const float now =
                    fmaxf(m, mx[0] == -INFINITY ? mx[0] : __fsub_ru(mx[0] * f, 15.f));
                const float from = now == -INFINITY ? 0.f : now;
                const float alpha = exp2_of(m - from);
                m = now;
                // Values that are not finite: the conversion left them out, and
                // the rows that attend them take them below.  (Read before P
                // goes out, after which the buffer's next page may come.)
                uint64_t bad = 0;
                auto look = [&]() {
                    if constexpr (kEdge) {
                        const int n = turn_of(g, t);
                        wait(cm.vready[n & 3], n >> 2);
                        bad = (uint64_t)*(volatile uint32_t *)&cm.badtok[n & 3][0] |
                              (uint64_t)*(volatile uint32_t *)&cm.badtok[n & 3][1] << 32;
                    }
                };
                if constexpr (L::kQuant) look();
                // ---- O of the page before, which also frees P
                if constexpr (!kTwoP) flush();
                // (f16: with two sets the O warp gets to this page only now)
                if constexpr (!L::kQuant) look();
                // ---- P
                float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    uint32_t d[32];
                    scores(half, d);
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        float p = exp2_of(fmaf(__uint_as_float(d[i]), f, -from));
                        if constexpr (kEdge)  // (f may be a NaN)
                            if (!((uint32_t)(ok >> (32 * half)) >> i & 1)) p = 0.f;
                        sum[i & 3] += p;
                        d[i] = __float_as_uint(p);
                    }
                    uint32_t hi[16], lo[16];
#pragma unroll
                    for (int o = 0; o < 4; ++o)
#pragma unroll
                        for (int h = 0; h < 4; ++h)
                            split(__uint_as_float(d[8 * o + oct_a<FMT>(h)]),
                                  __uint_as_float(d[8 * o + oct_b<FMT>(h)]), hi[4 * o + h],
                                  lo[4 * o + h]);
                    tc_store16(mine + pcol(t) + 16 * half, hi);
                    tc_store16(mine + pcol(t) + 32 + 16 * half, lo);
                }
                l = fmaf(l, alpha, (sum[0] + sum[1]) + (sum[2] + sum[3]));
                if constexpr (kTwoP) {
                    tc_stored();
                    tc_before();
                    __syncwarp();
                    if (lane == 0) {
                        if constexpr (!kEdge) kq::mbar_arrive(bar(cm.sfree[sb]));
                        kq::mbar_arrive(bar(cm.pready[t & 3]));
                    }
                    flush();
                }
                before = t, factor = alpha;
                if constexpr (kEdge) {
                    if (bad && !dead()) {
                        const int64_t pgi = page_of(a.q, g.b, pg);
                        if (pgi >= 0) {
                            const uint8_t *block = a.q.data + (pgi * a.q.heads + g.head) * L::kBlock;
#pragma unroll
                            for (int i = 0; i < D; ++i) O[i] *= factor;
                            factor = 1.f;
                            while (bad) {
                                const int at = __ffsll((long long)bad) - 1;
                                bad &= bad - 1;
                                uint32_t d[32];
                                scores(at >> 5, d);
                                float p = 0.f;
#pragma unroll
                                for (int i = 0; i < 32; ++i) p = i == (at & 31) ? __uint_as_float(d[i]) : p;
                                p = exp2_of(fmaf(p, f, -from));
                                if ((ok >> at) & 1) {
#pragma unroll
                                    for (int i = 0; i < D; ++i)
                                        O[i] = add_not_finite<FMT, D>(block, at, i, p, O[i]);
                                }
                                __syncwarp();
                            }
                        }
                        __syncwarp();
                    }
                }
                tc_stored();
                tc_before();
                __syncwarp();
                if (lane == 0 && (!kTwoP || kEdge)) {
                    kq::mbar_arrive(bar(cm.sfree[sb]));
                    if constexpr (!kTwoP) kq::mbar_arrive(bar(cm.pready[t & 3]));
                }
            };
            for (int t = g.t0 + ((set - g.t0) & (ns - 1)); t < g.t0 + g.npg; t += ns) {
                if (g.s.ctx - (g.pg0 + (t - g.t0)) * kPage < kPage) page(t, std::true_type());
                else page(t, std::false_type());
                // (with four sets the next S waits for this O's turn)
                if (ns == 4) flush();
            }
            flush();
            cm.m[32 * w + lane] = m;
            cm.l[32 * w + lane] = l;
            float4 *to = reinterpret_cast<float4 *>(rows + (32 * w + lane) * (D + 4));
            __syncthreads();  // every MMA and copy of the segment is done
#pragma unroll
            for (int i = 0; i < D / 4; ++i)
                to[i] = make_float4(O[4 * i], O[4 * i + 1], O[4 * i + 2], O[4 * i + 3]);
            finish(g);
        });
    } else if (w < 4 + kConvWarps) {
        // ---------------------------------------------- conversion warps
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kConvRegs));
        const int ct = tid - 128;
        int use = 0, turn = 0;
        auto put = [&](uint8_t *tile, uint32_t at, const uint32_t (&c)[4], const __half2 (&sc)[4]) {
            uint4 hi, lo;
            uint32_t *h = &hi.x, *o = &lo.x;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __half2 x = __hmul2(half2_of(c[i]), sc[i]);
                h[i] = bits_of(x);
                o[i] = bits_of(__hfma2(half2_of(c[i]), sc[i], __hneg2(x)));
            }
            *reinterpret_cast<uint4 *>(tile + at) = hi;
            *reinterpret_cast<uint4 *>(tile + M::kTile + at) = lo;
        };
        // Which of the 8 tokens from `first` on are in the page but not finite,
        // by the exponents of x; those and the ones past the page's end
        // become zero.
        auto clean = [](uint32_t (&x)[4], int first, int held) {
            uint32_t bad = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t m = 0xFFFFu << (16 * (k & 1));
                const uint32_t inf = 0x7C00u << (16 * (k & 1));
                const bool in = first + k < held;
                const bool nf = (x[k >> 1] & inf) == inf;
                if (in && nf) bad |= 1u << k;
                if (!in || nf) x[k >> 1] &= ~m;
            }
            return bad;
        };
        if constexpr (!L::kQuant) {
            // f16: the raw slots are the MMAs' operands; only an edge page's
            // values are gone over, in place, when the O warp says so
            segments([&](const Seg &g) {
                __syncthreads();
                for (int pg = g.pe; pg < g.pg0 + g.npg; ++pg) {
                    const int t = g.t0 + (pg - g.pg0), n = turn_of(g, t);
                    const int held = g.s.ctx + g.s.n - pg * kPage, slot = 2 * t + 1;
                    wait(cm.edge[n & 3], n >> 2);
                    wait(cm.rawfull[slot % M::kSlots], slot / M::kSlots);
                    uint8_t *vt = smem + M::kRaw + slot % M::kSlots * M::kHalf;
                    if (ct == 0) cm.badtok[(n + 2) & 3][0] = cm.badtok[(n + 2) & 3][1] = 0;
                    for (int at = ct; at < D * 8; at += kConvThreads) {
                        const int e = at >> 3, j = at & 7;  // tokens 8 j ..
                        uint4 *p = reinterpret_cast<uint4 *>(vt + raw_at((j >> 2) * D + e, j & 3));
                        uint4 v = *p;
                        uint32_t x[4] = {v.x, v.y, v.z, v.w};
                        const uint32_t bad = clean(x, 8 * j, held);
                        if (bad) atomicOr(&cm.badtok[n & 3][j >> 2], bad << (8 * (j & 3)));
                        *p = make_uint4(x[0], x[1], x[2], x[3]);
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) kq::mbar_arrive(bar(cm.vready[n & 3]));
                }
                __syncthreads();
                finish(g);
            });
        } else {
            // A page's keys, then its values; with two sets the next page's keys
            // come before them, as the values wait for the O of two pages before
            // and fewer pages are on their way (64 rows, the case above, 8-bit:
            // 158 us against 167; with one set 45.8 against 44.4 for the tree
            // above, with four 460 against 413 for 32 sequences, 4 drafts, 64 / 8
            // heads, though 355 against 376 for 64 of one token, 32 rows, width 64).
            constexpr int kOctets = D / 8;
            constexpr int kN = kPage * kOctets / kConvThreads;  // octets of keys of a thread
            constexpr int kM = D * 8 / kConvThreads;            // and of values
            constexpr int ahead = ns == 2;
            segments([&](const Seg &g) {
                __syncthreads();
                for (int k = -ahead; k < g.npg; ++k) {
                    const int t = g.t0 + k, pg = g.pg0 + k, tk = t + ahead;
                    const bool vals = k >= 0, keys = k + ahead < g.npg;
                    const int left = g.s.ctx - pg * kPage;
                    const bool edge = left < kPage;
                    const int held = left + g.s.n;  // tokens of the page that exist
                    // their raw slots: `use` and the one after it
                    const bool second = use + 1 == M::kSlots;
                    const int other = second ? 0 : use + 1;
                    const bool kfirst = !ahead || !vals;
                    const int ks = kfirst ? use : other, vs = ahead ? use : other;
                    const int kturn = kfirst ? turn : turn + second;
                    const int vturn = ahead ? turn : turn + second;
                    typename Octet<FMT>::T raws[kN], vraw[kM];
                    __half sc1[kN];
                    uint4 svs[kM];
                    __half2 kup, vup;
                    if (keys) {
                        wait(cm.scaled[ks], kturn);
                        wait(cm.rawfull[ks], kturn);
                        const uint8_t *raw = smem + M::kRaw + ks * M::kHalf;
                        kup = half2_of(*(volatile uint32_t *)&cm.up[ks]);
#pragma unroll
                        for (int i = 0; i < kN; ++i) {
                            const int at = ct + kConvThreads * i, row = at / kOctets, o = at % kOctets;
                            raws[i] =
                                *reinterpret_cast<const typename Octet<FMT>::T *>(raw + L::k_octet(row, o));
                            sc1[i] = *reinterpret_cast<const __half *>(raw + L::k_scale(row, o >> 2));
                        }
                        if (tk >= 2) wait(cm.kfree[tk & 1], (tk >> 1) - 1);
                        uint8_t *kt = smem + M::kTiles0 + (tk & 1) * M::kBuf;
#pragma unroll
                        for (int i = 0; i < kN; ++i) {
                            // 8 lanes make one 128-byte row of the tile
                            const int at = ct + kConvThreads * i, row = at / kOctets, o = at % kOctets;
                            uint8_t *half = kt + (o >> 3) * (kPage * 128);
                            const uint32_t to = tile_at(row, o & 7);
                            uint32_t c[4];
                            octet_codes<FMT>(raws[i], c);
                            const __half2 s2 = __hmul2(__half2half2(sc1[i]), kup);
                            const __half2 sc[4] = {s2, s2, s2, s2};
                            put(half, to, c, sc);
                        }
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        __syncwarp();
                        if (lane == 0) {
                            kq::mbar_arrive(bar(cm.rawempty[ks]));
                            kq::mbar_arrive(bar(cm.kready[tk & 1]));
                        }
                    }
                    if (vals) {
                        wait(cm.scaled[vs], vturn);
                        wait(cm.rawfull[vs], vturn);
                        if (t >= 2) wait(cm.vfree[t & 1], (t >> 1) - 1);
                        const uint8_t *raw = smem + M::kRaw + vs * M::kHalf - L::kV;
                        vup = half2_of(*(volatile uint32_t *)&cm.up[vs]);
#pragma unroll
                        for (int i = 0; i < kM; ++i) {
                            const int at = ct + kConvThreads * i, e = at >> 3, j = at & 7;  // tokens 8 j ..
                            vraw[i] = *reinterpret_cast<const typename Octet<FMT>::T *>(
                                raw + L::v_word(e, 8 * j / L::kVPerWord));
                            svs[i] =
                                *reinterpret_cast<const uint4 *>(raw + L::v_scale(8 * j, e / kGroup));
                        }
                        if (ct == 0) cm.badtok[(t + 2) & 3][0] = cm.badtok[(t + 2) & 3][1] = 0;
                        uint8_t *vt = smem + M::kTiles0 + (2 + (t & 1)) * M::kBuf;
#pragma unroll
                        for (int i = 0; i < kM; ++i) {
                            const int at = ct + kConvThreads * i, e = at >> 3, j = at & 7;
                            const uint32_t to = tile_at(e, j);
                            if (edge) {
                                uint32_t x[4] = {svs[i].x, svs[i].y, svs[i].z, svs[i].w};
                                const uint32_t bad = clean(x, 8 * j, held);
                                if (bad) atomicOr(&cm.badtok[t & 3][j >> 2], bad << (8 * (j & 3)));
                                svs[i] = make_uint4(x[0], x[1], x[2], x[3]);
                            }
                            uint32_t c[4];
                            octet_codes<FMT>(vraw[i], c);
                            __half2 sc[4] = {half2_of(svs[i].x), half2_of(svs[i].y), half2_of(svs[i].z),
                                             half2_of(svs[i].w)};
                            if constexpr (FMT == KQ_KV_Q4) {
                                const __half2 s01 = sc[0], s23 = sc[1], s45 = sc[2], s67 = sc[3];
                                sc[0] = __lows2half2(s01, s45), sc[1] = __highs2half2(s01, s45);
                                sc[2] = __lows2half2(s23, s67), sc[3] = __highs2half2(s23, s67);
                            }
#pragma unroll
                            for (int k2 = 0; k2 < 4; ++k2) sc[k2] = __hmul2(sc[k2], vup);
                            put(vt, to, c, sc);
                        }
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        __syncwarp();
                        if (lane == 0) {
                            kq::mbar_arrive(bar(cm.rawempty[vs]));
                            kq::mbar_arrive(bar(cm.vready[t & 3]));
                        }
                    }
                    for (int i = vals + keys; i; --i)
                        if (++use == M::kSlots) use = 0, ++turn;
                }
                __syncthreads();
                finish(g);
            });
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        int use = 0, turn = 0;  // (producer) the next raw slot and how often it was filled
        // 2^(8 - ex) for the page's scales, all below 2^ex, and 2^(ex - 8):
        // a code times a scale then stays below 2^15.  (tokens from `held`
        // on and scales that are not finite do not count)
        auto normal = [&](const uint8_t *scales, bool keys, int held, uint32_t &up) {
            constexpr int kEach = kPage * L::kGroups / 32;  // of a lane: 4 or 8
            uint32_t x[kEach / 2];
            if constexpr (kEach == 8) {
                const uint4 v = *reinterpret_cast<const uint4 *>(scales + 16 * lane);
                x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
            } else {
                const uint2 v = *reinterpret_cast<const uint2 *>(scales + 8 * lane);
                x[0] = v.x, x[1] = v.y;
            }
            uint32_t top = 0;  // magnitudes, two at a time
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                uint32_t h = (x[i / 2] >> (16 * (i & 1))) & 0x7FFFu;
                const int at = lane * kEach + i;
                if (held < kPage && (keys ? at / L::kGroups : at % kPage) >= held) h = 0;
                top = max(top, h >= 0x7C00u ? 0u : h);
            }
            top = __reduce_max_sync(~0u, top);
            const int ex = max((int)(top >> 10) - 14, -7);
            const uint32_t b = (uint32_t)(23 - ex) << 10;
            up = b | b << 16;
            return __uint_as_float((uint32_t)(127 + ex - 8) << 23);
        };
        segments([&](const Seg &g) {
            // --------------------------------------------- producer warp
            int issued = 0;
            const bool issuer = w == kFirstOther + 1 && lane == 0;
            int64_t page = -1, next = issuer ? page_of(a.q, g.b, g.pg0) : -1;
            auto pump = [&](int until) {
                for (; issued < until; ++issued) {
                    if (turn > 0) wait(cm.rawempty[use], turn - 1);
                    if (dead()) break;
                    if ((issued & 1) == 0) {  // keys: the next page is looked up ahead
                        page = next;
                        if (issued + 2 < 2 * g.npg)
                            next = page_of(a.q, g.b, g.pg0 + (issued >> 1) + 1);
                    }
                    // (the entry of eight tiles ago has been read: the keys' slot
                    // was given back after an S or an O of a later tile was asked for)
                    if ((issued & 1) == 0)
                        *(volatile int *)&cm.badpage[(g.t0 + (issued >> 1)) & 7] = page < 0;
                    kq::mbar_expect_tx(bar(cm.rawfull[use]), M::kHalf);
                    const int64_t block = max(page, (int64_t)0) * a.q.heads + g.head;
                    const uint32_t to = base + M::kRaw + use * M::kHalf;
                    if constexpr (L::kQuant)
                        kq::bulk_g2s(to, a.q.data + block * L::kBlock + (issued & 1) * M::kHalf,
                                     M::kHalf, bar(cm.rawfull[use]));
                    else
                        tensor3d_g2s(to, &a.map, (issued & 1) * 2 * D, (int)block,
                                     bar(cm.rawfull[use]));
                    if (++use == M::kSlots) use = 0, ++turn;
                }
            };
            if (issuer) pump(min(2 * g.npg, M::kSlots));
            __syncthreads();
            if (issuer) pump(2 * g.npg);
            // ------- scale warp: each raw slot's powers of two, ahead of the
            // conversion (a quantised cache's only)
            if (L::kQuant && w == kFirstOther + 3) {
                for (int k = 0; k < 2 * g.npg; ++k) {
                    const int t = g.t0 + (k >> 1), pg = g.pg0 + (k >> 1);
                    const bool keys = (k & 1) == 0;
                    wait(cm.rawfull[use], turn);
                    // (the entry of four tiles ago has been read: its slot was
                    // given back after that, and there are at most 8)
                    uint32_t up;
                    const float f =
                        normal(smem + M::kRaw + use * M::kHalf + L::kKScale, keys,
                               g.s.ctx + g.s.n - pg * kPage, up);
                    if (lane == 0) {
                        *(volatile uint32_t *)&cm.up[use] = up;
                        *(volatile float *)(keys ? &cm.kf[t & 7] : &cm.vf[t & 7]) = f;
                        kq::mbar_arrive(bar(cm.scaled[use]));
                    }
                    __syncwarp();
                    if (++use == M::kSlots) use = 0, ++turn;
                }
            }
            // -------------------------------------- MMA warps: S, and O
            constexpr int kTerms = L::kQuant ? 3 : 2;  // hi hi, lo hi, hi lo
            const uint32_t tm = uniform(tmem);
            if (w == kFirstOther) {
                tc_after();
                for (int t = g.t0; t < g.t0 + g.npg; ++t) {
                    const int slot = 2 * t;  // f16: the keys' raw slot
                    if constexpr (L::kQuant) wait(cm.kready[t & 1], t >> 1);
                    else wait(cm.rawfull[slot % M::kSlots], slot / M::kSlots);
                    const int sb = t % kSB;
                    if (t >= kSB) wait(cm.sfree[sb], t / kSB - 1);
                    tc_after();
                    if (__any_sync(~0u, dead())) continue;
                    const uint32_t buf = uniform(t & 1);
                    const uint32_t usb = uniform(sb), done = uniform(t & 3);
                    const uint32_t raw = uniform(slot % M::kSlots);
                    const uint64_t kt = L::kQuant ? tile_desc(base + M::kTiles0 + buf * M::kBuf)
                                                  : raw_desc(base + M::kRaw + raw * M::kHalf);
                    const uint32_t d = tm + M::kS + 64 * usb;
                    if (elected()) {
#pragma unroll
                        for (int term = 0; term < kTerms; ++term)
#pragma unroll
                            for (int i = 0; i < D / 16; ++i) {
                                const uint32_t q = tm + M::kQ + (term == 1 ? D / 2 : 0) + 8 * i;
                                const int at = L::kQuant ? (i >> 2) * (kPage * 128) + (i & 3) * 32
                                                         : (i >> 1) * (kPage * 64) + (i & 1) * 32;
                                const uint64_t b = kt + (((term == 2 ? M::kTile : 0) + at) >> 4);
                                if (term + i) tc_mma<true>(d, q, b, tile_idesc(kPage));
                                else tc_mma<false>(d, q, b, tile_idesc(kPage));
                            }
                        tc_commit(L::kQuant ? bar(cm.kfree[0]) + 8 * buf : bar(cm.rawempty[0]) + 8 * raw);
                        tc_commit(bar(cm.sdone[0]) + 8 * done);
                    }
                    __syncwarp();
                }
            } else if (w == kFirstOther + 2) {
                tc_after();
                for (int t = g.t0; t < g.t0 + g.npg; ++t) {
                    const int slot = 2 * t + 1, n = turn_of(g, t);
                    if constexpr (!L::kQuant) wait(cm.rawfull[slot % M::kSlots], slot / M::kSlots);
                    if (!L::kQuant && n >= g.e0 && lane == 0 && !dead())
                        kq::mbar_arrive(bar(cm.edge[n & 3]));
                    if (L::kQuant || n >= g.e0) wait(cm.vready[n & 3], n >> 2);
                    wait(cm.pready[t & 3], t >> 2);
                    if (t > 0) wait(cm.ofree, t - 1);
                    tc_after();
                    if (__any_sync(~0u, dead())) continue;
                    const uint32_t buf = uniform(t & 1);
                    const uint32_t set = uniform(bar(cm.pvdone[t & 3]));
                    const uint32_t pp = uniform(tm + pcol(t));
                    const uint32_t raw = uniform(slot % M::kSlots);
                    const uint64_t vt = L::kQuant ? tile_desc(base + M::kTiles0 + (2 + buf) * M::kBuf)
                                                  : raw_desc(base + M::kRaw + raw * M::kHalf);
                    if (elected()) {
#pragma unroll
                        for (int term = 0; term < kTerms; ++term)
#pragma unroll
                            for (int i = 0; i < kPage / 16; ++i) {
                                const uint32_t p = pp + (term == 1 ? 32 : 0) + 8 * i;
                                const int at = L::kQuant ? i * 32 : (i >> 1) * (D * 64) + (i & 1) * 32;
                                const uint64_t b = vt + (((term == 2 ? M::kTile : 0) + at) >> 4);
                                if (term + i) tc_mma<true>(tm + M::kO, p, b, tile_idesc(D));
                                else tc_mma<false>(tm + M::kO, p, b, tile_idesc(D));
                            }
                        tc_commit(L::kQuant ? bar(cm.vfree[0]) + 8 * buf : bar(cm.rawempty[0]) + 8 * raw);
                        tc_commit(set);
                    }
                    __syncwarp();
                }
            }
            __syncwarp();
            __syncthreads();
            // After an expired wait no copy and no MMA may run on past this.
            // (Not before the barrier: another role's wait may expire when the
            // producer or an MMA warp is done, with work of theirs on its way.)
            if (dead()) {
                if (issuer) {  // each slot's last copy: this turn's before `use`
                    for (int k = 0; k < M::kSlots; ++k) {
                        const int n = k < use ? turn : turn - 1;
                        if (n >= 0) kq::mbar_wait(bar(cm.rawfull[k]), n & 1, kq::kWaitLimitNs);
                    }
                }
                // (once: the segments after this one issue no MMAs)
                const int k = w == kFirstOther ? 0 : 1;
                if ((w == kFirstOther || w == kFirstOther + 2) && !*(volatile int *)&cm.drained[k]) {
                    if (elected()) tc_commit(bar(cm.drain[k]));
                    __syncwarp();
                    kq::mbar_wait(bar(cm.drain[k]), 0, kq::kWaitLimitNs);
                    __syncwarp();
                    if (lane == 0) *(volatile int *)&cm.drained[k] = 1;
                }
                __syncwarp();
            }
            finish(g);
        });
    }
    // (every role has left its last segment through finish())
    tc_before();
    __syncthreads();
    if (w == kFirstOther) {
        tc_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    }
}

template <int FMT, int D, int QW>
cudaError_t launch_block(const AttnArgs &args, int sms, cudaStream_t s, int64_t *floats) {
    using M = RowsSmem<FMT, D>;
    constexpr int rb = 32 * QW;
    RowsArgs a;
    static_cast<AttnArgs &>(a) = args;
    *floats = 2 * (int64_t)sms * part_floats(rb, D);
    if (!a.part) return cudaSuccess;
    a.meta = reinterpret_cast<int4 *>(a.part);
    a.part += 8 * (int64_t)sms;
    if (FMT == KQ_KV_F16) {
        const cudaError_t e = kqhost::rows_map(a.q.data, 4 * D, a.q.npages * a.q.heads, 2 * D, &a.map);
        if (e != cudaSuccess) return e;
    }
    return launch_pair<D, kq_attn_rows_kernel<FMT, D, QW>>(a, sms, sms, kRowsThreads, M::kTotal, rb, s);
}

// Rows of a block: 32, 64 or 128, the least that hold a key head's rows.
template <int FMT, int D>
cudaError_t launch_rows(const AttnArgs &a, int64_t rows, int sms, cudaStream_t s, int64_t *floats) {
    return rows <= 32   ? launch_block<FMT, D, 1>(a, sms, s, floats)
           : rows <= 64 ? launch_block<FMT, D, 2>(a, sms, s, floats)
                        : launch_block<FMT, D, 4>(a, sms, s, floats);
}

}  // namespace kqd
