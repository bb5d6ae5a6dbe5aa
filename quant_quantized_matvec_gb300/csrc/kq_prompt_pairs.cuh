// kq_prompt_pairs.cuh -- attention of whole prompts in 16 bits, widths 64 and
// 128.  Formula, items and what is not finite are those of kq_prompt_attn.cuh;
// an item has 256 rows here, two blocks of 128 over the same keys, and a CTA goes
// through several items.
//
// Both blocks' queries stay in shared memory; S, P and O are in tensor memory,
// each by itself: a tile's S is formed while the softmax warps (a row a thread)
// are at the tile before it, as soon as they have taken that one into registers,
// and O += P V adds up behind them.  Each block has a warp that issues its
// products, so neither block waits for the other.  O is only corrected when a
// row's maximum has grown by 2^8 or more over its reference: until then
// probabilities are held up to 2^8 times as large, in the sum too, and the
// quotient is the same.  The warps that hold the row do it themselves, as it is
// rare after the first tiles.  P is rounded to the type, as the product's two
// operands have one: held in two terms as in f32, O would take twice the products.
//
// 12001 tokens, 32 / 8 heads of 128, bf16: 808 us, 1460 TFLOP/s, 76% of what a
// large bf16 matrix product reaches, at the chip's power limit.  A tile of both
// blocks takes about 1800 clocks, of which the tensor core is at work for 1470
// (with 80 keys S reads more of shared memory, 52 clocks a step of 16 where the
// product takes 40).  Shorter prompts: an item begins and ends with 2 to 3 us in
// which the tensor core waits (first copies, first softmax, rows out).
#pragma once

#include "kq_prompt_attn.cuh"

namespace kqp {

// (width 128: 80 keys 870 us, 64 975, in the case above at the time; more do not
// fit beside P.  S and P of 128 keys in one place, so that S waits for the O
// before it: 937 us.)
constexpr int pair_tile(int d) { return d == 64 ? 128 : 80; }

template <class T, int D>
struct Pairs {
    static constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    // Keys of a tile: what tensor memory holds of S, P and O for two blocks.
    static constexpr int TK = pair_tile(D);
    static constexpr int kQTile = kRows * D * 2, kTile = TK * D * 2;
    static constexpr int kControl = 2048;
    static constexpr int kRing = kControl + 2 * kQTile;
    static constexpr int kOut = 8 * 2048;  // 32 rows of 64 bytes a softmax warp
    static constexpr int kRoom = (227 * 1024 - 1024 - kRing - kOut) / kTile;
    static constexpr int kSlots = kRoom < 8 ? kRoom : 8;
    static constexpr int kStage = kRing + kSlots * kTile;
    static constexpr int kBytes = kStage + kOut + 1024;
    // columns of tensor memory of a block: O, S, P
    static constexpr int kO = 0, kS = D, kP = D + TK, kBlock = 256;
    // P of f16 times 2^7: with the 2^8 below the correction it stays below 2^16
    static constexpr float kUp = kBf16 ? 0.f : 7.f;
    static_assert(kP + TK / 2 <= kBlock && kSlots >= 5 && TK % 16 == 0, "layout");
};
// Warps: 8 of softmax; two that issue products, one for copies, one that finds
// units; four that clean values.  (Two softmax warps for the same rows, half a
// tile's columns each: 898 us against 859.  Four more warps that write results:
// 870 against 855, as all others have fewer registers then.)
constexpr int kPairThreads = 512, kPairOther = 8, kPairClean = 12;
// Registers after the split: 256 * 200 + 256 * 56, the 512 * 128 at launch.
constexpr int kPairSoftRegs = 200, kPairOtherRegs = 56;
constexpr int kPairLaunchRegs = 65536 / kPairThreads;
static_assert(256 * kPairSoftRegs + 256 * kPairOtherRegs <= kPairThreads * kPairLaunchRegs &&
                  kPairSoftRegs > kPairLaunchRegs && kPairOtherRegs < kPairLaunchRegs,
              "setmaxnreg: the shares, and the way each goes");

// A unit: a part of an item's keys, with what each block sees of it.
struct Unit {
    Item item;      // of both blocks: up to 2 * tok tokens
    int32_t t0, t1; // tiles, last first
    int32_t edges;  // of them, from the last, that some row sees in part
    int32_t n[2];   // tiles of each block, the last n of the walk
    int32_t u;      // its number
};

constexpr int kUnits = 3;  // that are being worked on: a third is found while two are

struct PairShared {
    uint4 answer;  // of ask_for_cta
    Unit unit[kUnits];
    uint64_t ufull[kUnits], ufree[kUnits], qfull[2], qfree[2], full[8], empty[8], sdone[2], sfree[2], pready[2],
        odone[2], vraw[4], vclean[4], given, begun, drain[2];
    uint32_t tmem;
    int dead, bad[kUnits];
    int asked, claimed;  // after an expired wait: an answer to come; a unit that no role has seen
};
static_assert(sizeof(PairShared) <= 2048, "layout");

// Unit `u` into shared memory, by one warp; false past the last.
__device__ __forceinline__ bool find_unit(const PromptArgs &a, int u, int tile, Unit &g, int lane, Place &p) {
    const bool found = find_item<1>(a, u / a.splits, g.item, lane, p);
    const Item &it = g.item;
    if (found && lane == 0) {
        const int rank = u % a.splits, half = a.tok / 2;
        const int tiles = (it.keys() + tile - 1) / tile;
        g.t0 = (int)((int64_t)tiles * rank / a.splits);
        g.t1 = (int)((int64_t)tiles * (rank + 1) / a.splits);
        const int whole = max(0, it.limit(it.tok0) + 1) / tile;
        g.edges = min(max(g.t1 - max(whole, g.t0), 0), g.t1 - g.t0);
        // the first block's tokens end earlier (it may have all of them)
        const int first = min(half, it.nt);
        const int keys = max(0, min(it.m, it.limit(it.tok0 + first - 1) + 1));
        g.n[1] = it.nt > half ? g.t1 - g.t0 : 0;
        g.n[0] = max(0, min(g.t1, (keys + tile - 1) / tile) - g.t0);
        g.u = u;
    }
    __syncwarp();
    return found;
}

template <class T, int D>
__global__ void __launch_bounds__(kPairThreads, 1)
    kq_prompt_pairs(const __grid_constant__ PromptArgs a) {
    using M = Pairs<T, D>;
    constexpr int TK = M::TK;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024 - (kq::smem_addr(smem_raw) & 1023)) & 1023);
    PairShared &cm = *reinterpret_cast<PairShared *>(smem);
    const uint32_t base = kq::smem_addr(smem);
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    auto bar = [&](const uint64_t &b) { return kq::smem_addr(&b); };

    if (w == 0) {  // a lane a barrier, or a few
        const int i = lane;
        if (i < 2) {
            kq::mbar_init(bar(cm.qfull[i]), 1);
            kq::mbar_init(bar(cm.qfree[i]), 1);
            kq::mbar_init(bar(cm.sdone[i]), 1);
            kq::mbar_init(bar(cm.sfree[i]), 4);
            kq::mbar_init(bar(cm.pready[i]), 4);
            kq::mbar_init(bar(cm.odone[i]), 1);
            kq::mbar_init(bar(cm.drain[i]), 1);
        } else if (i < 10) {
            kq::mbar_init(bar(cm.full[i - 2]), 1), kq::mbar_init(bar(cm.empty[i - 2]), 2);
        } else if (i < 14) {
            kq::mbar_init(bar(cm.vraw[i - 10]), 1), kq::mbar_init(bar(cm.vclean[i - 10]), 4);
        } else if (i < 14 + kUnits) {
            kq::mbar_init(bar(cm.ufree[i - 14]), 8 + 3 + 4);
        } else if (i == 31) {
            kq::mbar_init(bar(cm.given), 1), kq::mbar_init(bar(cm.begun), 1);
            for (int j = 0; j < kUnits; ++j) kq::mbar_init(bar(cm.ufull[j]), 1);
            cm.dead = 0, cm.asked = 0, cm.claimed = -1;
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    } else if (w == kPairOther) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                         kq::smem_addr(&cm.tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    } else if (w == kPairOther + 2 && lane < 3) {
        const CUtensorMap *map = lane == 0 ? &a.qmap : lane == 1 ? &a.kmap : &a.vmap;
        asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
    }
    // the first unit: the CTA's number
    Place place;
    if (w == kPairOther + 3) {
        if (lane < kUnits) cm.bad[lane] = 0, cm.unit[lane].u = -1;
        __syncwarp();
        const bool found = find_unit(a, blockIdx.x, TK, cm.unit[0], lane, place);
        if (!found && lane == 0) cm.unit[0].u = -1;
    }
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = cm.tmem;

    auto dead = [&]() { return *(volatile int *)&cm.dead != 0; };
    auto wait = [&](const uint64_t &b, int phase) {  // the completion of the barrier's phase
        if (kq::mbar_test(bar(b), phase & 1) || dead()) return;
        if (!kq::mbar_wait_awake(bar(b), phase & 1, a.wait_ns, a.suspend_ns)) {
            *(volatile int *)&cm.dead = 1;
            atomicOr(a.err, 1u);
        }
    };
    // The same by a whole warp: false after an expired wait of any (which is only
    // looked for where the barrier is not there yet).
    auto arrived = [&](const uint64_t &b, int phase) {
        if (__all_sync(~0u, kq::mbar_test(bar(b), phase & 1))) return true;
        wait(b, phase);
        return !__any_sync(~0u, dead());
    };
    // The next unit as a role reads it; false at the end.  (After an expired
    // wait there is none.)  Its place is handed back once all have read it, and
    // the softmax warps are done with it.
    auto next = [&](int k, Unit &g) {
        const int at = k % kUnits;
        wait(cm.ufull[at], k / kUnits);
        if (__any_sync(~0u, dead())) return false;
        g = cm.unit[at];
        __syncwarp();
        if (lane == 0) kq::mbar_arrive(bar(cm.ufree[at]));
        return g.u >= 0;
    };
    // Copies of tiles, of values that are cleaned, and of blocks' queries, that
    // were begun.  (Values that are cleaned have barriers of their own: who
    // waits for some tiles only could be two phases ahead of a slot's, and take
    // the phase before for it.)
    int copied = 0, raw = 0, queries[2] = {0, 0};

    if (w < kPairOther) {
        // ------------------------------------------------- softmax warps
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPairSoftRegs));
        const int block = w >> 2, r = 32 * (w & 3) + lane;
        const uint32_t mine = tmem + M::kBlock * block + ((uint32_t)(32 * (w & 3)) << 16);
        const uint32_t sa = mine + M::kS, pa = mine + M::kP, oa = mine + M::kO;
        const float sc = fmaxf(fabsf(a.scale) * kLog2E, 1.4e-45f);  // (not 0: -infinity * 0)
        const int half = a.tok / 2, t = r / a.hb, hq = r - t * a.hb;
        int turn = 0;  // tiles of all units
        for (int k = 0;; ++k) {
            const int slot = k % kUnits;
            wait(cm.ufull[slot], k / kUnits);
            if (__any_sync(~0u, dead())) break;
            const Unit &g = cm.unit[slot];  // (ours until it is handed back)
            if (g.u < 0) break;
            const Item &it = g.item;
            const int tok = it.tok0 + block * half + t;
            const bool on = t < half && tok < it.tok0 + it.nt && hq < it.nh;
            const int limit = on ? it.limit(tok) : -1;
            const int count = g.n[block], top = g.t0 + count;  // tiles t0..top-1, last first
            const int whole = g.t1 - g.edges;                  // tiles below are seen by all rows
            float m = -INFINITY, l = 0.f;
            for (int i = 0; i < count; ++i) {
                if (!arrived(cm.sdone[block], turn + i)) break;
                tc_after();
                uint32_t d[TK];
#pragma unroll
                for (int j = 0; j + 32 <= TK; j += 32) tc_load32(d + j, sa + j);
                if constexpr (TK % 32 != 0) tc_load16(d + TK - 16, sa + TK - 16);
                tc_loaded();
                tc_before();
                __syncwarp();
                if (lane == 0) kq::mbar_arrive(bar(cm.sfree[block]));
                const int at = top - 1 - i;
                if (at >= whole) {
                    const int seen = limit + 1 - at * TK;
#pragma unroll
                    for (int j = 0; j < TK; ++j)
                        if (j >= seen) d[j] = 0xFF800000u;
                }
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int j = 0; j < TK; ++j) mx[j & 3] = fmaxf(mx[j & 3], __uint_as_float(d[j]));
                const float now = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), m);
                // (-infinity before the first key that the row attends)
                const bool grown = now > m && !((now - m) * sc <= kLazy);
                if (__any_sync(~0u, grown)) {
                    const float f = !grown ? 1.f : m == -INFINITY ? 0.f : exp2_fast((m - now) * sc);
                    if (grown) m = now;
                    l *= f;
                    if (i > 0) {
                        if (!arrived(cm.odone[block], turn + i - 1)) break;
                        tc_after();
#pragma unroll
                        for (int j = 0; j < D; j += 16) {
                            uint32_t o[16];
                            tc_load16(o, oa + j);
                            tc_loaded();
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tc_store16(oa + j, o);
                        }
                    }
                }
                // p = 2^(s sc - m sc + up).  With a product m sc past 2^10 its
                // rounding would show: that row's difference is taken first.
                // (Lanes without a row hold anything, and have no say in it.)
                float c = m == -INFINITY ? M::kUp : M::kUp - m * sc;
                const bool far = on && !(fabsf(c) < 1024.f);
                if (__any_sync(~0u, far)) {
                    const float from = far ? m : 0.f;
#pragma unroll
                    for (int j = 0; j < TK; ++j) d[j] = __float_as_uint(__uint_as_float(d[j]) - from);
                    if (far) c = M::kUp;
                }
                float2 sum0 = make_float2(0.f, 0.f), sum1 = sum0;
                uint32_t p[TK / 2];
#pragma unroll
                for (int j = 0; j < TK / 2; ++j) {
                    const float2 x = fma2(make_float2(__uint_as_float(d[2 * j]), __uint_as_float(d[2 * j + 1])),
                                          make_float2(sc, sc), make_float2(c, c));
                    const float2 y = make_float2(exp2_fast(x.x), exp2_fast(x.y));
                    if (j & 1) sum1 = add2(sum1, y);
                    else sum0 = add2(sum0, y);
                    p[j] = pack2<T>(y.x, y.y);
                }
                sum0 = add2(sum0, sum1);
                l += sum0.x + sum0.y;
                // ---- P, once the O before it has read its place
                if (i > 0) {
                    if (!arrived(cm.odone[block], turn + i - 1)) break;
                    tc_after();
                }
#pragma unroll
                for (int j = 0; j + 32 <= TK / 2; j += 32) tc_store32(pa + j, p + j);
                if constexpr (TK / 2 % 32 != 0) tc_store8(pa + TK / 2 - 8, p + TK / 2 - 8);
                tc_stored();
                tc_before();
                __syncwarp();
                if (lane == 0) kq::mbar_arrive(bar(cm.pready[block]));
            }
            turn += count;
            if (__any_sync(~0u, dead())) break;
            // ---- the rows' results
            if (count) wait(cm.odone[block], turn - 1);
            if (__any_sync(~0u, dead())) break;
            tc_after();
            const int row = block * kRows + r;
            const float inv = limit < 0 ? 0.f : __fdiv_rn(1.f, l);
            const bool bad = *(volatile int *)&cm.bad[slot] != 0;
            // the block's first row, the lane's from there, and which lanes have one
            T *to = static_cast<T *>(a.out) +
                    ((int64_t)(it.first + it.tok0 + block * half) * a.q_heads + it.hq) * D;
            const uint32_t place = t * a.q_heads + hq, rows = __ballot_sync(~0u, on);
            float *part = a.part + (int64_t)g.u * (2 * kRows) * (D + 2);
            // Rows go out 64 bytes by four lanes, through shared memory (a lane's
            // own 32 bytes of its row: 215 against 207 us for nine prompts).
            uint8_t *stage = smem + M::kStage + w * 2048;
#pragma unroll 1
            for (int j = 0; j < D; j += 32) {
                uint32_t o[32];
                if (count) {
                    tc_load32(o, oa + j);
                    tc_loaded();
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0;
                }
                if (bad && on) {
                    // values that are not finite, of the tiles that left them out
                    for (int y = whole * TK; y < min(g.t1 * TK, limit + 1); ++y) {
                        const T *v = static_cast<const T *>(a.v) + (int64_t)(it.kfirst + y) * a.v_stride +
                                     (int64_t)it.head * D + j;
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const float x = to_f32<T>(v[e]);
                            if (!(fabsf(x) < INFINITY)) o[e] = __float_as_uint(__uint_as_float(o[e]) + x);
                        }
                    }
                }
                __syncwarp();
                if (a.splits > 1) {
                    // by values, of 32 rows each: part[32 rows][D][32]
                    uint32_t *by = reinterpret_cast<uint32_t *>(part) + (row - lane) * D + 32 * j + lane;
#pragma unroll
                    for (int e = 0; e < 32; ++e) by[32 * e] = o[e];
                    continue;
                }
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t q[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        q[e] = pack2<T>(__uint_as_float(o[8 * c + 2 * e]) * inv,
                                        __uint_as_float(o[8 * c + 2 * e + 1]) * inv);
                    *reinterpret_cast<uint4 *>(stage + lane * 64 + ((c ^ (lane >> 1 & 3)) << 4)) =
                        make_uint4(q[0], q[1], q[2], q[3]);
                }
                __syncwarp();
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    const int at = 8 * z + (lane >> 2), c = lane & 3;
                    const uint4 x = *reinterpret_cast<const uint4 *>(stage + at * 64 + ((c ^ (at >> 1 & 3)) << 4));
                    const uint32_t far = __shfl_sync(~0u, place, at);
                    if (rows >> at & 1) *reinterpret_cast<uint4 *>(to + (int64_t)far * D + j + 8 * c) = x;
                }
                __syncwarp();
            }
            if (a.splits > 1) part[2 * kRows * D + row] = m, part[2 * kRows * (D + 1) + row] = l;
            tc_before();
            __syncwarp();
            if (lane == 0) kq::mbar_arrive(bar(cm.ufree[slot]));
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPairOtherRegs));
        if (w == kPairOther + 3) {
            // ----------------------------------------- the units, one ahead
            // A CTA begins with the unit of its number, and then takes over those
            // of CTAs that have not begun, as a rule in their order (which no
            // result goes by): a sequence's longest first.  (Dealt out evenly
            // beforehand, in rounds there and back: 234 against 224 us for nine
            // prompts of up to 2049 tokens.)
            int u = blockIdx.x, asks = 0;
            bool lost = false;
            auto given = [&]() {  // another CTA's number; -1: none, or (lost) not in time
                if (lane == 0) {
                    kq::mbar_expect_tx(bar(cm.given), 16);
                    ask_for_cta(kq::smem_addr(&cm.answer), bar(cm.given));
                }
                __syncwarp();
                wait(cm.given, asks++);
                if (__any_sync(~0u, dead())) {
                    if (lane == 0) cm.asked = asks;
                    lost = true;
                    return -1;
                }
                const int x = cta_given(kq::smem_addr(&cm.answer));
                __syncwarp();
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                return x;
            };
            for (int k = 0;; ++k) {
                const int slot = k % kUnits;
                if (k >= kUnits) wait(cm.ufree[slot], k / kUnits - 1);
                if (__any_sync(~0u, dead())) {
                    if (lane == 0) cm.claimed = u;
                    break;
                }
                Unit &g = cm.unit[slot];
                auto find = [&](int x) { return find_unit(a, x, TK, g, lane, place); };
                if (u >= 0 && !(k == 0 ? g.u >= 0 : find(u))) {
                    if (lane == 0) g.u = -1;
                    u = first_found(given, find);
                    if (lost) break;
                }
                if (lane == 0) {
                    if (u < 0) g.u = -1;
                    *(volatile int *)&cm.bad[slot] = 0;
                    __threadfence_block();
                    kq::mbar_arrive(bar(cm.ufull[slot]));
                }
                __syncwarp();
                if (u < 0) break;
                // The next one is taken when the last few copies for this one are
                // made: not before, as others may be free earlier.
                wait(cm.begun, k);
                u = given();
                if (lost) break;
            }
        } else if (w == kPairOther + 2) {
            // --------------------------------------------- copies
            Unit g;
            for (int k = 0; next(k, g); ++k) {
                const Item &it = g.item;
                const int count = g.t1 - g.t0;
                if (lane == 0) {
                    const uint32_t bytes = (uint32_t)(a.tok / 2) * a.hb * 128;
                    // The queries' place is free when the last S of the unit before
                    // has been formed: a few tiles are copied before that.
                    const int when = k == 0 ? 0 : min(3, 2 * count - 1);
                    if (count == 0) kq::mbar_arrive(bar(cm.begun));
                    for (int n = 0; n < 2 * count; ++n) {
                        // (asking and finding take two microseconds, about two tiles)
                        if (n == max(0, 2 * count - 8)) kq::mbar_arrive(bar(cm.begun));
                        for (int b = 0; b < 2 && n == when; ++b) {
                            if (g.n[b] == 0) continue;
                            if (queries[b]) wait(cm.qfree[b], queries[b] - 1);
                            if (dead()) break;
                            kq::mbar_expect_tx(bar(cm.qfull[b]), bytes * (D / 64));
                            for (int c = 0; c < D / 64; ++c)
                                tensor3d_g2s(base + M::kControl + b * M::kQTile + c * (kRows * 128), &a.qmap, 64 * c,
                                             it.hq, it.first + it.tok0 + b * (a.tok / 2), bar(cm.qfull[b]));
                            ++queries[b];
                        }
                        const int s = copied % M::kSlots;
                        if (copied >= M::kSlots) wait(cm.empty[s], copied / M::kSlots - 1);
                        if (dead()) break;
                        uint32_t done = bar(cm.full[s]);
                        if ((n & 1) && (n >> 1) < g.edges) {
                            kq::mbar_arrive(done);
                            done = bar(cm.vraw[raw++ & 3]);
                        }
                        kq::mbar_expect_tx(done, M::kTile);
                        ++copied;
#pragma unroll
                        for (int c = 0; c < D / 64; ++c)
                            tensor2d_g2s(base + M::kRing + s * M::kTile + c * (TK * 128), n & 1 ? &a.vmap : &a.kmap,
                                         it.head * D + 64 * c, it.kfirst + (g.t1 - 1 - (n >> 1)) * TK,
                                         done);
                    }
                }
                __syncwarp();
            }
        } else if (w < kPairOther + 2) {
            // ------------------------------------- products of a block
            const int b = w - kPairOther;
            const uint32_t tm = uniform(tmem + M::kBlock * b);
            const uint64_t qd = desc_k(uniform(base + M::kControl + b * M::kQTile));
            const uint32_t is = mma_idesc(TK, M::kBf16, false) | (a.scale < 0.f ? 1u << 13 : 0u);
            constexpr uint32_t io = mma_idesc(D, M::kBf16, true);
            int tile = 0, cleaned = 0;  // tiles of both blocks so far, and those that were cleaned
            int turn = 0, have = 0;     // tiles of this block; units with some
            Unit g;
            for (int k = 0; next(k, g); ++k) {
                const int count = g.t1 - g.t0, n = g.n[b], from = count - n;
                // Copy x of the walk (keys, values by turns) is there; and is
                // given back: once the products so far are done, or at once.
                auto there = [&](int x) { return arrived(cm.full[x % M::kSlots], x / M::kSlots); };
                bool stop = false;
                for (int i = 0; i < from; ++i) {  // tiles that only the other block sees
                    for (int x = 2 * (tile + i); x < 2 * (tile + i) + 2; ++x) {
                        // (not for values to be cleaned: a slot is only copied to
                        // again when its values four tiles ago are done with)
                        stop = !there(x);
                        if (stop) break;
                        if (lane == 0) kq::mbar_arrive(bar(cm.empty[x % M::kSlots]));
                        __syncwarp();
                    }
                    if (stop) break;
                }
                if (stop) break;
                if (n > 0 && !arrived(cm.qfull[b], have++)) break;
                auto scores = [&](int i) {
                    const int x = 2 * (tile + i);
                    if (!there(x)) return false;
                    if (i > from && !arrived(cm.sfree[b], turn + i - from - 1)) return false;
                    tc_after();
                    const uint32_t s = uniform(x % M::kSlots);
                    const uint64_t kd = desc_k(uniform(base + M::kRing) + s * M::kTile);
                    if (elected()) {
#pragma unroll
                        for (int j = 0; j < D / 16; ++j) {
                            const uint64_t qj = qd + (((j >> 2) * (kRows * 128) + (j & 3) * 32) >> 4);
                            const uint64_t kj = kd + (((j >> 2) * (TK * 128) + (j & 3) * 32) >> 4);
                            if (j) tc_add_ss(tm + M::kS, qj, kj, is);
                            else tc_mma_ss(tm + M::kS, qj, kj, is, false);
                        }
                        tc_commit(bar(cm.sdone[b]));
                        tc_commit(bar(cm.empty[0]) + 8 * s);
                        if (i == count - 1) tc_commit(bar(cm.qfree[b]));
                    }
                    __syncwarp();
                    return true;
                };
                if (n > 0 && !scores(from)) break;
                for (int i = from; i < count; ++i) {
                    if (i + 1 < count && !scores(i + 1)) {
                        stop = true;
                        break;
                    }
                    const int x = 2 * (tile + i) + 1;
                    const int e = cleaned + i;
                    stop = !there(x) || (i < g.edges && !arrived(cm.vclean[e & 3], e >> 2)) ||
                           !arrived(cm.pready[b], turn + i - from);
                    if (stop) break;
                    tc_after();
                    const uint32_t s = uniform(x % M::kSlots), more = uniform(i > from);
                    const uint64_t vd = desc_n(uniform(base + M::kRing) + s * M::kTile, TK * 128);
                    if (elected()) {
                        tc_mma_ts(tm + M::kO, tm + M::kP, vd, io, more);
#pragma unroll
                        for (int j = 1; j < TK / 16; ++j)
                            tc_add_ts(tm + M::kO, tm + M::kP + 8 * j, vd + j * (2048 >> 4), io);
                        tc_commit(bar(cm.odone[b]));
                        tc_commit(bar(cm.empty[0]) + 8 * s);
                    }
                    __syncwarp();
                }
                if (stop) break;
                tile += count;
                cleaned += g.edges;
                turn += n;
            }
        } else if (w >= kPairClean) {
            // ------------- values that are not finite, of tiles seen in part
            int tile = 0, cleaned = 0;
            Unit g;
            for (int k = 0; next(k, g); ++k) {
                for (int i = 0; i < g.edges; ++i, ++cleaned) {
                    const int s = (2 * (tile + i) + 1) % M::kSlots;  // (values are the odd copies)
                    wait(cm.vraw[cleaned & 3], cleaned >> 2);
                    if (__any_sync(~0u, dead())) break;
                    uint4 *v = reinterpret_cast<uint4 *>(smem + M::kRing + s * M::kTile) +
                               (w - kPairClean) * (M::kTile / 64) + lane;
                    bool odd = false;
#pragma unroll 5
                    for (int c = 0; c < M::kTile / 64; c += 32) {
                        uint4 x = v[c];
                        if (not_finite<T>(x.x) | not_finite<T>(x.y) | not_finite<T>(x.z) | not_finite<T>(x.w)) {
                            odd = true;
                            uint32_t *e = &x.x;
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const uint32_t f = not_finite<T>(e[j]);
                                if (f & 0x8000u) e[j] &= 0xFFFF0000u;
                                if (f & 0x80000000u) e[j] &= 0x0000FFFFu;
                            }
                            v[c] = x;
                        }
                    }
                    if (odd) *(volatile int *)&cm.bad[k % kUnits] = 1;
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) kq::mbar_arrive(bar(cm.vclean[cleaned & 3]));
                }
                tile += g.t1 - g.t0;
            }
        }
        __syncwarp();
    }
    __syncwarp();
    tc_before();
    __syncthreads();
    // After an expired wait no copy and no product may run on past this; what
    // the CTA had to write is NaN.
    if (dead()) {
        if (w == kPairOther + 2 && lane == 0) {
            for (int n = max(0, copied - M::kSlots); n < copied; ++n)
                kq::mbar_wait(bar(cm.full[n % M::kSlots]), (n / M::kSlots) & 1, kq::kWaitLimitNs);
            for (int n = max(0, raw - 4); n < raw; ++n)
                kq::mbar_wait(bar(cm.vraw[n & 3]), (n >> 2) & 1, kq::kWaitLimitNs);
            for (int b = 0; b < 2; ++b)
                if (queries[b]) kq::mbar_wait(bar(cm.qfull[b]), (queries[b] - 1) & 1, kq::kWaitLimitNs);
        }
        if (w == kPairOther || w == kPairOther + 1) {
            const uint64_t &drain = cm.drain[w - kPairOther];
            tc_after();
            if (elected()) tc_commit(bar(drain));
            __syncwarp();
            kq::mbar_wait(bar(drain), 0, kq::kWaitLimitNs);
            __syncwarp();
        }
        if (w == kPairOther + 3 && lane == 0 && cm.asked) {
            if (kq::mbar_wait(bar(cm.given), (cm.asked - 1) & 1, kq::kWaitLimitNs))
                cm.claimed = cta_given(kq::smem_addr(&cm.answer));
        }
        for (int k = 0; k <= kUnits; ++k) {  // the units that roles were at, and one that none has seen
            __syncthreads();
            if (k == kUnits) {
                const int u = cm.claimed;
                __syncthreads();
                Place p;
                if (w == 0 && (u < 0 || !find_unit(a, u, TK, cm.unit[0], lane, p)) && lane == 0)
                    cm.unit[0].u = -1;
                __syncthreads();
            }
            const Unit &g = cm.unit[k % kUnits];
            if (g.u < 0) continue;
            const Item &it = g.item;
            if (a.splits > 1) {
                float *part = a.part + (int64_t)g.u * (2 * kRows) * (D + 2);
                for (int i = tid; i < 2 * kRows; i += kPairThreads)
                    part[2 * kRows * D + i] = -INFINITY, part[2 * kRows * (D + 1) + i] = quiet_nan();
                continue;
            }
            const int across = it.nh * (D / 8);
            for (int i = tid; i < it.nt * across; i += kPairThreads) {
                const int tok = it.tok0 + i / across, e = i % across;
                const uint32_t n = pack2<T>(quiet_nan(), quiet_nan());
                *reinterpret_cast<uint4 *>(static_cast<T *>(a.out) +
                                           ((int64_t)(it.first + tok) * a.q_heads + it.hq) * D + 8 * e) =
                    make_uint4(n, n, n, n);
            }
        }
        __syncthreads();
    }
    if (w == kPairOther) {
        tc_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    }
}

template <class T, int D>
cudaError_t launch_pairs(PromptArgs &a, cudaStream_t s) {
    using M = Pairs<T, D>;
    cudaError_t e = allow_shared<kq_prompt_pairs<T, D>>(M::kBytes);
    if (e == cudaSuccess && a.nkeys > 0) {
        e = keys_map<T>(a.k, a.k_stride, a, D, M::TK, &a.kmap);
        if (e == cudaSuccess) e = keys_map<T>(a.v, a.v_stride, a, D, M::TK, &a.vmap);
    }
    if (e != cudaSuccess) return e;
    e = queries_map<T>(a, D, a.tok / 2, &a.qmap);  // (a block's)
    if (e != cudaSuccess) return e;
    kq_prompt_pairs<T, D><<<(unsigned)(a.items * a.splits), kPairThreads, M::kBytes, s>>>(a);
    return cudaGetLastError();
}

}  // namespace kqp
