// kq_decode.cuh -- what the decode-step kernels share: the cache layout of
// kq_decode.h, the sequences of a batch, and rotary pairs.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kq_decode.h"

namespace kqd {

constexpr int kPage = KQ_KV_PAGE;
constexpr int kGroup = 32;  // values that share a scale

// ------------------------------------------------------------ cache layout
// Byte offsets inside the block of one page and head, for D = head_dim.
template <int FMT, int D>
struct Kv {
    static constexpr int kBits = FMT == KQ_KV_F16 ? 16 : FMT == KQ_KV_Q8 ? 8 : 4;
    static constexpr bool kQuant = FMT != KQ_KV_F16;
    static constexpr int kGroups = D / kGroup;  // scale groups of a head
    // keys: groups of a slab, bytes of an octet (8 values), of a token's slab
    static constexpr int kSlabGroups =
        FMT == KQ_KV_F16 ? 1 : FMT == KQ_KV_Q8 ? 2 : (kGroups < 4 ? kGroups : 4);
    static constexpr int kOctet = kBits;
    static constexpr int kSlabBytes = kSlabGroups * 4 * kOctet;
    static constexpr int kSlabs = kGroups / kSlabGroups;
    // values: tokens of a slab, bytes of a value's row in it
    static constexpr int kVTokens = FMT == KQ_KV_F16 ? 32 : 64;
    static constexpr int kVRow = kVTokens * kBits / 8;
    static constexpr int kVSlabs = kPage / kVTokens;

    static constexpr int kCodes = kPage * D * kBits / 8;
    static constexpr int kScales = kQuant ? kPage * kGroups * 2 : 0;
    static constexpr int kKScale = kCodes;
    static constexpr int kV = kCodes + kScales;
    static constexpr int kVScale = kV + kCodes;
    static constexpr int kBlock = 2 * (kCodes + kScales);

    // octet o (values 8 o ..) of token t's key
    __host__ __device__ static constexpr int k_octet(int t, int o) {
        const int slab = o / (4 * kSlabGroups), r = o % (4 * kSlabGroups);
        return slab * kPage * kSlabBytes + t * kSlabBytes +
               ((r & 3) * kSlabGroups + (r >> 2)) * kOctet;
    }
    // 32-bit word w of value e's row in the values' codes; it holds the
    // tokens w * 32 / kBits and on
    static constexpr int kVPerWord = 32 / kBits;
    static constexpr int kVWords = kPage / kVPerWord;  // words of a value, all slabs
    __host__ __device__ static constexpr int v_word(int e, int w) {
        constexpr int per = kVRow / 4;  // words of a row in a slab
        return kV + (w / per) * D * kVRow + e * kVRow + (w % per) * 4;
    }
    __host__ __device__ static constexpr int k_scale(int t, int g) {
        return kKScale + (t * kGroups + g) * 2;
    }
    __host__ __device__ static constexpr int v_scale(int t, int g) {
        return kVScale + (g * kPage + t) * 2;
    }
};

inline int64_t kv_block_bytes(int fmt, int d) {
    const int bits = fmt == KQ_KV_F16 ? 16 : fmt == KQ_KV_Q8 ? 8 : 4;
    return 2 * ((int64_t)kPage * d * bits / 8 + (bits == 16 ? 0 : kPage * (d / kGroup) * 2));
}

// ---------------------------------------------------------------- batches
// kq_kv and kq_batch as the kernels take them.
struct Seqs {
    uint8_t *data;
    int64_t npages;       // pages of the cache
    const int32_t *start, *ctx, *table;
    int64_t max_pages;
    int32_t nseq, max_new, heads;
    int32_t ntok;
};

// Sequence b's first new token, how many it has, and its committed tokens,
// cut to what the arguments allow.
struct Seq {
    int first, n, ctx;
};
__device__ __forceinline__ Seq seq_of(const int32_t *start, const int32_t *ctx, int ntok,
                                      int max_new, int b) {
    int lo = __ldg(start + b), hi = __ldg(start + b + 1);
    lo = min(max(lo, 0), ntok);
    hi = min(max(hi, lo), ntok);
    Seq s;
    s.first = lo;
    s.n = min(hi - lo, max_new);
    // 2^30 keeps places within 32 bits; no page table is that long (2^24
    // pages are 2^30 places)
    s.ctx = ctx ? min(max(__ldg(ctx + b), 0), 1 << 30) : 0;
    return s;
}
__device__ __forceinline__ Seq seq_of(const Seqs &q, int b) {
    return seq_of(q.start, q.ctx, q.ntok, q.max_new, b);
}
// The cache's page of sequence b's pg-th page, or -1.
__device__ __forceinline__ int64_t page_of(const Seqs &q, int b, int64_t pg) {
    if (pg >= q.max_pages) return -1;
    const int64_t p = __ldg(q.table + (int64_t)b * q.max_pages + pg);
    return p >= 0 && p < q.npages ? p : -1;
}

// ----------------------------------------------------------------- rotary
// Both products and the sum rounded, no fused step: the same f32 operations
// wherever a head is rotated.
__device__ __forceinline__ float rot_a(float a, float b, float c, float s) {
    return __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
}
__device__ __forceinline__ float rot_b(float a, float b, float c, float s) {
    return __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
}
__device__ __forceinline__ float quiet_nan() { return __int_as_float(0x7FC00000); }

}  // namespace kqd
