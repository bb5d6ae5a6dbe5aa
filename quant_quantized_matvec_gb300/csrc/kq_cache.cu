// kq_cache.cu -- the quantised key/value cache: written (append), read back
// (read), and closed up after a verification (move).
//
// One CTA per (page of a sequence, head, keys or values), so that every
// byte of a page's keys or values is written by one CTA: a byte of 4-bit
// values holds two tokens, and whole words are read, changed and written
// where a call covers only some of their tokens.
//
// Quantisation: four lanes hold a group of 32 values, eight each; the value of
// largest magnitude comes from two shuffles.
//
// Bound by: memory in principle, 4 bytes a value on the f32 side and bits/8 on
// the other; in fact by the issue of the arithmetic on codes (8-bit write: 70%
// of the issue slots, ALU at 51%) and, for short runs, by latency.  Up to 6001
// tokens of three sequences, 8 heads of 128, keys rotated: 4-bit write 37.2 us
// (floor 18), read 25.8 (18); 8-bit 37.0 and 27.7.  16 sequences of up to 300
// tokens, 8 heads of 64, f16: 7.9 and 5.8 us.  Move, 8-bit, 2 heads of 128, 1
// / 4 / 16 tokens: 2.9 / 4.6 / 12.1 us for one sequence, 3.2 / 5.6 / 12.6 for
// 32: a token's fetches (path, page, word) one behind the other, as one token
// is moved after the other.  With five CTAs an SM and no load ahead the 8-bit
// write took 39.8 us, with six 39.5.
#include "kq_decode.cuh"
#include "kq_decode_launch.h"

namespace kqd {

constexpr int kCacheThreads = 256;

// ------------------------------------------------------------------ codes
// The eight codes of a lane (of four that hold a group), in the low byte of
// each, and the group's scale; every lane of the warp takes part.
struct Codes {
    int c[8];
    __half d;
};
template <int FMT>
__device__ __forceinline__ Codes quantise(const float (&x)[8]) {
    // The magnitudes as integers, a positive one before a negative one of the
    // same size: one maximum gives the largest value with its sign, and
    // whether any is a NaN or an infinity (their bits are the largest).
    uint32_t key = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t b = __float_as_uint(x[i]);
        key = max(key, FMT == KQ_KV_Q8 ? b << 1 : b << 1 | ((b >> 31) ^ 1));
    }
    key = max(key, __shfl_xor_sync(~0u, key, 1));
    key = max(key, __shfl_xor_sync(~0u, key, 2));
    const bool bad = key >= 0xFF000000u;
    const float top = __uint_as_float(key >> 1);
    float d = FMT == KQ_KV_Q8 ? __fdiv_rn(top, 127.f) : (key & 1 ? top : -top) * -0.125f;
    d = fminf(fmaxf(d, -65504.f), 65504.f);
    Codes r;
    r.d = __float2half_rn(bad ? quiet_nan() : d);
    const float df = __half2float(r.d);
    float inv;  // 1 / d to the last place or so; no scale, no codes
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(df));
    inv = bad || df == 0.f ? 0.f : inv;
    const float hi = FMT == KQ_KV_Q8 ? 127.f : 7.f, lo = FMT == KQ_KV_Q8 ? -127.f : -8.f;
    // x / d rounded to nearest, by way of 1 / d: where the product is near a
    // half, the division itself decides.  (0.499 is far from what the product's
    // error needs, below 3e-5 at 127: one value in 500 passes it, so two rounds
    // of a warp in five divide.)  Added to 1.5 * 2^23 a number is
    // rounded to a whole one, which then stands in the low bits.
    constexpr float kWhole = 12582912.f;
    float q[8], worst = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        q[i] = fminf(fmaxf(x[i] * inv, lo), hi);
        worst = fmaxf(worst, fabsf(q[i] - ((q[i] + kWhole) - kWhole)));
    }
    if (worst > 0.499f) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (fabsf(q[i] - ((q[i] + kWhole) - kWhole)) > 0.499f)
                q[i] = fminf(fmaxf(__fdiv_rn(x[i], df), lo), hi);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) r.c[i] = __float_as_int(q[i] + kWhole);
    return r;
}
// The low bytes of four numbers, side by side.
__device__ __forceinline__ uint32_t bytes4(const int *c) {
    return __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
}

__device__ __forceinline__ float4 load4(const float *p) {
    return *reinterpret_cast<const float4 *>(p);
}

// Values on their way from [token][value] to the cache's [value][token], four
// of a token a word (f16: two).
template <int FMT, int D>
struct Stage {
    static constexpr int kWords = FMT == KQ_KV_F16 ? D / 2 : D / 4;
    uint32_t v[kPage][kWords + 1];
};

// Bytes of four words turned: word i of the result has byte i of each.
__device__ __forceinline__ void turn4(uint32_t (&w)[4]) {
    const uint32_t a = __byte_perm(w[0], w[1], 0x5140), b = __byte_perm(w[0], w[1], 0x7362);
    const uint32_t c = __byte_perm(w[2], w[3], 0x5140), d = __byte_perm(w[2], w[3], 0x7362);
    w[0] = __byte_perm(a, c, 0x5410), w[1] = __byte_perm(a, c, 0x7632);
    w[2] = __byte_perm(b, d, 0x5410), w[3] = __byte_perm(b, d, 0x7632);
}
// The low nibbles of four bytes, side by side.
__device__ __forceinline__ uint32_t nibbles(uint32_t w) {
    w &= 0x0F0F0F0Fu;
    w = (w | w >> 4) & 0x00FF00FFu;
    return (w | w >> 8) & 0xFFFFu;
}

// The part of a page that the CTA's sequence has new tokens in: its tokens
// [t0, t1), the first of which is new token `tok` of the step.
struct Part {
    uint8_t *block;  // NULL: nothing to do, or no valid page
    int t0, t1, tok;
};
template <int FMT, int D>
__device__ __forceinline__ Part part_of(const Seqs &q, int b, int64_t rel, int head) {
    const Seq s = seq_of(q, b);
    const int64_t pg = s.ctx / kPage + rel;
    const int64_t lo = max((int64_t)s.ctx, pg * kPage), hi = min((int64_t)s.ctx + s.n, pg * kPage + kPage);
    Part r{nullptr, 0, 0, 0};
    if (lo >= hi) return r;
    r.t0 = (int)(lo - pg * kPage), r.t1 = (int)(hi - pg * kPage);
    r.tok = s.first + (int)(lo - s.ctx);
    const int64_t page = page_of(q, b, pg);
    if (page >= 0) r.block = q.data + (page * q.heads + head) * Kv<FMT, D>::kBlock;
    return r;
}

template <int FMT, int D>
__global__ void __launch_bounds__(kCacheThreads, 4)
    kq_kv_append_kernel(const __grid_constant__ Seqs q, const __grid_constant__ AppendArgs a) {
    using L = Kv<FMT, D>;
    __shared__ Stage<FMT, D> st;
    const int head = blockIdx.y >> 1;
    const bool values = blockIdx.y & 1;
    const Part part = part_of<FMT, D>(q, blockIdx.z, blockIdx.x, head);
    if (!part.block) return;
    const int n = part.t1 - part.t0;
    // a thread takes the same eight values of every kStep-th token
    constexpr int kOctets = D / 8, kStep = kCacheThreads / kOctets;
    const int e = 8 * (threadIdx.x % kOctets), j0 = threadIdx.x / kOctets;
    const int64_t stride = values ? a.v_stride : a.k_stride;
    const float *src = (values ? a.v : a.k) + (int64_t)(part.tok + j0) * stride + head * D + e;
    const bool keys = !values && a.table, turn = keys && e < a.rot;
    const int half = a.rot / 2;
    // (halves may meet inside the eight values: each four has its partner)
    const int to0 = e < half ? half : -half, to1 = e + 4 < half ? half : -half;
    const int pair0 = e < half ? e : e - half, pair1 = e + 4 < half ? e + 4 : e + 4 - half;
    uint8_t *kout = part.block + L::k_octet(part.t0 + j0, e / 8);
    // every lane runs every round: quantise() shuffles; the next round's values
    // are on their way meanwhile
    float4 u = make_float4(0.f, 0.f, 0.f, 0.f), v = u;
    if (j0 < n) u = load4(src), v = load4(src + 4);
    for (int r = 0; r < (n + kStep - 1) / kStep; ++r) {
        const int j = j0 + r * kStep, t = part.t0 + j;
        const bool on = j < n;
        float x[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
        if (j + kStep < n) u = load4(src + kStep * stride), v = load4(src + kStep * stride + 4);
        if (keys && on) {
            const int pos = __ldg(a.pos + part.tok + j);
            if (pos < 0 || pos >= a.positions) {
                // (all of the key, also what is not rotated)
#pragma unroll
                for (int k = 0; k < 8; ++k) x[k] = quiet_nan();
            } else if (turn && a.inter) {
                const float4 *p =
                    reinterpret_cast<const float4 *>(a.table + (int64_t)pos * a.rot + e);
                const float4 c0 = __ldg(p), c1 = __ldg(p + 1);
                const float y[8] = {rot_a(x[0], x[1], c0.x, c0.y), rot_b(x[0], x[1], c0.x, c0.y),
                                    rot_a(x[2], x[3], c0.z, c0.w), rot_b(x[2], x[3], c0.z, c0.w),
                                    rot_a(x[4], x[5], c1.x, c1.y), rot_b(x[4], x[5], c1.x, c1.y),
                                    rot_a(x[6], x[7], c1.z, c1.w), rot_b(x[6], x[7], c1.z, c1.w)};
#pragma unroll
                for (int k = 0; k < 8; ++k) x[k] = y[k];
            } else if (turn) {
                const float *row = a.table + (int64_t)pos * a.rot;
                const float4 y0 = load4(src + to0), y1 = load4(src + 4 + to1);
                const float4 *p0 = reinterpret_cast<const float4 *>(row + 2 * pair0);
                const float4 *p1 = reinterpret_cast<const float4 *>(row + 2 * pair1);
                const float4 c[4] = {__ldg(p0), __ldg(p0 + 1), __ldg(p1), __ldg(p1 + 1)};
                const float y[8] = {y0.x, y0.y, y0.z, y0.w, y1.x, y1.y, y1.z, y1.w};
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float cc = k & 1 ? c[k / 2].z : c[k / 2].x;
                    const float ss = k & 1 ? c[k / 2].w : c[k / 2].y;
                    const bool first = (k < 4 ? to0 : to1) > 0;
                    x[k] = first ? rot_a(x[k], y[k], cc, ss) : rot_b(y[k], x[k], cc, ss);
                }
            }
        }
        if constexpr (FMT == KQ_KV_F16) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const __half2 h = __floats2half2_rn(x[2 * k], x[2 * k + 1]);
                memcpy(&w[k], &h, 4);
            }
            if (on && values) {
#pragma unroll
                for (int k = 0; k < 4; ++k) st.v[t][e / 2 + k] = w[k];
            } else if (on) {
                *reinterpret_cast<uint4 *>(kout) = make_uint4(w[0], w[1], w[2], w[3]);
            }
        } else {
            const Codes c = quantise<FMT>(x);
            const uint32_t w0 = bytes4(c.c), w1 = bytes4(c.c + 4);
            if (on && values) {
                st.v[t][e / 4] = w0, st.v[t][e / 4 + 1] = w1;
            } else if (on) {
                if constexpr (FMT == KQ_KV_Q8) *reinterpret_cast<uint2 *>(kout) = make_uint2(w0, w1);
                else *reinterpret_cast<uint32_t *>(kout) = nibbles(w0) | nibbles(w1) << 16;
            }
            if (on && (threadIdx.x & 3) == 0) {
                const int g = e / kGroup;
                *reinterpret_cast<__half *>(part.block +
                                            (values ? L::v_scale(t, g) : L::k_scale(t, g))) = c.d;
            }
        }
        src += kStep * stride;
        kout += kStep * L::kSlabBytes;
    }
    if (!values) return;
    __syncthreads();
    // Words of the values' rows, along a row first (rows of a slab are
    // contiguous); tokens of a word that this call does not write stay.
    constexpr int kEach = FMT == KQ_KV_F16 ? 2 : 4;  // values of a staged word
    constexpr int kWords = L::kVRow / 4;             // words of a row in a slab
    for (int i = threadIdx.x; i < D / kEach * L::kVWords; i += kCacheThreads) {
        const int slab = i / (D / kEach * kWords), r = i % (D / kEach * kWords);
        const int e = r / kWords, w = slab * kWords + r % kWords;  // staged word, row word
        const int tw = w * L::kVPerWord;
        if (tw + L::kVPerWord <= part.t0 || tw >= part.t1) continue;
        uint32_t out[kEach];
        if constexpr (FMT == KQ_KV_F16) {
            const uint32_t x = st.v[tw][e], y = st.v[tw + 1][e];
            out[0] = __byte_perm(x, y, 0x5410), out[1] = __byte_perm(x, y, 0x7632);
        } else {
            uint32_t x[4] = {st.v[tw][e], st.v[tw + 1][e], st.v[tw + 2][e], st.v[tw + 3][e]};
            turn4(x);
#pragma unroll
            for (int k = 0; k < 4; ++k) out[k] = x[k];
            if constexpr (FMT == KQ_KV_Q4) {
                uint32_t y[4] = {st.v[tw + 4][e], st.v[tw + 5][e], st.v[tw + 6][e], st.v[tw + 7][e]};
                turn4(y);
#pragma unroll
                for (int k = 0; k < 4; ++k) out[k] = nibbles(x[k]) | nibbles(y[k]) << 16;
            }
        }
        uint32_t keep = 0;  // bits of tokens outside [t0, t1)
        if (tw < part.t0) keep = ~(~0u << (L::kBits * (part.t0 - tw)));
        if (tw + L::kVPerWord > part.t1) keep |= ~0u << (L::kBits * (part.t1 - tw));
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            uint32_t *o = reinterpret_cast<uint32_t *>(part.block + L::v_word(kEach * e + k, w));
            *o = keep ? (*o & keep) | (out[k] & ~keep) : out[k];
        }
    }
}

template <int FMT, int D>
__global__ void __launch_bounds__(kCacheThreads)
    kq_kv_read_kernel(const __grid_constant__ Seqs q, float *__restrict__ ko,
                      float *__restrict__ vo) {
    using L = Kv<FMT, D>;
    const int head = blockIdx.y >> 1;
    const bool values = blockIdx.y & 1;
    float *out = values ? vo : ko;
    if (!out) return;
    const Part part = part_of<FMT, D>(q, blockIdx.z, blockIdx.x, head);
    const int n = part.t1 - part.t0;
    const int64_t stride = (int64_t)q.heads * D;
    out += (int64_t)part.tok * stride + head * D;
    if (!part.block) {
        const float x = quiet_nan();
        for (int i = threadIdx.x; i < n * (D / 4); i += kCacheThreads)
            *reinterpret_cast<float4 *>(out + i / (D / 4) * stride + 4 * (i % (D / 4))) =
                make_float4(x, x, x, x);
        return;
    }
    if (values) {
        // A warp takes a group of 32 values, a lane each, and eight tokens of
        // its row at a time: a token's store is 128 contiguous bytes.
        const int lane = threadIdx.x & 31;
        for (int i = threadIdx.x / 32; i < L::kGroups * (kPage / 8); i += kCacheThreads / 32) {
            const int g = i % L::kGroups, tw = i / L::kGroups * 8;
            if (tw + 8 <= part.t0 || tw >= part.t1) continue;
            const uint8_t *row = part.block + L::v_word(g * kGroup + lane, tw / L::kVPerWord);
            float x[8];
            if constexpr (FMT == KQ_KV_F16) {
                const uint4 w = *reinterpret_cast<const uint4 *>(row);
                const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    x[k] = __half2float(__ushort_as_half((uint16_t)(ws[k / 2] >> (16 * (k & 1)))));
            } else {
                uint32_t ws[2];
                if constexpr (FMT == KQ_KV_Q8) {
                    const uint2 w = *reinterpret_cast<const uint2 *>(row);
                    ws[0] = w.x, ws[1] = w.y;
                } else {
                    ws[0] = *reinterpret_cast<const uint32_t *>(row);
                }
                const uint4 s = *reinterpret_cast<const uint4 *>(part.block + L::v_scale(tw, g));
                const uint32_t ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint32_t w = ws[k * L::kBits / 32];
                    const int c = (int)(w << (32 - L::kBits - k * L::kBits % 32)) >> (32 - L::kBits);
                    x[k] = (float)c *
                           __half2float(__ushort_as_half((uint16_t)(ss[k / 2] >> (16 * (k & 1)))));
                }
            }
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (tw + k >= part.t0 && tw + k < part.t1)
                    out[(tw + k - part.t0) * stride + g * kGroup + lane] = x[k];
        }
        return;
    }
#pragma unroll 4
    for (int i = threadIdx.x; i < n * (D / 4); i += kCacheThreads) {
        const int j = i / (D / 4), e = 4 * (i % (D / 4)), t = part.t0 + j, g = e / kGroup;
        const uint8_t *p = part.block + L::k_octet(t, e / 8) + (e & 4) * L::kBits / 8;
        float x[4];
        if constexpr (FMT == KQ_KV_F16) {
            const uint2 w = *reinterpret_cast<const uint2 *>(p);
            const uint32_t ws[2] = {w.x, w.y};
#pragma unroll
            for (int k = 0; k < 4; ++k)
                x[k] = __half2float(__ushort_as_half((uint16_t)(ws[k / 2] >> (16 * (k & 1)))));
        } else {
            const float d =
                __half2float(*reinterpret_cast<const __half *>(part.block + L::k_scale(t, g)));
            const uint32_t w = FMT == KQ_KV_Q8 ? *reinterpret_cast<const uint32_t *>(p)
                                               : *reinterpret_cast<const uint16_t *>(p);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                x[k] = (float)((int)(w << (32 - L::kBits * (k + 1))) >> (32 - L::kBits)) * d;
        }
        *reinterpret_cast<float4 *>(out + j * stride + e) = make_float4(x[0], x[1], x[2], x[3]);
    }
}

// One CTA per (sequence, head).  Tokens are moved one after another; a
// thread moves the same words and rows of every token, so it alone reads
// and writes them, in order, and needs no barrier.
template <int FMT, int D>
__global__ void __launch_bounds__(D)
    kq_kv_move_kernel(const __grid_constant__ Seqs q, const int32_t *__restrict__ path,
                      const int32_t *__restrict__ count) {
    using L = Kv<FMT, D>;
    const int b = blockIdx.x, head = blockIdx.y, e = threadIdx.x;
    const Seq s = seq_of(q, b);
    const int n = min(__ldg(count + b), s.n);
    int before = -1;
    for (int i = 0; i < n; ++i) {
        const int from = __ldg(path + s.first + i);
        if (from <= before || from >= s.n) return;
        before = from;
        if (from == i) continue;
        const int64_t ps = s.ctx + from, pd = s.ctx + i;
        const int64_t src_page = page_of(q, b, ps / kPage), dst_page = page_of(q, b, pd / kPage);
        if (src_page < 0 || dst_page < 0) continue;
        uint8_t *src = q.data + (src_page * q.heads + head) * L::kBlock;
        uint8_t *dst = q.data + (dst_page * q.heads + head) * L::kBlock;
        const int ts = (int)(ps % kPage), td = (int)(pd % kPage);
        if (e < D * L::kBits / 32) {  // a word of the key
            constexpr int kWords = L::kOctet / 4;
            const int w = (e % kWords) * 4;
            *reinterpret_cast<uint32_t *>(dst + L::k_octet(td, e / kWords) + w) =
                *reinterpret_cast<const uint32_t *>(src + L::k_octet(ts, e / kWords) + w);
        }
        {  // a value: bits of a word that holds other tokens too
            const uint32_t m = L::kBits == 16 ? 0xFFFFu : (1u << L::kBits) - 1u;
            const int ss = (ts % L::kVPerWord) * L::kBits, sd = (td % L::kVPerWord) * L::kBits;
            const uint32_t v =
                (*reinterpret_cast<const uint32_t *>(src + L::v_word(e, ts / L::kVPerWord)) >> ss) & m;
            uint32_t *o = reinterpret_cast<uint32_t *>(dst + L::v_word(e, td / L::kVPerWord));
            *o = (*o & ~(m << sd)) | (v << sd);
        }
        if (L::kQuant && e < L::kGroups) {
            *reinterpret_cast<uint16_t *>(dst + L::k_scale(td, e)) =
                *reinterpret_cast<const uint16_t *>(src + L::k_scale(ts, e));
            *reinterpret_cast<uint16_t *>(dst + L::v_scale(td, e)) =
                *reinterpret_cast<const uint16_t *>(src + L::v_scale(ts, e));
        }
    }
}

namespace {
// Pages that max_new tokens from any place on can touch.
unsigned pages_touched(int max_new) { return (unsigned)((max_new + kPage - 2) / kPage + 1); }

template <int FMT, int D>
struct Run {
    static cudaError_t append(const Seqs &q, const AppendArgs &a, cudaStream_t s) {
        const dim3 grid(pages_touched(q.max_new), 2 * q.heads, q.nseq);
        kq_kv_append_kernel<FMT, D><<<grid, kCacheThreads, 0, s>>>(q, a);
        return cudaGetLastError();
    }
    static cudaError_t read(const Seqs &q, float *k, float *v, cudaStream_t s) {
        const dim3 grid(pages_touched(q.max_new), 2 * q.heads, q.nseq);
        kq_kv_read_kernel<FMT, D><<<grid, kCacheThreads, 0, s>>>(q, k, v);
        return cudaGetLastError();
    }
    static cudaError_t move(const Seqs &q, const int32_t *path, const int32_t *count,
                            cudaStream_t s) {
        kq_kv_move_kernel<FMT, D><<<dim3(q.nseq, q.heads), D, 0, s>>>(q, path, count);
        return cudaGetLastError();
    }
};

// f<FMT, D> for the cache's format and width (checked before).
template <class F>
cudaError_t pick(int fmt, int dim, F f) {
    switch (fmt * 1000 + dim) {
    case KQ_KV_F16 * 1000 + 64: return f(Run<KQ_KV_F16, 64>());
    case KQ_KV_F16 * 1000 + 128: return f(Run<KQ_KV_F16, 128>());
    case KQ_KV_F16 * 1000 + 256: return f(Run<KQ_KV_F16, 256>());
    case KQ_KV_Q8 * 1000 + 64: return f(Run<KQ_KV_Q8, 64>());
    case KQ_KV_Q8 * 1000 + 128: return f(Run<KQ_KV_Q8, 128>());
    case KQ_KV_Q8 * 1000 + 256: return f(Run<KQ_KV_Q8, 256>());
    case KQ_KV_Q4 * 1000 + 64: return f(Run<KQ_KV_Q4, 64>());
    case KQ_KV_Q4 * 1000 + 128: return f(Run<KQ_KV_Q4, 128>());
    case KQ_KV_Q4 * 1000 + 256: return f(Run<KQ_KV_Q4, 256>());
    default: return cudaErrorInvalidValue;
    }
}
}  // namespace

cudaError_t kv_append(int fmt, int dim, const Seqs &q, const AppendArgs &a, cudaStream_t s) {
    return pick(fmt, dim, [&](auto r) { return r.append(q, a, s); });
}
cudaError_t kv_read(int fmt, int dim, const Seqs &q, float *k, float *v, cudaStream_t s) {
    return pick(fmt, dim, [&](auto r) { return r.read(q, k, v, s); });
}
cudaError_t kv_move(int fmt, int dim, const Seqs &q, const int32_t *path, const int32_t *count,
                    cudaStream_t s) {
    return pick(fmt, dim, [&](auto r) { return r.move(q, path, count, s); });
}

}  // namespace kqd
