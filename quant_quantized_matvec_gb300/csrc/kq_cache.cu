// kq_cache.cu -- the quantised key/value cache: written (append), read back
// (read), and closed up after a verification (move).
//
// One CTA per (page of a sequence, head, keys or values), so that every
// byte of a page's keys or values is written by one CTA: a byte of 4-bit
// values holds two tokens, and whole words are read, changed and written
// where a call covers only some of their tokens.
//
// Quantisation: eight lanes hold a group of 32 values, four each; its
// largest and smallest value come from three shuffles.
// Bound by memory: 4 bytes a value on the f32 side, bits/8 on the other.
#include "kq_decode.cuh"
#include "kq_decode_launch.h"

namespace kqd {

constexpr int kCacheThreads = 256;

// ------------------------------------------------------------------ codes
// The four codes of a lane (of eight that hold a group) and the group's
// scale; every lane of the warp takes part.
struct Codes {
    int c[4];
    __half d;
};
template <int FMT>
__device__ __forceinline__ Codes quantise(const float (&x)[4]) {
    float hi = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
    float lo = fminf(fminf(x[0], x[1]), fminf(x[2], x[3]));
    // a NaN or an infinity makes the sum of x * 0 a NaN
    float bad = x[0] * 0.f + x[1] * 0.f + x[2] * 0.f + x[3] * 0.f;
#pragma unroll
    for (int o = 1; o < 8; o *= 2) {
        hi = fmaxf(hi, __shfl_xor_sync(~0u, hi, o));
        lo = fminf(lo, __shfl_xor_sync(~0u, lo, o));
        bad += __shfl_xor_sync(~0u, bad, o);
    }
    float d = FMT == KQ_KV_Q8 ? __fdiv_rn(fmaxf(hi, -lo), 127.f) : (hi >= -lo ? hi : lo) * -0.125f;
    d = fminf(fmaxf(d, -65504.f), 65504.f);
    Codes r;
    r.d = __float2half_rn(bad == 0.f ? d : quiet_nan());
    const float df = __half2float(r.d);
    const float top = FMT == KQ_KV_Q8 ? 127.f : 7.f, bot = FMT == KQ_KV_Q8 ? -127.f : -8.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float c = df == 0.f || bad != 0.f ? 0.f : rintf(__fdiv_rn(x[i], df));
        r.c[i] = (int)fminf(fmaxf(c, bot), top);
    }
    return r;
}

__device__ __forceinline__ void load4(float (&x)[4], const float *p) {
    const float4 v = *reinterpret_cast<const float4 *>(p);
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
}

// Values e .. e+3 (e a multiple of 4) of the head at p, rotated.
__device__ __forceinline__ void load4_rotated(float (&x)[4], const float *p, int e, int tok,
                                              const AppendArgs &a) {
    load4(x, p + e);
    if (!a.table || e >= a.rot) return;
    const int pos = __ldg(a.pos + tok);
    if (pos < 0 || pos >= a.positions) {
        x[0] = x[1] = x[2] = x[3] = quiet_nan();
        return;
    }
    const float *row = a.table + (int64_t)pos * a.rot;
    if (a.inter) {
        const float4 cs = __ldg(reinterpret_cast<const float4 *>(row + e));
        const float y[4] = {rot_a(x[0], x[1], cs.x, cs.y), rot_b(x[0], x[1], cs.x, cs.y),
                            rot_a(x[2], x[3], cs.z, cs.w), rot_b(x[2], x[3], cs.z, cs.w)};
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = y[i];
        return;
    }
    const int half = a.rot / 2;
    const bool first = e < half;
    const int pair = first ? e : e - half;
    float y[4];
    load4(y, p + (first ? e + half : pair));
    const float4 c0 = __ldg(reinterpret_cast<const float4 *>(row + 2 * pair));
    const float4 c1 = __ldg(reinterpret_cast<const float4 *>(row + 2 * pair) + 1);
    const float c[4] = {c0.x, c0.z, c1.x, c1.z}, s[4] = {c0.y, c0.w, c1.y, c1.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        x[i] = first ? rot_a(x[i], y[i], c[i], s[i]) : rot_b(y[i], x[i], c[i], s[i]);
}

// Values in shared memory on their way between [token][value] and the
// cache's [value][token]: f16 bits or sign-extended codes.
template <int FMT, int D>
struct Stage {
    using T = typename std::conditional<FMT == KQ_KV_F16, uint16_t, int8_t>::type;
    static constexpr int kPad = 4 / sizeof(T);
    T v[kPage][D + kPad];
};

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
__global__ void __launch_bounds__(kCacheThreads)
    kq_kv_append_kernel(const __grid_constant__ Seqs q, const __grid_constant__ AppendArgs a) {
    using L = Kv<FMT, D>;
    __shared__ Stage<FMT, D> st;
    const int head = blockIdx.y >> 1;
    const bool values = blockIdx.y & 1;
    const Part part = part_of<FMT, D>(q, blockIdx.z, blockIdx.x, head);
    if (!part.block) return;
    const int n = part.t1 - part.t0;
    const int l8 = threadIdx.x & 7;
    constexpr int kPer = kCacheThreads / 8;  // groups at a time
    // every lane runs every round: quantise() shuffles
    for (int i0 = 0; i0 < n * L::kGroups; i0 += kPer) {
        const int i = i0 + threadIdx.x / 8;
        const bool on = i < n * L::kGroups;
        const int j = on ? i / L::kGroups : 0, g = on ? i % L::kGroups : 0;
        const int e = g * kGroup + 4 * l8, t = part.t0 + j;
        float x[4] = {0.f, 0.f, 0.f, 0.f};
        const int64_t row = part.tok + j;
        if (on) {
            if (values) load4(x, a.v + row * a.v_stride + head * D + e);
            else load4_rotated(x, a.k + row * a.k_stride + head * D, e, (int)row, a);
        }
        uint32_t w[2];  // the four values as the cache holds them
        if constexpr (FMT == KQ_KV_F16) {
            const __half2 h0 = __floats2half2_rn(x[0], x[1]), h1 = __floats2half2_rn(x[2], x[3]);
            w[0] = *reinterpret_cast<const uint32_t *>(&h0);
            w[1] = *reinterpret_cast<const uint32_t *>(&h1);
            if (on && values) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    st.v[t][e + k] = (uint16_t)(w[k / 2] >> (16 * (k & 1)));
            }
        } else {
            const Codes c = quantise<FMT>(x);
            const uint32_t m = FMT == KQ_KV_Q8 ? 0xFFu : 0xFu;
            w[0] = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) w[0] |= ((uint32_t)c.c[k] & m) << (L::kBits * k);
            if (on && values) {
#pragma unroll
                for (int k = 0; k < 4; ++k) st.v[t][e + k] = (int8_t)c.c[k];
            }
            if (on && l8 == 0)
                *reinterpret_cast<__half *>(part.block +
                                            (values ? L::v_scale(t, g) : L::k_scale(t, g))) = c.d;
        }
        if (on && !values) {
            uint8_t *o = part.block + L::k_octet(t, e / 8) + (e & 4) * L::kBits / 8;
            if constexpr (FMT == KQ_KV_F16)
                *reinterpret_cast<uint2 *>(o) = make_uint2(w[0], w[1]);
            else if constexpr (FMT == KQ_KV_Q8)
                *reinterpret_cast<uint32_t *>(o) = w[0];
            else
                *reinterpret_cast<uint16_t *>(o) = (uint16_t)w[0];
        }
    }
    if (!values) return;
    __syncthreads();
    // words of the values' rows, along a row first (rows of a slab are
    // contiguous); tokens of the word that this call does not write stay
    constexpr int kWords = L::kVRow / 4;
    for (int i = threadIdx.x; i < D * L::kVWords; i += kCacheThreads) {
        const int slab = i / (D * kWords), r = i % (D * kWords);
        const int e = r / kWords, w = slab * kWords + r % kWords;
        const int tw = w * L::kVPerWord;
        if (tw + L::kVPerWord <= part.t0 || tw >= part.t1) continue;
        uint32_t word = 0, keep = 0;
#pragma unroll
        for (int k = 0; k < L::kVPerWord; ++k) {
            const uint32_t m = L::kBits == 16 ? 0xFFFFu : (1u << L::kBits) - 1u;
            if (tw + k >= part.t0 && tw + k < part.t1)
                word |= ((uint32_t)st.v[tw + k][e] & m) << (L::kBits * k);
            else
                keep |= m << (L::kBits * k);
        }
        uint32_t *o = reinterpret_cast<uint32_t *>(part.block + L::v_word(e, w));
        *o = keep ? (*o & keep) | word : word;
    }
}

template <int FMT, int D>
__global__ void __launch_bounds__(kCacheThreads)
    kq_kv_read_kernel(const __grid_constant__ Seqs q, float *__restrict__ ko,
                      float *__restrict__ vo) {
    using L = Kv<FMT, D>;
    __shared__ Stage<FMT, D> st;
    const int head = blockIdx.y >> 1;
    const bool values = blockIdx.y & 1;
    float *out = values ? vo : ko;
    if (!out) return;
    const Part part = part_of<FMT, D>(q, blockIdx.z, blockIdx.x, head);
    const int n = part.t1 - part.t0;
    if (part.block && values) {
        constexpr int kWords = L::kVRow / 4;
        for (int i = threadIdx.x; i < D * L::kVWords; i += kCacheThreads) {
            const int slab = i / (D * kWords), r = i % (D * kWords);
            const int e = r / kWords, w = slab * kWords + r % kWords;
            const int tw = w * L::kVPerWord;
            if (tw + L::kVPerWord <= part.t0 || tw >= part.t1) continue;
            const uint32_t word = *reinterpret_cast<const uint32_t *>(part.block + L::v_word(e, w));
#pragma unroll
            for (int k = 0; k < L::kVPerWord; ++k) {
                if constexpr (FMT == KQ_KV_F16)
                    st.v[tw + k][e] = (uint16_t)(word >> (16 * k));
                else  // sign-extended
                    st.v[tw + k][e] =
                        (int8_t)((int)(word << (32 - L::kBits * (k + 1))) >> (32 - L::kBits));
            }
        }
        __syncthreads();
    }
    for (int i = threadIdx.x; i < n * (D / 4); i += kCacheThreads) {
        const int j = i / (D / 4), e = 4 * (i % (D / 4)), t = part.t0 + j, g = e / kGroup;
        float x[4];
        if (!part.block) {
            x[0] = x[1] = x[2] = x[3] = quiet_nan();
        } else if constexpr (FMT == KQ_KV_F16) {
            uint16_t h[4];
            if (values) {
#pragma unroll
                for (int k = 0; k < 4; ++k) h[k] = st.v[t][e + k];
            } else {
                const uint2 w = *reinterpret_cast<const uint2 *>(
                    part.block + L::k_octet(t, e / 8) + (e & 4) * 2);
                h[0] = (uint16_t)w.x, h[1] = (uint16_t)(w.x >> 16);
                h[2] = (uint16_t)w.y, h[3] = (uint16_t)(w.y >> 16);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) x[k] = __half2float(__ushort_as_half(h[k]));
        } else {
            const float d = __half2float(*reinterpret_cast<const __half *>(
                part.block + (values ? L::v_scale(t, g) : L::k_scale(t, g))));
            if (values) {
#pragma unroll
                for (int k = 0; k < 4; ++k) x[k] = (float)st.v[t][e + k] * d;
            } else {
                const uint8_t *p = part.block + L::k_octet(t, e / 8) + (e & 4) * L::kBits / 8;
                const uint32_t w = FMT == KQ_KV_Q8 ? *reinterpret_cast<const uint32_t *>(p)
                                                   : *reinterpret_cast<const uint16_t *>(p);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    x[k] = (float)((int)(w << (32 - L::kBits * (k + 1))) >> (32 - L::kBits)) * d;
            }
        }
        *reinterpret_cast<float4 *>(out + ((int64_t)(part.tok + j) * q.heads + head) * D + e) =
            make_float4(x[0], x[1], x[2], x[3]);
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
