// kq_host.h -- host helpers that the library's C entry points share
// (defined in kq_api.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kq.h"

namespace kqhost {

// Record a failed CUDA call for kq_last_cuda_error; returns KQ_ERR_CUDA.
kq_status cuda_failed(cudaError_t e);

// KQ_OK if p is memory of the current device or managed memory.
kq_status on_device(const void *p, int dev);

// The current device: its SM count, the device address of its error word
// (kq_device_error), and the wall-time limit of its kernels' waits.
struct Device {
    int sms;
    unsigned int *err;
    unsigned long long wait_ns;
};
cudaError_t device(Device &d);

// A tensor map over `blocks` blocks of `rows` rows of 64 bytes (f16), boxes of
// `box` rows, swizzled over 64 bytes.
cudaError_t rows_map(const void *data, int rows, int64_t blocks, int box, CUtensorMap *out);

// A tensor map of values of a type of kq_prompt.h, `rank` dimensions (strides in
// bytes, of the second and on), boxes of 128 bytes by the others, swizzled over
// 128 bytes, with zeros outside.
cudaError_t values_map(const void *data, int type, int rank, const uint64_t *dims,
                       const uint64_t *strides, const uint32_t *box, CUtensorMap *out);

struct Span {
    uintptr_t lo, hi;  // [lo, hi)
};
inline Span span(const void *p, int64_t bytes) {
    return {(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes};
}
inline bool meet(Span a, Span b) { return a.lo < b.hi && b.lo < a.hi; }


inline bool aligned(const void *p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

// Pointers of a call, for the alias and memory checks.
struct Pointers {
    Span in[12], out[4];
    const void *p[16];
    int ni = 0, no = 0, np = 0;
    void read(const void *q, int64_t bytes) { in[ni++] = span(q, bytes), p[np++] = q; }
    void write(const void *q, int64_t bytes) { out[no++] = span(q, bytes), p[np++] = q; }
    kq_status check() const {
        for (int i = 0; i < no; ++i) {
            for (int j = 0; j < ni; ++j)
                if (meet(out[i], in[j])) return KQ_ERR_ALIAS;
            for (int j = 0; j < i; ++j)
                if (meet(out[i], out[j])) return KQ_ERR_ALIAS;
        }
        return memory();
    }
    kq_status memory() const {
        int dev = 0;
        const cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return cuda_failed(e);
        for (int i = 0; i < np; ++i) {
            const kq_status s = on_device(p[i], dev);
            if (s != KQ_OK) return s;
        }
        return KQ_OK;
    }
};

inline kq_status launched(cudaError_t e) { return e == cudaSuccess ? KQ_OK : cuda_failed(e); }

}  // namespace kqhost
