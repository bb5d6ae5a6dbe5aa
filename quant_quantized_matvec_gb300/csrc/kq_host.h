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

struct Span {
    uintptr_t lo, hi;  // [lo, hi)
};
inline Span span(const void *p, int64_t bytes) {
    return {(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes};
}
inline bool meet(Span a, Span b) { return a.lo < b.hi && b.lo < a.hi; }

}  // namespace kqhost
