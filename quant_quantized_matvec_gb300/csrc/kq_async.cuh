// kq_async.cuh -- asynchronous copies and bounded waits that the library's
// kernels share.
#pragma once

#include <stdint.h>

namespace kq {

constexpr unsigned long long kWaitLimitNs = 2000000000ull;  // 2 s (default)
constexpr unsigned kSuspendNs = 100000;  // a thread's suspension by mbar_try

__device__ __forceinline__ uint32_t smem_addr(const void *p) {
    return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count));
}
__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar),
                 "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n"
        " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 100000;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
// Whether the phase of `parity` has completed, without waiting.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n"
        " mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ unsigned long long global_ns() {
    unsigned long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
// Wait for the phase of `parity` to complete; false once `limit_ns` of wall
// time have passed.  Between polls the thread sleeps, doubling from 32 ns up
// to `max_ns`, so that waiting warps leave the issue slots to working ones.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity,
                                          unsigned long long limit_ns,
                                          unsigned max_ns = 256) {
    if (mbar_try(bar, parity)) return true;
    const unsigned long long t0 = global_ns();
    unsigned ns = 32;
    while (!mbar_try(bar, parity)) {
        __nanosleep(ns);
        if (ns < max_ns) ns <<= 1;
        if (global_ns() - t0 > limit_ns) return false;
    }
    return true;
}
// mbar_wait with a limit that may be shorter than the 100 us for which
// mbar_try may suspend the thread (suspend_ns: the lesser of the two).  It
// sleeps before it looks at the time: the other way round 32 sequences of
// 16384 at most, 4 drafts, 64 / 8 heads, 8-bit, took 472 us and not 414.
__device__ __forceinline__ bool mbar_wait_for(uint32_t bar, uint32_t parity,
                                              unsigned long long limit_ns, uint32_t suspend_ns) {
    auto arrived = [&]() {
        uint32_t ok;
        asm volatile(
            "{\n .reg .pred p;\n"
            " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
            " selp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(ok)
            : "r"(bar), "r"(parity), "r"(suspend_ns)
            : "memory");
        return ok != 0;
    };
    if (arrived()) return true;
    const unsigned long long t0 = global_ns();
    unsigned ns = 32;
    while (!arrived()) {
        __nanosleep(ns);
        if (ns < 256) ns <<= 1;
        if (global_ns() - t0 > limit_ns) return false;
    }
    return true;
}
// The same without sleeping between tries, for waits that the work goes by.
__device__ __forceinline__ bool mbar_wait_awake(uint32_t bar, uint32_t parity,
                                                unsigned long long limit_ns, uint32_t suspend_ns) {
    unsigned long long t0 = 0;
    while (true) {
        uint32_t ok;
        asm volatile(
            "{\n .reg .pred p;\n"
            " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
            " selp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(ok)
            : "r"(bar), "r"(parity), "r"(suspend_ns)
            : "memory");
        if (ok) return true;
        const unsigned long long now = global_ns();
        if (t0 == 0) t0 = now;
        else if (now - t0 > limit_ns) return false;
    }
}
__device__ __forceinline__ void bulk_g2s(uint32_t dst, const void *src,
                                         uint32_t bytes, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes"
        " [%0], [%1], %2, [%3];" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(bar)
        : "memory");
}
// Programmatic dependent launch: let the next kernel on the stream launch,
// and wait for the preceding one (no-ops for an ordinary launch).
__device__ __forceinline__ void allow_dependents() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_prerequisites() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
}  // namespace kq
