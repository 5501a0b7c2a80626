// tma.cuh -- shared-memory barriers, tensor copies and asynchronous loads of the
// paged-cache kernels, and the host's tensor map over the pages.
#pragma once

#include <atomic>
#include <cuda.h>
#include <cudaTypedefs.h>

#include "common.cuh"
#include "paged.h"

namespace tsa {

#ifndef TSA_WAIT_SPINS
constexpr long kPagedSpins = 1L << 22;  // bounded mbarrier wait
#else
constexpr long kPagedSpins = TSA_WAIT_SPINS;  // a debug build's short limit
#endif

__device__ __forceinline__ unsigned su32(const void* p) { return (unsigned)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void mbar_init(unsigned bar, unsigned count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;\n" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_init_fence() { asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory"); }
__device__ __forceinline__ void mbar_arrive(unsigned bar) {
    asm volatile("{\n .reg .b64 st;\n mbarrier.arrive.shared::cta.b64 st, [%0];\n}\n" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_arrive_tx(unsigned bar, unsigned bytes) {
    asm volatile("{\n .reg .b64 st;\n mbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1;\n}\n" ::"r"(bar), "r"(bytes)
                 : "memory");
}
// bounded wait for the phase of the given parity; false = gave up (flag raised,
// unless flag is NULL: a drain wait at the end)
__device__ __forceinline__ bool mbar_wait(unsigned bar, unsigned parity, unsigned* flag) {
    for (long i = 0; i < kPagedSpins; ++i) {
        unsigned done;
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(done)
            : "r"(bar), "r"(parity)
            : "memory");
        if (done) return true;
    }
    if (flag) atomicOr(flag, kFlagTimeout);
    return false;
}

__device__ __forceinline__ uint64_t evict_first_policy() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;\n" : "=l"(p));
    return p;
}

// one box of the pages' tensor map (element, row in page, kv-head, page)
__device__ __forceinline__ void tma_4d(unsigned dst, const CUtensorMap* map, int x, int row, int head, int page,
                                       unsigned bar, uint64_t pol) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3, "
        "%4, %5}], [%6], %7;\n" ::"r"(dst),
        "l"(map), "r"(x), "r"(row), "r"(head), "r"(page), "r"(bar), "l"(pol)
        : "memory");
}

__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory"); }

// contiguous bytes (a multiple of 16, 16-byte aligned) out of shared memory; then wait until they are in memory
__device__ __forceinline__ void bulk_store(void* dst, unsigned src, int bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;\n" ::"l"(dst), "r"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_store_wait() {
    asm volatile("cp.async.bulk.commit_group;\n" ::: "memory");
    asm volatile("cp.async.bulk.wait_group 0;\n" ::: "memory");
}

// 16 bytes into shared memory, the last 16 - n of them zeros
__device__ __forceinline__ void cp_async16(unsigned dst, const void* src, int n) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}

// ---- host

// The pages of one pool as a 4-D tensor (element, row in page, kv-head, page),
// read in boxes of 64 elements x `rows` rows, 128-byte swizzle.
cudaError_t page_map(CUtensorMap* map, const Pages& c, void* base, int rows);

// Let a kernel use `bytes` of dynamic shared memory on the current device;
// `done` holds a bit per device that has been told.
inline cudaError_t smem_opt_in(const void* kernel, int bytes, std::atomic<unsigned long long>* done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && (done->load(std::memory_order_relaxed) >> dev & 1ull)) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < 64) done->fetch_or(1ull << dev, std::memory_order_relaxed);
    return e;
}

}  // namespace tsa
