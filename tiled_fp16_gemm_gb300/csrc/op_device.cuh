// Device helpers of the operators beside the GEMM (gemm_w4.cuh, norm.cuh).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace tg {

__device__ __forceinline__ float op_to_float(float v) { return v; }
__device__ __forceinline__ float op_to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float op_to_float(__nv_bfloat16 v) { return __bfloat162float(v); }

// fp32 to T, to the nearest (ties to even).
template <typename T>
__device__ __forceinline__ T op_round(float v);
template <>
__device__ __forceinline__ float op_round<float>(float v) {
    return v;
}
template <>
__device__ __forceinline__ __half op_round<__half>(float v) {
    return __float2half_rn(v);
}
template <>
__device__ __forceinline__ __nv_bfloat16 op_round<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}

// Dependent launch: wait for the previous kernel of the stream to complete
// before the first access to global memory, and let the next one set up.
__device__ __forceinline__ void op_wait_previous() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void op_release_next() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Bits of the device's word for waits that ran out (the GEMM's kernels have the low ones).
constexpr unsigned int kOpTimeoutW4 = 1u << 16;
constexpr unsigned int kOpTimeoutNorm = 1u << 17;
constexpr unsigned int kOpTimeoutI8 = 1u << 18;

// ------------------------------------------------------------------ mbarriers and TMA

__device__ __forceinline__ uint32_t op_smem(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void op_bar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void op_bar_init_done() {
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}
__device__ __forceinline__ void op_bar_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ uint32_t op_bar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok;
}
// Until the phase of `bar` with this parity is over, or `limit_ns` have passed: false.
// The clock is read only now and then, and no sleep time is asked for: a sleeping warp
// woke up late, and the roles of a block wait for one another all the time.
static __device__ __noinline__ bool op_bar_wait_slow(uint32_t bar, uint32_t parity,
                                                     uint64_t limit_ns) {
    uint64_t t0 = 0, t = 0;
    do {
#pragma unroll 1
        for (int i = 0; i < 64; ++i)
            if (op_bar_try(bar, parity)) return true;
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
        if (t0 == 0) t0 = t;
    } while (t - t0 <= limit_ns);
    return false;
}
__device__ __forceinline__ bool op_bar_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
    return op_bar_try(bar, parity) || op_bar_wait_slow(bar, parity, limit_ns);
}

// A box of a 2-D tensor map to shared memory; x is the contiguous coordinate.
__device__ __forceinline__ void op_tma_2d(uint32_t dst, const void* map, uint32_t bar, uint32_t x,
                                          uint32_t y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

}  // namespace tg
