// Device helpers of the operators beside the GEMM (gemm_w4.cuh, norm.cuh).
#pragma once

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

}  // namespace tg
