// Products of 8-bit integers with a scale per row of A (token) and per row of B (channel):
//
//   C[m][n] = out( act( sa[m] · sb[n] · Σ_k a[m][k]·b[n][k] + bias[n] ) + R[m][n] )
#pragma once

#include "op_device.cuh"

namespace tg {

struct I8Params {
    const int8_t* A;
    int64_t lda;
    const float* sa;
    const int8_t* B;
    int64_t ldb;
    const float* sb;
    void* C;
    int64_t ldc;
    const float* bias;
    const void* resid;  // of C's type
    int64_t ldr;
    int64_t M, N, K;
    int32_t relu;
};

// The epilogue of one sum, unrounded: scales, bias and activation in fp32.
__device__ __forceinline__ float i8_value(const I8Params& p, float sum, float sa, float sb, float bias) {
    const float v = fmaf(sum * sa, sb, bias);
    return p.relu && !(v > 0.0f) ? 0.0f : v;
}

// A warp per element of C: any size and layout.
template <typename TC>
__global__ void __launch_bounds__(256) tg_gemm_i8_simple(const I8Params p) {
    op_release_next();
    op_wait_previous();
    const int lane = threadIdx.x & 31;
    const int64_t warps = int64_t{gridDim.x} * 8;
    for (int64_t i = int64_t{blockIdx.x} * 8 + threadIdx.x / 32; i < p.M * p.N; i += warps) {
        const int64_t n = i / p.M, m = i % p.M;
        const int8_t *a = p.A + m * p.lda, *b = p.B + n * p.ldb;
        int sum = 0;
        for (int64_t k = lane; k < p.K; k += 32) sum += int{a[k]} * int{b[k]};
        sum = __reduce_add_sync(0xffffffffu, sum);
        if (lane == 0) {
            float v = i8_value(p, static_cast<float>(sum), p.sa[m], p.sb[n], p.bias != nullptr ? p.bias[n] : 0.0f);
            if (p.resid != nullptr) v += op_to_float((static_cast<const TC*>(p.resid) + m * p.ldr)[n]);
            (static_cast<TC*>(p.C) + m * p.ldc)[n] = op_round<TC>(v);
        }
    }
}

}  // namespace tg
