// Products with 4-bit weights and group scales:
//
//   W[n][k] = (code[n][k] - zero[k / G][n]) · scale[k / G][n]
//   C[m][n] = out(act(Σ_k A[m][k]·W[n][k] + bias[n]) + R[m][n])
//
// G = 32, 64 or 128; code and zero are 0..15 (zero = 8 where none are given).
// For few rows of A the sum is taken group by group,
//   Σ_groups scale · (Σ_{k in group} A[m][k]·(code - zero)),
// with code - zero exact and both sums in fp32: no weight is ever rounded.
#pragma once

#include "op_device.cuh"

namespace tg {

struct W4Params {
    const void* A;
    int64_t lda;
    const uint8_t* Bq;
    int64_t ldbq;
    const void* scale;
    int64_t lds;
    const uint8_t* zero;  // or null
    int64_t ldz;
    void* C;
    int64_t ldc;
    const float* bias;
    const void* resid;
    int64_t ldr;
    int64_t M, N, K;
    int32_t group;
    int32_t relu;
    int32_t out_f32;
};

template <typename T>
__device__ __forceinline__ void w4_store(const W4Params& p, int64_t m, int64_t n, float acc) {
    if (p.bias != nullptr) acc += p.bias[n];
    if (p.relu) acc = acc > 0.0f ? acc : 0.0f;
    if (p.resid != nullptr)
        acc += op_to_float(static_cast<const T*>(p.resid)[m * p.ldr + n]);
    if (p.out_f32)
        static_cast<float*>(p.C)[m * p.ldc + n] = acc;
    else
        static_cast<T*>(p.C)[m * p.ldc + n] = op_round<T>(acc);
}

// One warp per (row of W, 8 rows of A), lane l taking codes l, l + 32, ...
template <typename T>
__global__ void __launch_bounds__(256) tg_gemm_w4_simple(const W4Params p) {
    const int lane = threadIdx.x & 31;
    const int64_t tiles_m = (p.M + 7) / 8;
    const int64_t jobs = tiles_m * p.N;
    for (int64_t job = int64_t{blockIdx.x} * 8 + (threadIdx.x >> 5); job < jobs;
         job += int64_t{gridDim.x} * 8) {
        const int64_t n = job % p.N, m0 = job / p.N * 8;
        float acc[8] = {};
        for (int64_t k0 = 0; k0 < p.K; k0 += p.group) {
            const int64_t g = k0 / p.group;
            const float s = op_to_float(static_cast<const T*>(p.scale)[g * p.lds + n]);
            const int z = p.zero != nullptr ? p.zero[g * p.ldz + n] & 15 : 8;
            for (int64_t k = k0 + lane; k < k0 + p.group && k < p.K; k += 32) {
                const int byte = p.Bq[n * p.ldbq + k / 2];
                const float w = s * static_cast<float>((k & 1 ? byte >> 4 : byte & 15) - z);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (m0 + i < p.M)
                        acc[i] += w * op_to_float(
                                          static_cast<const T*>(p.A)[(m0 + i) * p.lda + k]);
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
            if (lane == i && m0 + i < p.M) w4_store<T>(p, m0 + i, n, acc[i]);
        }
    }
}

// W as a K×N matrix of T (row stride ldo, a multiple of 8), for the dense GEMM
// on many rows of A.  Here (code - zero)·scale is rounded to T, as the tensor
// cores read 16-bit operands: at most half an ulp of each weight, an error of
// the size that storing C in T has.  One 128 k × 64 n tile per block
// iteration, turned round in shared memory; a thread decodes 16 k of two
// neighbouring rows of W, so that it stores pairs of n.  256 threads.
template <typename T>
__global__ void __launch_bounds__(256)
    tg_w4_dequant(const W4Params p, T* __restrict__ out, int64_t ldo) {
    __shared__ __align__(16) uint32_t tile[128][32 + 4];  // [k][n / 2]
    const int64_t tiles_n = (p.N + 63) / 64;
    const int64_t tiles = tiles_n * ((p.K + 127) / 128);
    const int pair = threadIdx.x & 31, kq = threadIdx.x >> 5;
    op_release_next();  // (a plain launch) the GEMM on the decoded weights may set up meanwhile
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t n0 = t % tiles_n * 64, k0 = t / tiles_n * 128;
        const int64_t kb = k0 + 16 * kq;
        float v[2][16];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int64_t n = n0 + 2 * pair + i;
            float s = 0.0f;
            int z = 8;
            uint32_t w[2] = {0, 0};
            if (n < p.N && kb < p.K) {
                const int64_t g = kb / p.group;
                s = op_to_float(static_cast<const T*>(p.scale)[g * p.lds + n]);
                if (p.zero != nullptr) z = p.zero[g * p.ldz + n] & 15;
                const uint8_t* src = p.Bq + n * p.ldbq + kb / 2;
                if (kb + 16 <= p.K) {
                    const uint2 u = *reinterpret_cast<const uint2*>(src);
                    w[0] = u.x;
                    w[1] = u.y;
                } else {
                    for (int j = 0; kb + 2 * j < p.K; ++j)
                        w[j >> 2] |= static_cast<uint32_t>(src[j]) << (8 * (j & 3));
                }
            }
#pragma unroll
            for (int j = 0; j < 16; ++j)
                v[i][j] = s * static_cast<float>(static_cast<int>(w[j >> 3] >> (4 * (j & 7)) & 15u) - z);
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            alignas(4) const T two[2] = {op_round<T>(v[0][j]), op_round<T>(v[1][j])};
            tile[16 * kq + j][pair] = *reinterpret_cast<const uint32_t*>(two);
        }
        __syncthreads();
        for (int c = threadIdx.x; c < 128 * 8; c += 256) {
            const int64_t k = k0 + (c >> 3), n = n0 + 8 * (c & 7);
            if (k >= p.K || n >= p.N) continue;
            const uint4 u = *reinterpret_cast<const uint4*>(&tile[c >> 3][4 * (c & 7)]);
            // ldo is N rounded up to 8: the whole chunk is inside the buffer
            *reinterpret_cast<uint4*>(out + k * ldo + n) = u;
        }
        __syncthreads();
    }
}

}  // namespace tg
