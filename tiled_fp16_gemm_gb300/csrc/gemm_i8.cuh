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

// ------------------------------------------------------------------ few rows of A
//
// Up to 16 tokens: B's bytes are what counts, each read once and straight into the operands of
// mma.sync (m16n8k32, s8 to s32), B's rows on the side of 16, the tokens on that of 8.  The sums
// are 32-bit integers, exact in any order, so the order is free everywhere:
//   - k: a lane takes 16 neighbouring bytes of a row for two MMAs, and the same bytes of a token;
//   - the warps of a block share out steps of 16 rows by 64 k one by one, whatever tile they
//     belong to, and add what they have of a tile to its sums in shared memory;
//   - the blocks of a cluster share k too, and add to the sums in the shared memory of the
//     tile's owner.  No scratch in global memory, one join at the end.
// A warp has kI8Depth steps under way in registers (48 a lane), across the borders of tiles.
//
// The MMA's rate here is 273 products a cycle of an SM, 34 bytes of B: for 8 tokens more than
// memory delivers (23), for 16 half of it.

constexpr int kI8FewWarps = 16;
constexpr int kI8FewThreads = 32 * kI8FewWarps;
constexpr int kI8Depth = 6;

struct I8Few {
    I8Params p;
    int32_t cluster;   // blocks that share tiles and split k
    int32_t rounds;    // tiles of 16 rows of a cluster, at most
    int32_t tiles;     // in all
    int32_t chunks;    // of 64 k, in all
    int32_t x_pitch;   // bytes of a token in shared memory
    int32_t sums_pitch;  // words of a token's sums
};

__device__ __forceinline__ void i8_mma(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Bytes that are read once.
__device__ __forceinline__ uint4 i8_stream(const void* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.L2::128B.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
// 16 bytes of a row from byte k on, 0 past its `n`: of any alignment, and nothing outside it read.
__device__ __forceinline__ uint4 i8_bytes(const int8_t* row, int64_t k, int64_t n) {
    uint32_t w[4] = {0, 0, 0, 0};
    const int8_t* at = row + k;
    const uint32_t skip = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(at) & 3);
    if (k >= skip && k + 20 - skip <= n) {
        const uint32_t* words = reinterpret_cast<const uint32_t*>(at - skip);
        uint32_t v[5];
#pragma unroll
        for (int i = 0; i < 5; ++i) v[i] = words[i];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(v[i], v[i + 1], 8 * skip);
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (k + i < n) w[i / 4] |= static_cast<uint32_t>(static_cast<uint8_t>(at[i])) << (8 * (i % 4));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void i8_cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// NT: tokens / 8.  Grid: the clusters' blocks side by side.  Shared memory: the tokens' bytes
// of this block's k, then the sums of the tiles that it owns (every cluster-th of the cluster's).
template <typename TC, int NT>
__global__ void __launch_bounds__(kI8FewThreads, 1) tg_gemm_i8_few(const __grid_constant__ I8Few q) {
    extern __shared__ __align__(16) unsigned char i8_shared[];
    const I8Params& p = q.p;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int tokens = static_cast<int>(p.M);
    const int rank = blockIdx.x % q.cluster, cluster_no = blockIdx.x / q.cluster;
    const int clusters = gridDim.x / q.cluster;
    // this cluster's tiles, this block's k
    const int tile0 = q.tiles / clusters * cluster_no + min(q.tiles % clusters, cluster_no);
    const int tiles = q.tiles / clusters + (cluster_no < q.tiles % clusters ? 1 : 0);
    const int c0 = static_cast<int>(int64_t{q.chunks} * rank / q.cluster);
    const int chunks = static_cast<int>(int64_t{q.chunks} * (rank + 1) / q.cluster) - c0;
    int* sums = reinterpret_cast<int*>(i8_shared + tokens * q.x_pitch);
    op_release_next();
    for (int i = threadIdx.x; i < tokens * q.sums_pitch; i += kI8FewThreads) sums[i] = 0;
    op_wait_previous();

    // a lane's bytes of a step: rows g and g + 8 of the tile (the last row again past the last)
    const int dt = kI8FewWarps / chunks, dc = kI8FewWarps % chunks;
    const bool ragged = p.K % 16 != 0;  // the last row's last bytes are read one by one
    struct Place {
        int tile, chunk;
    };
    auto advance = [&](Place& at) {
        at.tile += dt;
        at.chunk += dc;
        if (at.chunk >= chunks) at.chunk -= chunks, ++at.tile;
    };
    auto load = [&](const Place& at, uint4 (&v)[2]) {
        const int64_t k = int64_t{c0 + at.chunk} * 64 + 16 * t;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            int64_t n = int64_t{tile0 + at.tile} * 16 + g + 8 * h;
            if (n >= p.N) n = p.N - 1;
            if (at.tile >= tiles || k >= p.K)
                v[h] = make_uint4(0, 0, 0, 0);
            else if (ragged && n == p.N - 1 && k + 16 > p.K)
                v[h] = i8_bytes(p.B + n * p.ldb, k, p.K);
            else
                v[h] = i8_stream(p.B + n * p.ldb + k);
        }
    };
    Place next{warp / chunks, warp % chunks}, here = next;
    uint4 v[kI8Depth][2];
#pragma unroll
    for (int i = 0; i < kI8Depth; ++i) {
        load(next, v[i]);
        advance(next);
    }
    {  // the tokens
        const bool wide = (reinterpret_cast<uintptr_t>(p.A) & 15) == 0 && p.lda % 16 == 0;
        const int pieces = 4 * chunks;
        for (int i = threadIdx.x; i < tokens * pieces; i += kI8FewThreads) {
            const int m = i / pieces, piece = i - m * pieces;
            const int64_t k = int64_t{c0} * 64 + 16 * piece;
            const int8_t* a = p.A + m * p.lda;
            *reinterpret_cast<uint4*>(i8_shared + m * q.x_pitch + 16 * piece) =
                wide && k + 16 <= p.K ? *reinterpret_cast<const uint4*>(a + k) : i8_bytes(a, k, p.K);
        }
    }
    if (q.cluster > 1)
        i8_cluster_sync();  // (the owners' sums are zero, too)
    else
        __syncthreads();

    int c[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) c[i][j] = 0;
    const uint32_t sums_at = op_smem(sums);
    auto flush = [&](int tile) {  // c[.][0, 1]: row g, tokens 2t and 2t + 1; [2, 3]: row g + 8
        const int slot = q.cluster > 1 ? tile / q.cluster : tile;
        uint32_t to = sums_at + 4 * (16 * slot + g);
        if (q.cluster > 1)
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(to), "r"(tile - slot * q.cluster));
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int m = 8 * i + 2 * t + (j & 1);
                if (m < tokens)
                    asm volatile("red.relaxed.cluster.shared::cluster.add.s32 [%0], %1;" ::"r"(
                                     to + 4 * (m * q.sums_pitch + 8 * (j >> 1))),
                                 "r"(c[i][j])
                                 : "memory");
                c[i][j] = 0;
            }
    };
    const unsigned char* x = i8_shared + g * q.x_pitch + 16 * t;
    while (here.tile < tiles) {
#pragma unroll
        for (int i = 0; i < kI8Depth; ++i) {
            if (here.tile < tiles) {
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    uint4 a = make_uint4(0, 0, 0, 0);
                    if (8 * j + g < tokens)
                        a = *reinterpret_cast<const uint4*>(x + 8 * j * q.x_pitch + 64 * here.chunk);
                    i8_mma(c[j], v[i][0].x, v[i][1].x, v[i][0].y, v[i][1].y, a.x, a.y);
                    i8_mma(c[j], v[i][0].z, v[i][1].z, v[i][0].w, v[i][1].w, a.z, a.w);
                }
                load(next, v[i]);
                advance(next);
                const int tile = here.tile;
                advance(here);
                if (here.tile != tile) flush(tile);
            }
        }
    }
    if (q.cluster > 1)
        i8_cluster_sync();  // and no block leaves before its sums have come
    else
        __syncthreads();

    const int owned = q.cluster > 1 ? (tiles - rank + q.cluster - 1) / q.cluster : tiles;
    for (int i = threadIdx.x; i < owned * 16 * tokens; i += kI8FewThreads) {
        const int m = i / (owned * 16), r = i - m * owned * 16;
        const int64_t n = int64_t{tile0 + r / 16 * q.cluster + rank} * 16 + r % 16;
        if (n >= p.N) continue;
        float y = i8_value(p, static_cast<float>(sums[m * q.sums_pitch + r]), p.sa[m], p.sb[n],
                           p.bias != nullptr ? p.bias[n] : 0.0f);
        if (p.resid != nullptr) y += op_to_float((static_cast<const TC*>(p.resid) + m * p.ldr)[n]);
        (static_cast<TC*>(p.C) + m * p.ldc)[n] = op_round<TC>(y);
    }
}

// ------------------------------------------------------------------ any size

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
