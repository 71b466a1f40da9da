// Products of 8-bit integers with a scale per row of A (token) and per row of B (channel):
//
//   C[m][n] = out( act( sa[m] · sb[n] · Σ_k a[m][k]·b[n][k] + bias[n] ) + R[m][n] )
#pragma once

#include <type_traits>

#include "op_device.cuh"
#include "tc_device.cuh"

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
// B's bytes are what counts, each read once.  They come by TMA (zeros past the edges) and go from
// shared memory into the operands of mma.sync, B's rows on the side of 16, the tokens on that of
// 8.  The order of sums of whole numbers is free everywhere:
//   - k: a lane takes 16 neighbouring bytes of a row, and the same bytes of a token;
//   - the warps of a block share its steps of 16 rows by 128 k evenly, whatever tiles they
//     belong to, and add what they have of a tile to its 32-bit sums in shared memory;
//   - the blocks of a cluster share k too, and in the end read one another's sums.  No scratch
//     in global memory.  (Sums added straight to those of another block, by its shared memory's
//     atomics: 512×8192 with 16 tokens 8.8 us.)
// Each warp has a ring of its own, which its first lane fills some steps ahead, across the
// borders of tiles.
//
// Up to 8 tokens the MMA is m16n8k32, s8 to s32.  Its rate is 273 products a cycle of an SM, 34
// bytes of B with 8 tokens: more than memory delivers (23).  For more tokens it is m16n8k16 in
// fp16, at 1028, on codes decoded in registers (five instructions for four) and tokens decoded
// into shared memory: whole numbers up to 2048 are exact in fp16, and their sums in fp32 up to
// 2^24, which eight steps do not pass; then they go to the 32-bit sums.  (16 tokens on s8:
// 16384×8192 in 40 us.  The tokens kept as bytes and decoded with each step's codes: 32 us.)
//
// Measured, bf16 results, random codes: 28672×4096 with 1 / 8 / 16 tokens 20.8 / 23.0 / 26.8 us (5.7
// TB/s with one), 16384×8192 24.3 / 25.5 / 28.9, 4096×28672 23.1 / 24.4 / 30.0 (16 tokens' fp16 takes
// clusters of eight, which hold 120 of the 152 SMs), 4096×4096 5.7 / 6.2 / 8.1, 1024×1024 3.1 / 3.8 / 3.9.
// Bound by memory, with some 3 us before the first codes and behind the last.  Three stages of a
// ring are enough (96 KB an SM): with six, 192 KB, more rows were under way at a time than memory
// keeps open, and one row of 16384×8192 took 27 us.

constexpr int kI8FewWarps = 16;
constexpr int kI8FewThreads = 32 * kI8FewWarps;
constexpr int kI8FewRows = 16;
constexpr int kI8FewK = 128;
constexpr int kI8FewStep = kI8FewRows * kI8FewK;
constexpr int kI8FewStages = 3;  // at most
constexpr int kI8FewRun = 8;     // steps whose sums are exact in fp32: 8 · 128 · 2^14 = 2^24
constexpr int kI8FewAhead = 3;   // steps of a warp, to L2 before the kernel may read
constexpr int kI8FewBars = kI8FewWarps * kI8FewStages * 8;

struct I8Few {
    I8Params p;
    uint64_t limit_ns;
    unsigned int* timeouts;  // set where a warp gives up on a wait
    int32_t inject;    // 1: block 0's first step is not fetched (for tests of the limit)
    int32_t cluster;   // blocks that share tiles and split k
    int32_t tiles;     // of 16 rows, in all
    int32_t chunks;    // of 128 k, in all
    int32_t stages;
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
// Four codes of a word as two pairs of fp16: with the sign turned, a byte u is code + 128, the
// fp16 number 0x6400 | u is 1024 + u, and 1152 less is the code, exactly.
__device__ __forceinline__ void i8_decode(uint32_t word, uint32_t& lo, uint32_t& hi) {
    const uint32_t u = word ^ 0x80808080u;
    const uint32_t off = 0x64806480u;  // 1152, twice
    uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(off));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(off));
}
__device__ __forceinline__ void i8_mma_half(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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
// A box of a 2-D tensor map to L2.
__device__ __forceinline__ void i8_prefetch(const void* map, uint32_t x, uint32_t y) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y)
                 : "memory");
}
__device__ __forceinline__ void i8_cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// NT: tokens / 8.  Grid: the clusters' blocks side by side.  Shared memory: the rings; their
// barriers; the tokens' bytes of this block's k; the sums of the cluster's tiles.
template <typename TC, int NT>
__global__ void __launch_bounds__(kI8FewThreads, 1)
    tg_gemm_i8_few(const __grid_constant__ I8Few q, const __grid_constant__ CUtensorMap codes) {
    constexpr bool kHalf = NT > 1, kKeep = NT == 2 || NT == 4;
    extern __shared__ __align__(1024) unsigned char i8_dynamic[];
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
    const uint32_t base = (op_smem(i8_dynamic) + 1023) & ~1023u;
    unsigned char* const shared = i8_dynamic + (base - op_smem(i8_dynamic));
    const uint32_t ring = base + warp * q.stages * kI8FewStep;
    unsigned char* const behind = shared + kI8FewWarps * q.stages * kI8FewStep;  // the rings
    const uint32_t bars = op_smem(behind) + warp * kI8FewStages * 8;
    unsigned char* const x_all = behind + kI8FewBars;
    int* const sums = reinterpret_cast<int*>(x_all + tokens * q.x_pitch);
    op_release_next();
    if (lane == 0) {
        for (int s = 0; s < q.stages; ++s) op_bar_init(bars + 8 * s, 1);
        op_bar_init_done();
    }
    for (int i = threadIdx.x; i < tokens * q.sums_pitch; i += kI8FewThreads) sums[i] = 0;
    __syncwarp();

    // This warp's steps: an even share of the block's, tile by tile, k inside.
    const int all = tiles * chunks;
    const int u0 = static_cast<int>(int64_t{all} * warp / kI8FewWarps);
    const int steps = static_cast<int>(int64_t{all} * (warp + 1) / kI8FewWarps) - u0;
    struct Place {
        int tile, chunk;
    };
    auto advance = [&](Place& at) {
        if (++at.chunk == chunks) at.chunk = 0, ++at.tile;
    };
    Place next{u0 / chunks, u0 % chunks}, here = next;
    int fill = 0, issued = 0;  // the stage that is filled next
    auto fetch = [&] {
        if (issued == steps) return;
        if (lane == 0 && !(q.inject == 1 && blockIdx.x == 0 && issued == 0)) {
            const uint32_t bar = bars + 8 * fill;
            op_bar_expect(bar, kI8FewStep);
            op_tma_2d(ring + fill * kI8FewStep, &codes, bar, (c0 + next.chunk) * kI8FewK,
                      (tile0 + next.tile) * kI8FewRows);
        }
        advance(next);
        ++issued;
        fill = fill + 1 == q.stages ? 0 : fill + 1;
    };
    if (lane == 0) {
        // While the kernel before this one ends, the first steps come as far as L2 (no value is
        // taken yet: that kernel may still write them).
        Place soon = next;
        for (int s = 0; s < kI8FewAhead && s < steps; ++s, advance(soon))
            i8_prefetch(&codes, (c0 + soon.chunk) * kI8FewK, (tile0 + soon.tile) * kI8FewRows);
    }
    op_wait_previous();
    for (int s = 0; s < q.stages; ++s) fetch();
    {  // the tokens
        const bool wide = (reinterpret_cast<uintptr_t>(p.A) & 15) == 0 && p.lda % 16 == 0;
        const int pieces = kI8FewK / 16 * chunks;
        if (!kHalf && wide) {
            for (int m = 0; m < tokens; ++m)
                for (int i = threadIdx.x; i < pieces; i += kI8FewThreads) {
                    const int64_t k = int64_t{c0} * kI8FewK + 16 * i;
                    const int8_t* a = p.A + m * p.lda;
                    unsigned char* to = x_all + m * q.x_pitch + 16 * i;
                    if (k + 16 <= p.K)
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(op_smem(to)), "l"(a + k)
                                     : "memory");
                    else if (k < p.K)  // zeros past the end (single bytes: 7 tokens of K = 4099 1.4 us more)
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(op_smem(to)), "l"(a + k),
                                     "r"(static_cast<int>(p.K - k))
                                     : "memory");
                    else
                        *reinterpret_cast<uint4*>(to) = make_uint4(0, 0, 0, 0);
                }
        } else {
            // four pieces of a thread under way at a time
            for (int i0 = threadIdx.x; i0 < tokens * pieces; i0 += 4 * kI8FewThreads) {
                uint4 v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int i = i0 + j * kI8FewThreads, m = i / pieces;
                    const int64_t k = int64_t{c0} * kI8FewK + 16 * (i - m * pieces);
                    if (m < tokens)
                        v[j] = wide && k + 16 <= p.K ? *reinterpret_cast<const uint4*>(p.A + m * p.lda + k)
                                                     : i8_bytes(p.A + m * p.lda, k, p.K);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int i = i0 + j * kI8FewThreads, m = i / pieces, piece = i - m * pieces;
                    if (m >= tokens) break;
                    if constexpr (kHalf) {
                        uint4 y[2];
                        i8_decode(v[j].x, y[0].x, y[0].y);
                        i8_decode(v[j].y, y[0].z, y[0].w);
                        i8_decode(v[j].z, y[1].x, y[1].y);
                        i8_decode(v[j].w, y[1].z, y[1].w);
                        // of each 64 k the first halves of the 16s, then the others
                        uint4* to =
                            reinterpret_cast<uint4*>(x_all + m * q.x_pitch + 128 * (piece >> 2) + 16 * (piece & 3));
                        to[0] = y[0];
                        to[4] = y[1];
                    } else {
                        *reinterpret_cast<uint4*>(x_all + m * q.x_pitch + 16 * piece) = v[j];
                    }
                }
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    }
    __syncthreads();

    // A lane's MMA row g is row r of the tile (g + 8: r + 8): so the eight lanes that read at a
    // time find their 16 bytes, swizzled by r, in all banks.
    const int r = (g >> 1) + 4 * (g & 1);
    typename std::conditional<kHalf, float, int>::type c[NT][4];
    int whole[kKeep ? NT : 1][4];  // kKeep: what fp32 does not hold exactly
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) c[i][j] = 0;
#pragma unroll
    for (int i = 0; i < (kKeep ? NT : 1); ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) whole[i][j] = 0;
    const uint32_t sums_at = op_smem(sums);
    auto flush = [&](int tile) {  // c[.][0, 1]: row g, tokens 2t and 2t + 1; [2, 3]: row g + 8
        const uint32_t to = sums_at + 4 * (kI8FewRows * tile + r);
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int m = 8 * i + 2 * t + (j & 1);
                if (m < tokens)
                    asm volatile("red.relaxed.cta.shared::cta.add.s32 [%0], %1;" ::"r"(
                                     to + 4 * (m * q.sums_pitch + 8 * (j >> 1))),
                                 "r"(static_cast<int>(c[i][j]) + (kKeep ? whole[kKeep ? i : 0][j] : 0))
                                 : "memory");
                c[i][j] = 0;
                if (kKeep) whole[kKeep ? i : 0][j] = 0;
            }
    };
    const unsigned char* x = x_all + g * q.x_pitch + 16 * t;
    int slot = 0, used = 0, run = 0;  // run: steps in c
    uint32_t parity = 0;
    bool lost = false;
    while (used < steps) {
        const bool ok = op_bar_wait(bars + 8 * slot, parity, q.limit_ns);
        if (!__all_sync(0xffffffffu, ok)) {
            lost = true;
            break;
        }
        const uint32_t row = ring + slot * kI8FewStep + r * kI8FewK;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t at = row + (((4 * h + t) ^ r) << 4);
            const uint4 v = tc_lds128(at), w = tc_lds128(at + 8 * kI8FewK);
            if constexpr (kHalf) {
                const uint32_t vs[4] = {v.x, v.y, v.z, v.w}, ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int f = 0; f < 2; ++f) {  // 8 of the 16 bytes
                    uint32_t a[2][4];
#pragma unroll
                    for (int o = 0; o < 2; ++o) {
                        i8_decode(vs[2 * f + o], a[o][0], a[o][2]);
                        i8_decode(ws[2 * f + o], a[o][1], a[o][3]);
                    }
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        uint4 b = make_uint4(0, 0, 0, 0);
                        if (8 * j + g < tokens)
                            b = *reinterpret_cast<const uint4*>(x + 8 * j * q.x_pitch + 2 * kI8FewK * here.chunk +
                                                                128 * h + 64 * f);
                        i8_mma_half(c[j], a[0][0], a[0][1], a[0][2], a[0][3], b.x, b.y);
                        i8_mma_half(c[j], a[1][0], a[1][1], a[1][2], a[1][3], b.z, b.w);
                    }
                }
            } else {
                uint4 a = make_uint4(0, 0, 0, 0);
                if (g < tokens) a = *reinterpret_cast<const uint4*>(x + kI8FewK * here.chunk + 64 * h);
                i8_mma(c[0], v.x, w.x, v.y, w.y, a.x, a.y);
                i8_mma(c[0], v.z, w.z, v.w, w.w, a.z, a.w);
            }
        }
        ++used;
        __syncwarp();  // all lanes have used the stage, which is filled again
        fetch();
        const int tile = here.tile;
        advance(here);
        if (here.tile != tile || used == steps || (kHalf && !kKeep && ++run == kI8FewRun)) {
            flush(tile);
            run = 0;
        } else if (kKeep && ++run == kI8FewRun) {
#pragma unroll
            for (int i = 0; i < (kKeep ? NT : 1); ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    whole[i][j] += static_cast<int>(c[i][j]);
                    c[i][j] = 0;
                }
            run = 0;
        }
        if (++slot == q.stages) slot = 0, parity ^= 1;
    }
    if (lost) {
        // copies under way have to land before the block ends
        bool ok = true;
        for (int i = used; ok && lane == 0 && i < issued; ++i)
            ok = op_bar_wait(bars + 8 * (i % q.stages), i / q.stages & 1, kTcLandNs);
        __syncwarp();
        if (lane == 0) atomicOr(q.timeouts, kOpTimeoutI8);
    }
    if (q.cluster > 1)
        i8_cluster_sync();  // the other blocks' sums are complete, too
    else
        __syncthreads();

    // The blocks of a cluster finish its tiles in turn, each with the sums of all.
    const int rows = (tiles - rank + q.cluster - 1) / q.cluster * kI8FewRows;
    for (int i = threadIdx.x; i < rows * tokens; i += kI8FewThreads) {
        const int m = i / rows, o = i - m * rows;
        const int place = (o / kI8FewRows * q.cluster + rank) * kI8FewRows + o % kI8FewRows;
        const int64_t n = int64_t{tile0} * kI8FewRows + place;
        if (n >= p.N) continue;
        int sum = 0;
        if (q.cluster > 1) {
            const uint32_t at = sums_at + 4 * (m * q.sums_pitch + place);
            for (int b = 0; b < q.cluster; ++b) {
                uint32_t there;
                int v;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(at), "r"(b));
                asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(there) : "memory");
                sum += v;
            }
        } else {
            sum = sums[m * q.sums_pitch + place];
        }
        float y = i8_value(p, static_cast<float>(sum), p.sa[m], p.sb[n], p.bias != nullptr ? p.bias[n] : 0.0f);
        if (p.resid != nullptr) y += op_to_float((static_cast<const TC*>(p.resid) + m * p.ldr)[n]);
        (static_cast<TC*>(p.C) + m * p.ldc)[n] = op_round<TC>(y);
    }
    if (q.cluster > 1) i8_cluster_sync();  // no block leaves while others read its sums
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
