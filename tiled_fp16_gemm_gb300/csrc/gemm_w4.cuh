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

#include <type_traits>

#include "op_device.cuh"
#include "tc_device.cuh"

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

// ------------------------------------------------------------------ few rows of A
//
// The weights are the A operand of mma.m16n8k16 (16 rows of W by 16 k), the rows of
// A ("tokens") its columns.  What bounds this is the decoding: at 6.8 TB/s an SM gets
// 47 codes per clock, so 2048 codes (32 lanes, 8 words each) may cost no more than
// about 130 instructions, all in all.  With w a word of 8 codes c0..c7 (k ascending):
//   fp16: (w & 0x000f000f) | 0x6400.. is the pair (1024 + c0, 1024 + c4), minus
//         (1024 + z) exactly c - z; (w & 0x00f000f0) | 0x6400.. is 1024 + 16·c1,
//         and ·1/16 - (64 + z) again exactly c1 - z; w >> 8 gives the other four;
//   bf16: w >> 4i in the same way around 128, whose last place is 1.
// So every operand is exactly c - z, every product exact, and the sums fp32; after
// each group its sum is scaled in fp32 and added up.  The pairs are (c_i, c_i+4):
// the block holds its k of A in shared memory with each 8 values in that order.
//
// A warp takes 32 rows of W by 128 k at a time (2 KB of codes), through a ring of its
// own in shared memory that its first lane fills by TMA a few steps ahead (zeros past
// the edges): the warps of a block meet only where they join their sums.  A block of 16 warps is wn tiles of 32 rows by
// wk k-pieces, and goes over its tiles round by round; the blocks of a cluster share
// the tiles and split k, and join over distributed shared memory at the end.  All sums
// are joined in a fixed order, with no scratch in global memory.
//
// Measured, one row: 28672×4096 bf16, G = 128, 18.5 us; 16384×8192 fp16 18.5 us (3.3 and
// 3.8 TB/s); 4096×28672 fp16, G = 32, 18.4 us; 1024×1024 3.7 us.  8 rows of 16384×8192
// 23.8 us.  Bound by latency: some 350 instructions for 4096 codes, issued at 2.1 to 2.3 of
// the 4 a cycle that an SM could; its 16 warps (96 to 128 registers) do not cover the way
// from a load over the decoding to the MMA.

constexpr int kW4Warps = 16;
constexpr int kW4Threads = 32 * kW4Warps;
constexpr int kW4Rows = 32;   // of W, in a warp's tile
constexpr int kW4K = 128;     // k of a step
constexpr int kW4StepCodes = kW4Rows * kW4K / 2;

template <int G>
struct W4Step {
    static constexpr int kGroups = kW4K / G;
    static constexpr int kScaleBytes = kGroups * kW4Rows * 2;
    static constexpr int kZeroBytes = kGroups * kW4Rows;
    // codes, scales, zero points; TMA writes to multiples of 128 bytes, and its
    // 64-byte swizzle repeats every 512
    static constexpr int kZeroAt = kW4StepCodes + 256;
    static constexpr int kBytes = 2560;
    static_assert(kScaleBytes <= 256 && kZeroAt + kZeroBytes <= kBytes, "a step's place");
};


struct W4Launch {
    W4Params p;
    uint64_t limit_ns;
    unsigned int* timeouts;  // set where a warp gives up on a wait
    int32_t inject;    // 1: block 0's first fetch is left out (for tests of the limit)
    int32_t wn, wk;    // tiles of a block at a time, k-pieces
    int32_t tokens;    // rows of A per block
    int32_t steps;     // k steps in all
    int32_t cluster;   // blocks that share tiles and split k
    int32_t clusters;  // per block of tokens
    int32_t tiles;     // of 32 rows of W
    int32_t rounds;    // tiles of a block / wn
    int32_t stages;    // 2 to 4
    int32_t x_bytes;   // A in shared memory
    int32_t join_bytes;  // the k-pieces' sums
};

__device__ __forceinline__ uint32_t w4_lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}

// (a & mask) | bits in one instruction.
__device__ __forceinline__ uint32_t w4_and_or(uint32_t a, uint32_t mask, uint32_t bits) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "r"(mask), "r"(bits));
    return d;
}

template <typename T>
struct W4Decode;

template <>
struct W4Decode<__half> {
    uint32_t lo, hi;  // -(1024 + z), -(64 + z), twice each
    __device__ __forceinline__ explicit W4Decode(uint32_t z)
        : lo(0xE400E400u + z * 0x00010001u), hi(0xD400D400u + z * 0x00100010u) {}
    // v[i] = (c_i - z, c_i+4 - z)
    __device__ __forceinline__ void operator()(uint32_t w, uint32_t (&v)[4]) const {
        const uint32_t u = w >> 8;
        v[0] = add(w4_and_or(w, 0x000f000fu, 0x64006400u));
        v[1] = fma(w4_and_or(w, 0x00f000f0u, 0x64006400u));
        v[2] = add(w4_and_or(u, 0x000f000fu, 0x64006400u));
        v[3] = fma(w4_and_or(u, 0x00f000f0u, 0x64006400u));
    }
    __device__ __forceinline__ uint32_t add(uint32_t a) const {
        uint32_t d;
        asm("add.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(lo));
        return d;
    }
    __device__ __forceinline__ uint32_t fma(uint32_t a) const {
        uint32_t d;
        asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(0x2C002C00u), "r"(hi));
        return d;
    }
};

template <>
struct W4Decode<__nv_bfloat16> {
    uint32_t lo;  // -(128 + z), twice
    __device__ __forceinline__ explicit W4Decode(uint32_t z) : lo(0xC300C300u + z * 0x00010001u) {}
    __device__ __forceinline__ void operator()(uint32_t w, uint32_t (&v)[4]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t a = w4_and_or(w >> (4 * i), 0x000f000fu, 0x43004300u);
            asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(v[i]) : "r"(a), "r"(lo));
        }
    }
};

// d = a·b + c
template <typename T>
__device__ __forceinline__ void w4_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                       uint32_t a3, uint32_t b0, uint32_t b1, float c0, float c1,
                                       float c2, float c3) {
    if constexpr (std::is_same<T, __half>::value)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
            "{%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2),
              "f"(c3));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
            "{%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2),
              "f"(c3));
}

// Shared address `a` of block `rank` of the cluster, read from here.
__device__ __forceinline__ float w4_cluster_load(uint32_t a, int rank) {
    uint32_t m;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(m) : "memory");
    return v;
}

// grid: x = clusters × cluster (the blocks of a cluster side by side), y = blocks of
// tokens.  Shared memory: A; the warps' rings; the k-pieces' sums; where there is a
// cluster, the sums of all tiles.
template <typename T, int G, int NT, bool ZERO>
__global__ void __launch_bounds__(kW4Threads, 1) tg_gemm_w4(const __grid_constant__ W4Launch q, const __grid_constant__ CUtensorMap codes,
               const __grid_constant__ CUtensorMap scales, const __grid_constant__ CUtensorMap zeros) {
    using Step = W4Step<G>;
    extern __shared__ __align__(1024) unsigned char w4_shared[];
    const W4Params& p = q.p;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int wn = warp / q.wk, wk = warp % q.wk;
    const int rank = blockIdx.x % q.cluster, cluster_no = blockIdx.x / q.cluster;
    const int64_t m0 = int64_t{blockIdx.y} * q.tokens;
    const int tokens = static_cast<int>(p.M - m0 < q.tokens ? p.M - m0 : q.tokens);
    const int s0 = static_cast<int>(int64_t{q.steps} * rank / q.cluster);
    const int s1 = static_cast<int>(int64_t{q.steps} * (rank + 1) / q.cluster);
    const int mine = s1 - s0 > wk ? (s1 - s0 - wk + q.wk - 1) / q.wk : 0;  // steps per tile

    // the rings' barriers, then A
    const uint32_t x_base = op_smem(w4_shared) + kW4Warps * 4 * 8;
    const uint32_t bars = op_smem(w4_shared) + warp * 4 * 8;
    const uint32_t ring = x_base + q.x_bytes + warp * q.stages * Step::kBytes;
    op_release_next();
    if (lane == 0) {
        for (int s = 0; s < q.stages; ++s) op_bar_init(bars + 8 * s, 1);
        op_bar_init_done();
    }
    __syncwarp();
    op_wait_previous();

    // ---- filling the ring: tile after tile, step after step
    const uint32_t rows = static_cast<uint32_t>(p.N);
    int f_round = 0, f_step = 0, f_slot = 0;  // what is fetched next
    uint32_t f_n = (cluster_no * q.wn + wn) * kW4Rows;
    const uint32_t tile_step = static_cast<uint32_t>(q.clusters) * q.wn * kW4Rows;
    auto fetch = [&] {
        if (f_round >= q.rounds || f_n >= rows) return;
        if (lane == 0) {
            const uint32_t step = s0 + wk + f_step * q.wk;
            const uint32_t to = ring + f_slot * Step::kBytes, bar = bars + 8 * f_slot;
            if (!(q.inject == 1 && blockIdx.x == 0 && f_round == 0 && f_step == 0)) {
                op_bar_expect(bar, kW4StepCodes + Step::kScaleBytes + (ZERO ? Step::kZeroBytes : 0));
                op_tma_2d(to, &codes, bar, step * (kW4K / 2), f_n);
                op_tma_2d(to + kW4StepCodes, &scales, bar, f_n, step * Step::kGroups);
                if (ZERO) op_tma_2d(to + Step::kZeroAt, &zeros, bar, f_n, step * Step::kGroups);
            }
        }
        f_slot = f_slot + 1 == q.stages ? 0 : f_slot + 1;
        if (++f_step == mine) {
            f_step = 0;
            ++f_round;
            f_n += tile_step;
        }
    };
    if (mine > 0)
        for (int s = 0; s < q.stages - 1; ++s) fetch();

    // ---- A: [32 k][token][4 lanes][x0 x4 x2 x6 x1 x5 x3 x7]
    {
        const int chunks = (s1 - s0) * (kW4K / 8);
        const int64_t k_first = int64_t{s0} * kW4K;
        const bool vec = (reinterpret_cast<uintptr_t>(p.A) & 15) == 0 && p.lda % 8 == 0;
        for (int m = 0; m < tokens; ++m) {
            const T* a = static_cast<const T*>(p.A) + (m0 + m) * p.lda + k_first;
            for (int c = threadIdx.x; c < chunks; c += kW4Threads) {
                uint4 x;
                if (vec && k_first + 8 * c + 8 <= p.K) {
                    x = *reinterpret_cast<const uint4*>(a + 8 * c);
                } else {
                    uint32_t h[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        h[i] = k_first + 8 * c + i < p.K
                                   ? reinterpret_cast<const uint16_t*>(a)[8 * c + i]
                                   : 0;
                    x = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16,
                                   h[6] | h[7] << 16);
                }
                uint4 v;
                v.x = __byte_perm(x.x, x.z, 0x5410);
                v.y = __byte_perm(x.y, x.w, 0x5410);
                v.z = __byte_perm(x.x, x.z, 0x7632);
                v.w = __byte_perm(x.y, x.w, 0x7632);
                *reinterpret_cast<uint4*>(w4_shared + kW4Warps * 4 * 8 + ((c >> 2) * q.tokens + m) * 64 +
                                           (c & 3) * 16) = v;
            }
        }
        __syncthreads();
    }

    const uint32_t x_pitch = q.tokens * 64;  // of 32 k
    uint32_t x_lane[NT];  // this lane's token of each column tile (the last one past the end)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int m = 8 * nt + g;
        x_lane[nt] = x_base + (m < tokens ? m : tokens - 1) * 64 + t * 16;
    }
    const uint32_t w_lane = g * 64 + ((g >> 1 & 3) << 4) + t * 4;
    float* pieces = reinterpret_cast<float*>(w4_shared + kW4Warps * 4 * 8 + q.x_bytes +
                                             kW4Warps * q.stages * Step::kBytes);
    float* results = pieces + q.join_bytes / 4;
    int slot = 0;
    uint32_t parity = 0;
    bool given_up = false, lost = false;
    for (int round = 0; round < q.rounds; ++round) {
        const int64_t n0 = ((int64_t{round} * q.clusters + cluster_no) * q.wn + wn) * kW4Rows;
        float sum[2][NT][4];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) sum[mt][nt][i] = 0.0f;
        uint32_t x_at = wk * 4 * x_pitch;
        if (n0 < p.N) {
            for (int i = 0; i < mine; ++i) {
                if (!lost && !op_bar_wait(bars + 8 * slot, parity, q.limit_ns)) {
                    // reported; nothing more is fetched once copies do not come at all
                    given_up = true;
                    lost = !op_bar_wait(bars + 8 * slot, parity, kTcLandNs);
                }
                lost = __any_sync(0xffffffffu, lost);
                __syncwarp();  // all lanes have read the slot before, which is filled again
                if (!lost) fetch();
                const uint32_t at = ring + slot * Step::kBytes;
                const uint32_t wl = at + w_lane;
                const unsigned char* tail = w4_shared + (at - op_smem(w4_shared)) + kW4StepCodes;
#pragma unroll
                for (int gr = 0; gr < Step::kGroups; ++gr) {
                    uint32_t z[2][2];
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            z[mt][h] = ZERO ? tail[Step::kZeroAt - kW4StepCodes + gr * kW4Rows + 16 * mt + 8 * h + g] & 15u
                                            : 8u;
                    float acc[2][NT][4];
#pragma unroll
                    for (int jj = 0; jj < G / 32; ++jj) {
                        const int j = gr * (G / 32) + jj;
                        uint32_t v[2][2][4];
#pragma unroll
                        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const W4Decode<T> decode(z[mt][h]);
                                decode(w4_lds32((wl ^ (j << 4)) + (16 * mt + 8 * h) * 64), v[mt][h]);
                            }
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const uint4 x = tc_lds128(x_lane[nt] + x_at + j * x_pitch);
#pragma unroll
                            for (int mt = 0; mt < 2; ++mt) {
                                float(&a)[4] = acc[mt][nt];
                                if (jj == 0)
                                    w4_mma<T>(a, v[mt][0][0], v[mt][1][0], v[mt][0][2], v[mt][1][2],
                                              x.x, x.y, 0.0f, 0.0f, 0.0f, 0.0f);
                                else
                                    w4_mma<T>(a, v[mt][0][0], v[mt][1][0], v[mt][0][2], v[mt][1][2],
                                              x.x, x.y, a[0], a[1], a[2], a[3]);
                                w4_mma<T>(a, v[mt][0][1], v[mt][1][1], v[mt][0][3], v[mt][1][3], x.z,
                                          x.w, a[0], a[1], a[2], a[3]);
                            }
                        }
                    }
                    const T* sc = reinterpret_cast<const T*>(tail) + gr * kW4Rows + g;
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt) {
                        const float sa = op_to_float(sc[16 * mt]), sb = op_to_float(sc[16 * mt + 8]);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            sum[mt][nt][0] = fmaf(sa, acc[mt][nt][0], sum[mt][nt][0]);
                            sum[mt][nt][1] = fmaf(sa, acc[mt][nt][1], sum[mt][nt][1]);
                            sum[mt][nt][2] = fmaf(sb, acc[mt][nt][2], sum[mt][nt][2]);
                            sum[mt][nt][3] = fmaf(sb, acc[mt][nt][3], sum[mt][nt][3]);
                        }
                    }
                }
                x_at += q.wk * 4 * x_pitch;
                if (++slot == q.stages) slot = 0, parity ^= 1;
            }
        }
        // ---- joining the k-pieces of a tile, lane by lane
        if (q.wk > 1) {
            const int threads = 32 * q.wk;
            if (wk > 0) {
                float* to = pieces + (wn * (q.wk - 1) + wk - 1) * (256 * NT) + lane;
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < 4; ++i) to[((mt * NT + nt) * 4 + i) * 32] = sum[mt][nt][i];
            }
            if (threads == kW4Threads)
                __syncthreads();
            else
                asm volatile("bar.sync %0, %1;" ::"r"(wn + 1), "r"(threads) : "memory");
            if (wk == 0) {
                for (int k = 1; k < q.wk; ++k) {
                    const float* from = pieces + (wn * (q.wk - 1) + k - 1) * (256 * NT) + lane;
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                sum[mt][nt][i] += from[((mt * NT + nt) * 4 + i) * 32];
                }
            }
            if (round + 1 < q.rounds) {  // before the next round's sums come
                if (threads == kW4Threads)
                    __syncthreads();
                else
                    asm volatile("bar.sync %0, %1;" ::"r"(wn + 1), "r"(threads) : "memory");
            }
        }
        if (wk == 0) {
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int m = 8 * nt + 2 * t + (i & 1), r = 16 * mt + g + 8 * (i >> 1);
                        if (m >= tokens) continue;
                        if (q.cluster > 1)
                            results[((round * q.wn + wn) * q.tokens + m) * kW4Rows + r] = sum[mt][nt][i];
                        else if (n0 + r < p.N)
                            w4_store<T>(p, m0 + m, n0 + r, sum[mt][nt][i]);
                    }
        }
    }
    if (given_up && lane == 0) atomicOr(q.timeouts, kOpTimeoutW4);
    if (q.cluster > 1) {
        tc_cluster_sync();
        const uint32_t from = op_smem(results);
        const int outs = q.rounds * q.wn * q.tokens * kW4Rows;
        for (int i = rank * kW4Threads + threadIdx.x; i < outs; i += q.cluster * kW4Threads) {
            const int r = i % kW4Rows, m = i / kW4Rows % q.tokens;
            const int tile = i / (kW4Rows * q.tokens);  // of this block: round · wn + wn
            const int64_t n =
                ((int64_t{tile / q.wn} * q.clusters + cluster_no) * q.wn + tile % q.wn) * kW4Rows + r;
            if (m >= tokens || n >= p.N) continue;
            float a = 0.0f;
            for (int k = 0; k < q.cluster; ++k) a += w4_cluster_load(from + i * 4, k);
            w4_store<T>(p, m0 + m, n, a);
        }
        tc_cluster_sync();  // no block leaves while another reads its shared memory
    }
}

// Any k: where not even one token's k fits into a cluster's shared memory.  One
// warp per (row of W, 8 rows of A), lane l taking codes l, l + 32, ...
template <typename T>
__global__ void __launch_bounds__(256) tg_gemm_w4_simple(const W4Params p) {
    op_release_next();
    op_wait_previous();
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

// Both halves times s, each rounded once.
__device__ __forceinline__ uint32_t w4_scale(uint32_t v, __half s) {
    const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&v), __half2half2(s));
    return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t w4_scale(uint32_t v, __nv_bfloat16 s) {
    const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&v), __bfloat162bfloat162(s));
    return *reinterpret_cast<const uint32_t*>(&r);
}

// What the rounding to `high` = v·s left, exactly.
__device__ __forceinline__ uint32_t w4_scale_rest(uint32_t v, __half s, uint32_t high) {
    const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&v), __half2half2(s),
                              __hneg2(*reinterpret_cast<const __half2*>(&high)));
    return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t w4_scale_rest(uint32_t v, __nv_bfloat16 s, uint32_t high) {
    const __nv_bfloat162 r = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&v), __bfloat162bfloat162(s),
                                     __hneg2(*reinterpret_cast<const __nv_bfloat162*>(&high)));
    return *reinterpret_cast<const uint32_t*>(&r);
}

// W as a K×N matrix of T (row stride ldo, a multiple of 8), for the dense GEMM
// on very many rows of A.  Here (code - zero)·scale is rounded to T, as the tensor
// cores read 16-bit operands: at most half an ulp of each weight, an error of
// the size that storing C in T has.  One 128 k × 64 n tile per block
// iteration, turned round in shared memory; a thread decodes 16 k of two
// neighbouring rows of W, so that it stores pairs of n.  256 threads.
// 16384×8192 takes about 100 us for 336 MB (3.3 TB/s).
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
        uint32_t v[2][2][4];  // of two rows and two words: pairs (w_i, w_i+4)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int64_t n = n0 + 2 * pair + i;
            T s = op_round<T>(0.0f);
            uint32_t z = 8, w[2] = {0, 0};
            if (n < p.N && kb < p.K) {
                const int64_t g = kb / p.group;
                s = static_cast<const T*>(p.scale)[g * p.lds + n];
                if (p.zero != nullptr) z = p.zero[g * p.ldz + n] & 15u;
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
            const W4Decode<T> decode(z);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                decode(w[j], v[i][j]);  // code - zero point, exactly
#pragma unroll
                for (int e = 0; e < 4; ++e) v[i][j][e] = w4_scale(v[i][j][e], s);
            }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                tile[16 * kq + 8 * j + e][pair] = __byte_perm(v[0][j][e], v[1][j][e], 0x5410);
                tile[16 * kq + 8 * j + 4 + e][pair] = __byte_perm(v[0][j][e], v[1][j][e], 0x7632);
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
