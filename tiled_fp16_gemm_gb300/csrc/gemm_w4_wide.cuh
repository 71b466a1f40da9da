// Products of many rows of A with 4-bit weights, on tcgen05: W·Aᵀ with W decoded into
// tensor memory, for a 16-bit result each weight rounded to T.
//
// As in gemm_w4_tc.cuh the weights are the MMA's A operand (units of 128 rows of W by
// 128 k), decoded by threads that own a row.  Here (code - z) · s is rounded to T before
// it is stored, as a dense 16-bit weight would be: an error of at most half an ulp of
// each weight, below that of a 16-bit result's rounding for all but cancelling sums.  So
// one accumulator of up to 256 tokens runs over the whole of k, and the MMAs (1024 cycles
// a unit at 256 tokens) hide the decoding (some 270 instructions of each scheduler).
//
// EXACT, for an fp32 result: the rounding's error, (code - z) · s minus the rounded value,
// is a T too (the product has 15 bits at most, its last place that of s or above), and one
// fused multiplication and addition gives it.  It is the operand of a second set of MMAs on
// the same tokens, so no weight is rounded; units take two places in tensor memory.  Where
// that adds up to NaN the sum is taken again from the definition (wide_again): an infinite
// activation times a remainder of 0, or of the other sign, is NaN where the weight is not 0,
// and a weight beyond T's range is inf minus inf.
//
// The blocks work in pairs (cta_group::2): the MMA takes 256 rows of W, 128 in each block's
// tensor memory, and half of the tokens from each block's shared memory.  With blocks of
// their own, the tokens multicast to both, a unit took 1370 cycles; the MMAs' reads and the
// copies' writes then ask for all of the shared memory's 128 bytes a cycle.  Now it takes
// 1070 with 256 tokens (the MMAs bound it) and 780 with 128 (the codes' arrival does).  An
// arrival at the even block with release.cluster cost 1900 cycles; the plain form does not.
//
// Measured, 16384×8192, fp16, G = 128: 65 / 128 / 256 / 512 / 2048 rows 34 / 35 / 47 / 87 /
// 324 us; the last two are 1580 and 1700 TFLOP/s.  (In long runs, under the power cap, 91 and
// 365 us.  Decoding to memory, then the dense GEMM: 160 us for 256 rows, 193 for 512.)  At 512
// rows 64 of the 76 pairs work, on whole tiles.  With an fp32 result 65 / 128 / 256 / 512 rows
// 41 / 46 / 81 / 149 us (by passes of 64 rows through gemm_w4_tc.cuh 62 / 84 / 170 / 340).
//
// Roles of a block's 24 warps (all meet on mbarriers):
//   0             fetches codes, scales and zero points by TMA
//   1             of the even block: issues the pair's MMAs, and the commits to both
//   2             fetches this block's half of the tokens by TMA
//   4-7, 20-23    read the accumulator back and write C, 16 tokens at a time in turn
//   8-19          decode, in three groups of four warps that take units in turn
// The clusters have whole tiles, or share all units (tile by tile, k inside) evenly: then
// each block leaves its sums of a shared tile in the workspace, and the last one to come
// adds all of them, in the order of k: the same bits every time.
#pragma once

#include "gemm_w4_tc.cuh"

namespace tg {

constexpr int kWideStages = 6;           // of codes
constexpr int kWideXStages = 4;
constexpr int kWideTokens = 256;         // of a tile at most
constexpr int kWideCodeBytes = 10240;    // codes 8192, scales ≤ 1024, zero points ≤ 512
constexpr int kWideScaleAt = 8192;
constexpr int kWideZeroAt = 9216;
constexpr int kWideXBytes = kWideTokens / 2 * 256;
constexpr int kWideNanBytes = 256 * 16;  // EXACT: which of a thread's 8 times 16 sums are NaN
constexpr int kWideSmem =
    1024 + kWideXStages * kWideXBytes + kWideStages * kWideCodeBytes + 512 + kWideNanBytes;

struct WideLaunch {
    W4Params p;
    uint64_t limit_ns;
    unsigned int* timeouts;  // set where a warp gives up on a wait
    int32_t inject;      // 1: block 0's first codes are left out (for tests of the limit)
    int32_t tokens;      // of a tile: a multiple of 32
    int32_t m_tiles;
    int32_t k_units;
    int64_t units;       // in all: (row blocks / cluster) · m_tiles · k_units
    int32_t grain;       // units that stay together: k_units (whole tiles) or 1
    int32_t clusters;
    float* slots;        // two per block: the sums of its first and last tile
    uint32_t* counters;  // eight per block
};

// EXACT: sums that came out NaN, by the definition: Σ a·((c - z)·s), each weight exact in
// fp32, and their epilogue.  A row of A with NaN or infinities has the sum of their products,
// whatever the others are.  `seen`: which 16 of each 32 tokens from m0 on, `nan`: which of them.
// (At the end of a tile, and no call: either took registers from its loop.)  512 rows of
// 16384×8192, fp16: one infinity in one row 0.27 ms instead of 0.15, in every row 36 ms, all
// of A infinite or NaN 0.9 ms; every weight beyond fp16's range 0.2 s.
template <typename T>
__device__ __forceinline__ void wide_again(const W4Params& p, int64_t m0, int64_t n, uint32_t seen,
                                        const uint16_t* nan) {
    auto finite = [](float x) { return x - x == 0.0f; };
    // 8 products, k a multiple of 8: of all activations, or of those that are not finite
    auto eight = [&](const T* a, int64_t k, bool all, float sum) {
        const int64_t g = k / p.group;
        const int z = p.zero != nullptr ? p.zero[g * p.ldz + n] & 15 : 8;
        const float s = op_to_float(static_cast<const T*>(p.scale)[g * p.lds + n]);
        const uint8_t* codes = p.Bq + n * p.ldbq + k / 2;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (k + j >= p.K) break;
            const float x = op_to_float(a[k + j]);
            const float w = static_cast<float>((codes[j / 2] >> (4 * (j & 1)) & 15) - z) * s;
            if (all || !finite(x)) sum = fmaf(x, w, sum);
        }
        return sum;
    };
#pragma unroll 1
    for (int c = 0; seen >> c != 0; ++c) {
        if ((seen >> c & 1) == 0) continue;
#pragma unroll 1
        for (int i = 0; i < 16; ++i) {
            const int64_t m = m0 + 32 * c + i;
            if ((nan[c] >> i & 1) == 0 || m >= p.M) continue;
            const T* a = static_cast<const T*>(p.A) + m * p.lda;
            float sum = 0.0f;
            bool clean = true;
#pragma unroll 1
            for (int64_t k = 0; k < p.K && sum == sum; k += 32) {
                bool fine = true;
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    fine = finite(op_to_float(a[k + j < p.K ? k + j : k])) && fine;
                if (fine) continue;
                clean = false;
#pragma unroll 1
                for (int64_t l = k; l < k + 32 && l < p.K; l += 8) sum = eight(a, l, false, sum);
            }
            if (clean)
#pragma unroll 1
                for (int64_t k = 0; k < p.K; k += 8) sum = eight(a, k, true, sum);
            w4_store<T>(p, m, n, sum);
        }
    }
}
// Which of 16 sums are NaN, noted for the end of the tile.
__device__ __forceinline__ void wide_note(const float (&v)[16], int c, uint16_t* nan, uint32_t* seen) {
    bool any = false;
#pragma unroll
    for (int i = 0; i < 16; ++i) any = any || v[i] != v[i];
    if (any) {
        uint32_t bits = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) bits |= (v[i] != v[i] ? 1u : 0u) << i;
        nan[c >> 5] = static_cast<uint16_t>(bits);
        *seen |= 1u << (c >> 5);
    }
}
// Epilogue and store of 16 tokens of row n, `most` of them.
template <typename T, typename TC>
__device__ __forceinline__ void wide_store(const W4Params& p, int64_t m, int64_t n, int most, float bias,
                                           float (&v)[16]) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        v[i] += bias;
        if (p.relu) v[i] = v[i] > 0.0f ? v[i] : 0.0f;
    }
    if (p.resid != nullptr) {
        const char* r = static_cast<const char*>(p.resid) + 2 * (m * p.ldr + n);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if (i < most) v[i] += op_to_float(*reinterpret_cast<const T*>(r));
            r = wide_step(r, 2 * p.ldr);
        }
    }
    char* c = static_cast<char*>(p.C) + sizeof(TC) * (m * p.ldc + n);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        if (i < most) *reinterpret_cast<TC*>(c) = op_round<TC>(v[i]);
        c = wide_step(c, sizeof(TC) * p.ldc);
    }
}

template <typename T, int G, bool ZERO, bool EXACT>
__global__ void __launch_bounds__(kWideThreads, 1)
    tg_gemm_w4_wide(const __grid_constant__ WideLaunch q, const __grid_constant__ CUtensorMap codes,
                    const __grid_constant__ CUtensorMap scales, const __grid_constant__ CUtensorMap zeros,
                    const __grid_constant__ CUtensorMap order) {
    constexpr int kGroups = kTcK / G;
    constexpr int kABufs = EXACT ? 2 : 4, kACols = 256 / kABufs;
    using TC = typename std::conditional<EXACT, float, T>::type;
    extern __shared__ __align__(1024) unsigned char wide_dynamic[];
    const W4Params& p = q.p;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rank = blockIdx.x % kWideCluster, cluster_no = blockIdx.x / kWideCluster;
    const uint32_t base = (op_smem(wide_dynamic) + 1023) & ~1023u;
    unsigned char* const shared = wide_dynamic + (base - op_smem(wide_dynamic));
    const uint32_t xs = base, cs = xs + kWideXStages * kWideXBytes;
    const uint32_t bars = cs + kWideStages * kWideCodeBytes;
    const uint32_t c_full = bars, c_empty = c_full + 8 * kWideStages;
    const uint32_t x_full = c_empty + 8 * kWideStages, x_empty = x_full + 8 * kWideXStages;
    const uint32_t a_full = x_empty + 8 * kWideXStages, done = a_full + 8 * kABufs;
    const uint32_t d_full = done + 8 * kTcDone, d_empty = d_full + 8;
    unsigned char* after = shared + (d_empty + 8 - base);
    uint32_t* tmem_at = reinterpret_cast<uint32_t*>(after);
    volatile int* dead = reinterpret_cast<volatile int*>(after + 4);  // a wait ran out: reported at the end

    op_release_next();
    if (warp == 0 && lane == 0) {
        for (int i = 0; i < kWideStages; ++i) {
            op_bar_init(c_full + 8 * i, 1);
            op_bar_init(c_empty + 8 * i, 4);
        }
        for (int i = 0; i < kWideXStages; ++i) {
            op_bar_init(x_full + 8 * i, 1);  // of the even block: both blocks' copies
            op_bar_init(x_empty + 8 * i, 1);
        }
        for (int i = 0; i < kABufs; ++i) op_bar_init(a_full + 8 * i, 8);  // of the even block
        for (int i = 0; i < kTcDone; ++i) op_bar_init(done + 8 * i, 1);
        op_bar_init(d_full, 1);
        op_bar_init(d_empty, 16);  // of the even block
        op_bar_init_done();
        *dead = 0;
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                         op_smem(tmem_at))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_before_sync();
    __syncthreads();
    tc_cluster_sync();  // no copy or commit reaches a block before its barriers are there
    tc_after_sync();
    // all columns are this block's, so they begin at 0
    constexpr uint32_t tmem = 0;
    constexpr uint32_t d_cols = tmem + 256;

    const int64_t grains = q.units / q.grain;
    const int64_t u0 = tc_first(grains, q.clusters, cluster_no) * q.grain;
    const int n_units =
        static_cast<int>(tc_first(grains, q.clusters, cluster_no + 1) * q.grain - u0);
    int64_t tile = u0 / q.k_units;
    int kb = static_cast<int>(u0 - tile * q.k_units);
    // A warp waits; false once a wait has run out, here or in another warp.
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (__all_sync(0xffffffffu, op_bar_try(bar, parity))) return true;
        const bool ok = *dead == 0 && op_bar_wait_slow(bar, parity, q.limit_ns);
        if (__all_sync(0xffffffffu, ok)) return true;
        if (lane == 0) *dead = 1;
        __syncwarp();
        return false;
    };
    auto next_unit = [&] {
        if (++kb == q.k_units) kb = 0, ++tile;
    };
    auto first_row = [&] { return (tile / q.m_tiles * kWideCluster + rank) * kTcRows; };
    auto first_token = [&] { return tile % q.m_tiles * q.tokens; };

    if (warp == 0) {
        // ------------------------------------------------------------ codes
        // No wait for the ordering kernel: see gemm_w4_tc.cuh.
        int issued = 0;
        for (int i = 0; i < n_units; ++i, next_unit()) {
            const int s = i % kWideStages;
            if (i >= kWideStages && !wait(c_empty + 8 * s, (i / kWideStages - 1) & 1)) break;
            if (lane == 0 && !(q.inject == 1 && blockIdx.x == 0 && i == 0)) {
                const uint32_t to = cs + s * kWideCodeBytes, bar = c_full + 8 * s;
                const uint32_t n = static_cast<uint32_t>(first_row());
                op_bar_expect(bar, 8192 + (ZERO ? 384 : 256) * kGroups);
                op_tma_2d(to, &codes, bar, kb * 64, n);
                op_tma_2d(to + kWideScaleAt, &scales, bar, n, kb * kGroups);
                if (ZERO) op_tma_2d(to + kWideZeroAt, &zeros, bar, n, kb * kGroups);
            }
            issued = i + 1;
        }
        // copies under way have to land before the block ends
        bool ok = true;
        for (int i = issued > kWideStages ? issued - kWideStages : 0; ok && i < issued; ++i)
            if (lane == 0) ok = op_bar_wait(c_full + 8 * (i % kWideStages), i / kWideStages & 1, kTcLandNs);
    } else if (warp == 2) {
        // ------------------------------------------------------------ A
        op_wait_previous();
        const uint32_t part = q.tokens / 2;
        int issued = 0;
        for (int i = 0; i < n_units; ++i, next_unit()) {
            const int s = i % kWideXStages;
            if (i >= kWideXStages && !wait(x_empty + 8 * s, (i / kWideXStages - 1) & 1)) break;
            if (lane == 0) {
                const uint32_t to = xs + s * kWideXBytes, bar = wide_at(x_full + 8 * s, 0);
                const uint32_t m = static_cast<uint32_t>(first_token()) + rank * part;
                if (rank == 0) op_bar_expect(x_full + 8 * s, q.tokens * 256);
                wide_tma(to, &order, bar, kb * kTcK, m);
                wide_tma(to + part * 128, &order, bar, kb * kTcK + 64, m);
            }
            issued = i + 1;
        }
        // the copies have to land, and the commits to arrive, before this block ends
        bool ok = true;
        for (int i = issued > kWideXStages ? issued - kWideXStages : 0; ok && i < issued; ++i)
            if (lane == 0) ok = op_bar_wait(x_empty + 8 * (i % kWideXStages), i / kWideXStages & 1, kTcLandNs);
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMAs
        constexpr uint32_t fmt = std::is_same<T, __half>::value ? 0u : 1u;
        const uint32_t idesc = (1u << 4) | (fmt << 7) | (fmt << 10) |
                               (static_cast<uint32_t>(q.tokens >> 3) << 17) | (16u << 24);
        int issued = 0, tiles = 0;
        for (int i = 0; rank == 0 && i < n_units; ++i) {
            const int s = i % kWideXStages, a = i % kABufs;
            const bool first = i == 0 || kb == 0;
            if (!wait(x_full + 8 * s, i / kWideXStages & 1)) break;
            if (first && tiles++ > 0 && !wait(d_empty, tiles & 1)) break;
            if (!wait(a_full + 8 * a, i / kABufs & 1)) break;
            tc_after_sync();
            const uint64_t x = tc_desc(xs + s * kWideXBytes);
            wide_unit<!EXACT>(d_cols, tmem + kACols * a, x, q.tokens / 2 * 128 / 16, idesc, first ? 0 : 1,
                              done + 8 * (i % kTcDone), x_empty + 8 * s);
            if (EXACT)
                wide_unit<true>(d_cols, tmem + kACols * a + 64, x, q.tokens / 2 * 128 / 16, idesc, 1,
                                done + 8 * (i % kTcDone), x_empty + 8 * s);
            if (kb + 1 == q.k_units || i + 1 == n_units) wide_commit(d_full);
            issued = i + 1;
            next_unit();
        }
        // the MMAs have to be over before the tensor memory is given back
        if (issued > 0 && lane == 0)
            op_bar_wait(done + 8 * ((issued - 1) % kTcDone), (issued - 1) / kTcDone & 1, kTcLandNs);
        __syncwarp();
    } else if (warp >= 8 && warp < 20) {
        // ------------------------------------------------------------ decoding
        const int group = (warp - 8) >> 2;
        const uint32_t row = 32 * (warp & 3) + lane;
        const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        for (int i = group; i < n_units; i += kTcGroups) {
            const int s = i % kWideStages, a = i % kABufs;
            if (!wait(c_full + 8 * s, i / kWideStages & 1)) break;
            const uint32_t at = cs + s * kWideCodeBytes;
            uint4 w[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) w[c] = tc_lds128(at + row * 64 + ((c ^ (row >> 1 & 3)) << 4));
            uint32_t z[kGroups];
            T scale[kGroups];
#pragma unroll
            for (int c = 0; c < kGroups; ++c) {
                scale[c] = *reinterpret_cast<const T*>(shared + (at - base) + kWideScaleAt +
                                                       (c * kTcRows + row) * 2);
                z[c] = ZERO ? shared[at - base + kWideZeroAt + c * kTcRows + row] & 15u : 8u;
            }
            const int old = i - kABufs;
            if (old >= 0 && !wait(done + 8 * (old % kTcDone), old / kTcDone & 1)) break;
            tc_after_sync();
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const W4Decode<T> decode(z[c * 32 / G]);
                const uint32_t words[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
                uint32_t r[16], low[16];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t v[4];
                    decode(words[j], v);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        r[4 * j + e] = w4_scale(v[e], scale[c * 32 / G]);
                        if (EXACT) low[4 * j + e] = w4_scale_rest(v[e], scale[c * 32 / G], r[4 * j + e]);
                    }
                }
                tc_store16(tmem + lanes + kACols * a + 16 * c, r);
                if (EXACT) tc_store16(tmem + lanes + kACols * a + 64 + 16 * c, low);
            }
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            tc_before_sync();
            __syncwarp();
            if (lane == 0) {
                wide_arrive(wide_at(a_full + 8 * a, 0));
                // not before the codes have been used: with the arrival right behind the
                // loads, stages were refilled before these had taken effect
                tc_arrive(c_empty + 8 * s);
            }
        }
    } else if (warp >= 4) {
        // ------------------------------------------------------------ C
        op_wait_previous();
        const int quarter = warp & 3, set = warp < 8 ? 0 : 1;
        const uint32_t row = 32 * quarter + lane;
        const uint32_t at = d_cols + (static_cast<uint32_t>(32 * quarter) << 16);
        const int64_t slot = int64_t{q.tokens} * kTcRows;
        uint16_t* const nan = reinterpret_cast<uint16_t*>(shared + (bars + 512 - base)) + (set * kTcRows + row) * 8;
        int i = 0;
        uint32_t tiles = 0;
        while (i < n_units) {
            const int kb0 = kb;
            const int len = q.k_units - kb < n_units - i ? q.k_units - kb : n_units - i;
            // (a barrier of its own: a parity says nothing of a phase further off than one)
            if (!wait(d_full, tiles++ & 1)) break;
            tc_after_sync();
            const int64_t n = first_row() + row, m0 = first_token();
            const int tokens = static_cast<int>(p.M - m0 < q.tokens ? p.M - m0 : q.tokens);
            const bool whole = len == q.k_units;
            const float bias = p.bias != nullptr && n < p.N ? p.bias[n] : 0.0f;
            float* mine = q.slots + (2 * int64_t{blockIdx.x} + (kb0 > 0 ? 0 : 1)) * slot + row * 4;
            uint32_t seen = 0;
            for (int c = 16 * set; c < tokens; c += 32) {
                uint32_t r[16];
                tc_load(at + c, r);
                if (whole) {
                    float v[16];
#pragma unroll
                    for (int m = 0; m < 16; ++m) v[m] = __uint_as_float(r[m]);
                    if constexpr (EXACT) wide_note(v, c, nan, &seen);
                    if (n < p.N) wide_store<T, TC>(p, m0 + c, n, tokens - c, bias, v);
                } else {
#pragma unroll
                    for (int m = 0; m < 16; m += 4)
                        __stcg(reinterpret_cast<float4*>(mine + (c + m) * kTcRows),
                               make_float4(__uint_as_float(r[m]), __uint_as_float(r[m + 1]),
                                           __uint_as_float(r[m + 2]), __uint_as_float(r[m + 3])));
                }
            }
            tc_before_sync();
            __syncwarp();
            if (lane == 0) wide_arrive(wide_at(d_empty, 0));
            if (!whole) {  // a share of a tile
                __threadfence();
                __syncwarp();
                const int head = static_cast<int>(tc_block_of(q.units, q.clusters, tile * q.k_units));
                const int tail = static_cast<int>(tc_block_of(q.units, q.clusters, (tile + 1) * q.k_units - 1));
                uint32_t before = 0;
                if (lane == 0) {
                    uint32_t* count = q.counters + 8 * (head * kWideCluster + rank) + 4 * set + quarter;
                    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;"
                                 : "=r"(before)
                                 : "l"(count)
                                 : "memory");
                    if (before == static_cast<uint32_t>(tail - head)) *count = 0;  // for the next launch
                }
                before = __shfl_sync(0xffffffffu, before, 0);
                __threadfence();
                if (before == static_cast<uint32_t>(tail - head)) {
                    // the head's share is in its second slot, the others' in their first
                    for (int c = 16 * set; c < tokens; c += 32) {
                        float sum[16];
                        const float* from = q.slots + (2 * (int64_t{head} * kWideCluster + rank) + 1) * slot +
                                            c * kTcRows + row * 4;
                        wide_load(from, sum);
                        // two at a time under way
                        from = q.slots + 2 * (int64_t{head + 1} * kWideCluster + rank) * slot + c * kTcRows +
                               row * 4;
                        const int64_t step = 2 * kWideCluster * slot;
                        for (int b = head + 1; b <= tail; b += 2, from += 2 * step) {
                            float v[16], w[16];
                            wide_load(from, v);
                            if (b < tail) wide_load(from + step, w);
#pragma unroll
                            for (int m = 0; m < 16; ++m) sum[m] += v[m];
                            if (b < tail) {
#pragma unroll
                                for (int m = 0; m < 16; ++m) sum[m] += w[m];
                            }
                        }
                        if constexpr (EXACT) wide_note(sum, c, nan, &seen);
                        if (n < p.N) wide_store<T, TC>(p, m0 + c, n, tokens - c, bias, sum);
                    }
                }
            }
            if constexpr (EXACT) {
                if (seen != 0 && n < p.N) wide_again<T>(p, m0 + 16 * set, n, seen, nan);
            }
            i += len;
            kb = 0;
            ++tile;
        }
    }
    tc_before_sync();
    __syncthreads();
    if (threadIdx.x == 0 && *dead != 0) atomicOr(q.timeouts, kOpTimeoutW4);
    __syncwarp();
    tc_cluster_sync();  // neither block's memory or barriers are used by the other any more
    if (warp == 1) {
        __syncwarp();
        tc_after_sync();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(*tmem_at)
                     : "memory");
    }
}

}  // namespace tg
