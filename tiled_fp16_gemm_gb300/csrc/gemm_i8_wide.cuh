// Products of many rows of A with 8-bit integers, on tcgen05.
//
// sm_103a has no integer form of tcgen05.mma, and that of mma.sync has a fifteenth of the rate of
// tcgen05 in fp16; but whole numbers up to 2048 are exact in fp16, their products exact in the
// fp16 MMA, and sums of them exact in its fp32 accumulator up to 2^24.  So B is decoded to
// fp16 on the way: the structure of gemm_w4_wide.cuh, with a weight's bytes instead of nibbles,
// no scale before the epilogue, and A as fp16 in the workspace (tg_i8_expand).
//
// Units of 128 rows of B by 128 k are the MMA's A operand, decoded by threads that own a row
// into tensor memory; the pair of blocks of a cluster multiplies 256 rows of B by up to 256
// tokens.  Roles of a block's 24 warps, as there: 0 fetches B, 2 this block's half of the
// tokens, 1 of the even block issues the MMAs, 8-19 decode, 4-7 and 20-23 write C.  The
// clusters have whole tiles, equal parts of a tile, or even runs of all units.  Of a shared tile
// each adds its sums to 32-bit ones in the workspace, and the last one to come writes C.  These are
// whole numbers, so their order is free, and none passes 2^31.  (Each cluster's sums left in a place of
// their own, for the last one to read: 1024×8192 with 128 rows 22 us, now 14; 4096×28672 43, now 37.)
//
// Every sum is exact, whatever cancels in it: the accumulator takes a run of units that no sum can
// leave 2^24 in.  A sum is at most 128 times that of its token's |codes|, and those tg_i8_expand adds up
// (I8Peak): where no token's pass 2^17 a run is all of K (8192 columns, where some are larger than the
// others; 4000 of normally distributed values), else as many units as fit at the largest |codes| of a
// unit (some 30; 15 of evenly distributed values).  After a run the C warps look at the sums, and the next run
// goes on with them; 16 tokens of a warp with one past 2^22 among them go to 32-bit whole numbers in the
// workspace and begin again from zero.  A look is 1 to 2 us in which the MMAs rest; giving all sums to the
// workspace after each run took 4 to 6.
//
// Measured, bf16 results, random codes (they draw more power than zeros: 512 rows 84 to 88 us where a
// constant weight takes 80), K in one run: 16384×8192 with 64 / 128 / 256 / 512 / 1024 rows 32 / 34 / 47 / 86 /
// 155 us (normally distributed 33 / 36 / 50 / 92 / 164, evenly 34 / 38 / 55 / 104 / 180), 28672×4096 33 with
// 64, 73 with 512, 4096×4096 with 64 / 256 rows 13 / 20, 256 rows of 1024×1024 8.6.  A unit takes 0.62 us with 256 tokens (0.54 at full clocks), bound by the MMAs;
// with few tokens the blocks fetch B at 5.5 TB/s, and 6 to 8 us go to two launches, the start and the
// end.  The C warps have what the epilogue needs before the sums are there, and give the accumulator
// back when they have read it, before they have stored: 512 rows of 28672×4096 73 us instead of 84.
// Registers are full (80).
#pragma once

#include "gemm_i8.cuh"
#include "tc_device.cuh"

namespace tg {

// Of B.  A decoding group meets every phase of a stage, or none: its parity says nothing of a
// phase that the group has not waited for the one before of.
constexpr int kI8Stages = 6;
static_assert(kI8Stages % kTcGroups == 0, "unit i + kI8Stages is the same group's as unit i");
constexpr int kI8XStages = 4;
constexpr int kI8Tokens = 256;  // of a tile at most
constexpr int kI8CodeBytes = kTcRows * kTcK;
constexpr int kI8XBytes = kI8Tokens / 2 * 256;
constexpr int kI8WideSmem = 1024 + kI8XStages * kI8XBytes + kI8Stages * kI8CodeBytes + 512;
static_assert(kI8WideSmem <= 227 * 1024, "shared memory of a block");
constexpr int kI8MaxClusters = 80;
constexpr int64_t kI8CounterBytes = 8192;
static_assert(kI8MaxClusters * kWideCluster * 32 <= kI8CounterBytes, "eight counters per block");
constexpr int kI8WideRun = 8;  // units whose sums are exact in fp32: 8 · 128 · 2^14 = 2^24
constexpr float kI8Keep = 4194304.0f;  // 2^22: sums that a further run begins with, at most

// What a block of tg_i8_expand saw, in its 4096 columns: the largest sum of |codes| of a token in a
// unit of 128 k, and a bound on that of a token in all of the columns (each warp's largest, added up).
struct I8Peak {
    uint32_t unit, part;
};
constexpr int kI8Peaks = 2048;     // blocks of tg_i8_expand, at most
constexpr int kI8PeakColumns = 4096;  // of a block
constexpr int64_t kI8PeakBytes = kI8Peaks * sizeof(I8Peak);
static_assert((131071 + kI8PeakColumns - 1) / kI8PeakColumns <= 32, "a lane or more for each 4096 columns");

struct I8Wide {
    I8Params p;
    uint64_t limit_ns;
    unsigned int* timeouts;  // set where a warp gives up on a wait
    int32_t inject;      // 1: block 0's first codes are left out (for tests of the limit)
    int32_t tokens;      // of a tile: a multiple of 32
    int32_t m_tiles;
    int32_t k_units;
    int64_t units;       // in all: (row blocks / cluster) · m_tiles · k_units
    int32_t parts;       // clusters of a tile, each with a run of its units (clusters = tiles · parts); 0:
    int32_t grain;       // the clusters have even runs of all units, of k_units (whole tiles) or 1 at least
    int32_t clusters;
    int32_t* sums;       // of the shared tiles, zeroed by tg_i8_expand: 128 rows for each token and block
    int32_t by_tile;     // the tiles' places: their own numbers, else those of their first clusters
    int32_t places;      // of shared tiles; behind them each cluster has one for its own tiles' runs
    uint32_t* counters;  // eight per block, zeroed by tg_i8_expand
    const I8Peak* peaks;  // of tg_i8_expand's blocks, across × down; null where kI8WideRun units are all of K
    int32_t across, down;
};

// A cluster's first unit.
__device__ __forceinline__ int64_t i8_first(const I8Wide& q, int cluster) {
    if (q.parts == 0) return tc_first(q.units / q.grain, q.clusters, cluster) * q.grain;
    const int tile = cluster / q.parts;
    return int64_t{tile} * q.k_units + tc_first(q.k_units, q.parts, cluster - tile * q.parts);
}

// Sum of the sizes of 16 codes.
__device__ __forceinline__ uint32_t i8_size(uint4 x) {
    const uint32_t sign = 0x80808080u;  // (a code + 128 is that far from 128)
    return __vsadu4(x.x ^ sign, sign) + __vsadu4(x.y ^ sign, sign) + __vsadu4(x.z ^ sign, sign) +
           __vsadu4(x.w ^ sign, sign);
}

// A as fp16 in rows of `ldo` (a multiple of 128), zero past column K; the counters and `zeros` 16 bytes of
// the shared tiles' sums zeroed; and, where `peaks` is given, the block's.
__global__ void __launch_bounds__(256)
    tg_i8_expand(const int8_t* __restrict__ A, int64_t lda, int64_t M, int64_t K, uint16_t* __restrict__ out,
                 int64_t ldo, uint32_t* counters, uint4* sums, int64_t zeros, I8Peak* peaks) {
    __shared__ I8Peak of_warp[8];
    op_wait_previous();
    op_release_next();
    if (blockIdx.x == 0 && blockIdx.y == 0)
        for (int i = threadIdx.x; i < kI8CounterBytes / 4; i += 256) counters[i] = 0;
    const int64_t c = int64_t{blockIdx.x} * 256 + threadIdx.x;
    const int64_t threads = int64_t{gridDim.x} * gridDim.y * 256;
    for (int64_t i = int64_t{blockIdx.y} * gridDim.x * 256 + c; i < zeros; i += threads)
        sums[i] = make_uint4(0, 0, 0, 0);
    const bool mine = 16 * c < ldo;
    const bool wide = (reinterpret_cast<uintptr_t>(A) & 15) == 0 && lda % 16 == 0 && 16 * c + 16 <= K;
    uint32_t unit = 0, part = 0;
    for (int64_t m = blockIdx.y; m < M; m += gridDim.y) {
        uint32_t size = 0;
        if (mine) {
            const int8_t* a = A + m * lda;
            const uint4 x = wide ? *reinterpret_cast<const uint4*>(a + 16 * c) : i8_bytes(a, 16 * c, K);
            uint4 y[2];
            i8_decode(x.x, y[0].x, y[0].y);
            i8_decode(x.y, y[0].z, y[0].w);
            i8_decode(x.z, y[1].x, y[1].y);
            i8_decode(x.w, y[1].z, y[1].w);
            uint4* to = reinterpret_cast<uint4*>(out + m * ldo + 16 * c);
            to[0] = y[0];
            to[1] = y[1];
            size = i8_size(x);
        }
        if (peaks != nullptr) {  // eight threads have a unit
#pragma unroll
            for (int o = 1; o < 8; o *= 2) size += __shfl_xor_sync(0xffffffffu, size, o);
            unit = max(unit, size);
#pragma unroll
            for (int o = 8; o < 32; o *= 2) size += __shfl_xor_sync(0xffffffffu, size, o);
            part = max(part, size);
        }
    }
    if (peaks == nullptr) return;
    unit = __reduce_max_sync(0xffffffffu, unit);
    if ((threadIdx.x & 31) == 0) of_warp[threadIdx.x / 32] = I8Peak{unit, part};
    __syncthreads();
    if (threadIdx.x == 0) {
        I8Peak all = of_warp[0];
#pragma unroll
        for (int w = 1; w < 8; ++w) {
            all.unit = max(all.unit, of_warp[w].unit);
            all.part += of_warp[w].part;
        }
        peaks[blockIdx.x * gridDim.y + blockIdx.y] = all;
    }
}

// How many units the accumulator may take from zero on, and from kI8Keep on, by the peaks; for a whole warp.
__device__ __forceinline__ int2 i8_runs(const I8Wide& q, int lane) {
    int lanes = 32;  // for each column of blocks
    while (lanes * q.across > 32) lanes /= 2;
    const int x = lane / lanes;
    uint32_t unit = 0, part = 0;
    const uint2* of = reinterpret_cast<const uint2*>(q.peaks) + x * q.down;
    for (int y = lane % lanes; x < q.across && y < q.down; y += 16 * lanes) {
        uint2 peak[16];  // under way at once: the MMAs of the first units wait for no longer than this
#pragma unroll
        for (int j = 0; j < 16; ++j)
            peak[j] = y + j * lanes < q.down ? __ldcg(of + y + j * lanes) : make_uint2(0, 0);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            unit = max(unit, peak[j].x);
            part = max(part, peak[j].y);
        }
    }
    unit = __reduce_max_sync(0xffffffffu, unit);
    for (int o = 1; o < lanes; o *= 2) part = max(part, __shfl_xor_sync(0xffffffffu, part, o));
    part = __reduce_add_sync(0xffffffffu, lane % lanes == 0 ? part : 0u);  // of a token's, all columns
    if (part <= 1u << 17) return make_int2(q.k_units, q.k_units);
    return make_int2(static_cast<int>((1u << 17) / unit), static_cast<int>((3u << 15) / unit));
}

// A sum in the workspace, which other clusters add to.
__device__ __forceinline__ int32_t i8_load(const int32_t* sum) {
    int32_t v;
    asm volatile("ld.relaxed.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(sum) : "memory");
    return v;
}

// Epilogue and store of 16 tokens of row n, `most` of them, whose scales the lanes from `first` on
// hold.
template <typename TC>
__device__ __forceinline__ void i8_wide_store(const I8Params& p, int64_t m, int64_t n, int most, float scales, int first,
                                              float sb, float bias, float (&v)[16]) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = i8_value(p, v[i], __shfl_sync(0xffffffffu, scales, first + i), sb, bias);
    if (n >= p.N) return;
    if (p.resid != nullptr) {
        const char* r = static_cast<const char*>(p.resid) + sizeof(TC) * (m * p.ldr + n);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if (i < most) v[i] += op_to_float(*reinterpret_cast<const TC*>(r));
            r = wide_step(r, sizeof(TC) * p.ldr);
        }
    }
    char* c = static_cast<char*>(p.C) + sizeof(TC) * (m * p.ldc + n);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        if (i < most) *reinterpret_cast<TC*>(c) = op_round<TC>(v[i]);
        c = wide_step(c, sizeof(TC) * p.ldc);
    }
}

template <typename TC>
__global__ void __launch_bounds__(kWideThreads, 1)
    tg_gemm_i8_wide(const __grid_constant__ I8Wide q, const __grid_constant__ CUtensorMap codes,
                    const __grid_constant__ CUtensorMap order) {
    constexpr int kABufs = 4, kACols = 64;
    extern __shared__ __align__(1024) unsigned char wide_dynamic[];
    const I8Params& p = q.p;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rank = blockIdx.x % kWideCluster, cluster_no = blockIdx.x / kWideCluster;
    const uint32_t base = (op_smem(wide_dynamic) + 1023) & ~1023u;
    unsigned char* const shared = wide_dynamic + (base - op_smem(wide_dynamic));
    const uint32_t xs = base, cs = xs + kI8XStages * kI8XBytes;
    const uint32_t bars = cs + kI8Stages * kI8CodeBytes;
    const uint32_t c_full = bars, c_empty = c_full + 8 * kI8Stages;
    const uint32_t x_full = c_empty + 8 * kI8Stages, x_empty = x_full + 8 * kI8XStages;
    const uint32_t a_full = x_empty + 8 * kI8XStages, done = a_full + 8 * kABufs;
    const uint32_t d_full = done + 8 * kTcDone, d_empty = d_full + 8, run_full = d_empty + 8;
    unsigned char* after = shared + (run_full + 8 - base);
    uint32_t* tmem_at = reinterpret_cast<uint32_t*>(after);
    volatile int* dead = reinterpret_cast<volatile int*>(after + 4);  // a wait ran out: reported at the end
    volatile int* run_at = reinterpret_cast<volatile int*>(after + 8);

    op_release_next();
    if (warp == 0 && lane == 0) {
        for (int i = 0; i < kI8Stages; ++i) {
            op_bar_init(c_full + 8 * i, 1);
            op_bar_init(c_empty + 8 * i, 4);
        }
        for (int i = 0; i < kI8XStages; ++i) {
            op_bar_init(x_full + 8 * i, 1);  // of the even block: both blocks' copies
            op_bar_init(x_empty + 8 * i, 1);
        }
        for (int i = 0; i < kABufs; ++i) op_bar_init(a_full + 8 * i, 8);  // of the even block
        for (int i = 0; i < kTcDone; ++i) op_bar_init(done + 8 * i, 1);
        op_bar_init(d_full, 1);
        op_bar_init(d_empty, 16);  // of the even block
        op_bar_init(run_full, 1);
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

    const int64_t u0 = i8_first(q, cluster_no);
    const int n_units = static_cast<int>(i8_first(q, cluster_no + 1) - u0);
    int64_t tile = u0 / q.k_units;
    int kb = static_cast<int>(u0 - tile * q.k_units);
    // the tile's place among the row blocks and the blocks of tokens, carried along: a 64-bit
    // division per unit costs the warps that fetch as much time as the unit's copies take
    int row_tile = static_cast<int>(tile / q.m_tiles);
    int m_tile = static_cast<int>(tile - int64_t{row_tile} * q.m_tiles);
    // A warp waits; false once a wait has run out, here or in another warp.
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (__all_sync(0xffffffffu, op_bar_try(bar, parity))) return true;
        const bool ok = *dead == 0 && op_bar_wait_slow(bar, parity, q.limit_ns);
        if (__all_sync(0xffffffffu, ok)) return true;
        if (lane == 0) *dead = 1;
        __syncwarp();
        return false;
    };
    auto next_tile = [&] {
        kb = 0;
        ++tile;
        if (++m_tile == q.m_tiles) m_tile = 0, ++row_tile;
    };
    auto next_unit = [&] {
        if (++kb == q.k_units) next_tile();
    };
    auto first_row = [&] { return (int64_t{row_tile} * kWideCluster + rank) * kTcRows; };
    auto first_token = [&] { return int64_t{m_tile} * q.tokens; };

    if (warp == 0) {
        // ------------------------------------------------------------ B
        // No wait for tg_i8_expand: B is not its work, and it let this kernel start only after
        // everything before it was done.
        int issued = 0;
        for (int i = 0; i < n_units; ++i, next_unit()) {
            const int s = i % kI8Stages;
            if (i >= kI8Stages && !wait(c_empty + 8 * s, (i / kI8Stages - 1) & 1)) break;
            if (lane == 0 && !(q.inject == 1 && blockIdx.x == 0 && i == 0)) {
                const uint32_t bar = c_full + 8 * s;
                op_bar_expect(bar, kI8CodeBytes);
                op_tma_2d(cs + s * kI8CodeBytes, &codes, bar, kb * kTcK, static_cast<uint32_t>(first_row()));
            }
            issued = i + 1;
        }
        // copies under way have to land before the block ends
        bool ok = true;
        for (int i = issued > kI8Stages ? issued - kI8Stages : 0; ok && i < issued; ++i)
            if (lane == 0) ok = op_bar_wait(c_full + 8 * (i % kI8Stages), i / kI8Stages & 1, kTcLandNs);
    } else if (warp == 2) {
        // ------------------------------------------------------------ A
        op_wait_previous();
        const uint32_t part = q.tokens / 2;
        int issued = 0;
        for (int i = 0; i < n_units; ++i, next_unit()) {
            const int s = i % kI8XStages;
            if (i >= kI8XStages && !wait(x_empty + 8 * s, (i / kI8XStages - 1) & 1)) break;
            if (lane == 0) {
                const uint32_t to = xs + s * kI8XBytes, bar = wide_at(x_full + 8 * s, 0);
                const uint32_t m = static_cast<uint32_t>(first_token()) + rank * part;
                if (rank == 0) op_bar_expect(x_full + 8 * s, q.tokens * 256);
                wide_tma(to, &order, bar, kb * kTcK, m);
                wide_tma(to + part * 128, &order, bar, kb * kTcK + 64, m);
            }
            issued = i + 1;
        }
        // the copies have to land, and the commits to arrive, before this block ends
        bool ok = true;
        for (int i = issued > kI8XStages ? issued - kI8XStages : 0; ok && i < issued; ++i)
            if (lane == 0) ok = op_bar_wait(x_empty + 8 * (i % kI8XStages), i / kI8XStages & 1, kTcLandNs);
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMAs
        const uint32_t idesc = (1u << 4) | (static_cast<uint32_t>(q.tokens >> 3) << 17) | (16u << 24);
        int issued = 0, runs = 0, taken = 0;  // units of this run
        int limit = kI8WideRun;  // of this run, once known
        bool known = false;
        for (int i = 0; rank == 0 && i < n_units; ++i) {
            const int s = i % kI8XStages, a = i % kABufs;
            const bool first = i == 0 || kb == 0;
            if (!wait(x_full + 8 * s, i / kI8XStages & 1)) break;
            if (taken == 0 && runs++ > 0 && !wait(d_empty, runs & 1)) break;
            if (!wait(a_full + 8 * a, i / kABufs & 1)) break;
            tc_after_sync();
            wide_unit<true>(d_cols, tmem + kACols * a, tc_desc(xs + s * kI8XBytes), q.tokens / 2 * 128 / 16, idesc,
                            first ? 0 : 1, done + 8 * (i % kTcDone), x_empty + 8 * s);
            issued = i + 1;
            // (as little as can be: what this warp does for a unit, all of its units wait for)
            const bool end = kb + 1 == q.k_units || i + 1 == n_units;
            if (end || ++taken == limit) {
                if (!end && !known) {
                    if (!wait(run_full, 0)) break;
                    known = true;
                    limit = run_at[0];
                }
                if (end || taken == limit) {
                    wide_commit(d_full);
                    taken = 0;
                    if (known) limit = run_at[end ? 0 : 1];
                }
            }
            next_unit();
        }
        // the MMAs have to be over before the tensor memory is given back
        if (issued > 0 && lane == 0)
            op_bar_wait(done + 8 * ((issued - 1) % kTcDone), (issued - 1) / kTcDone & 1, kTcLandNs);
        __syncwarp();
    } else if (warp == 3) {
        // ------------------------------------------------------------ the length of a run
        if (q.peaks != nullptr) {
            op_wait_previous();
            const int2 most = i8_runs(q, lane);
            if (lane == 0) {
                run_at[0] = most.x;
                run_at[1] = most.y;
                tc_arrive(run_full);
            }
            __syncwarp();
        }
    } else if (warp >= 8 && warp < 20) {
        // ------------------------------------------------------------ decoding
        const int group = (warp - 8) >> 2;
        const uint32_t row = 32 * (warp & 3) + lane;
        const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        for (int i = group; i < n_units; i += kTcGroups) {
            const int s = i % kI8Stages, a = i % kABufs;
            if (!wait(c_full + 8 * s, i / kI8Stages & 1)) break;
            const uint32_t at = cs + s * kI8CodeBytes + row * 128;
            uint4 w[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) w[c] = tc_lds128(at + ((c ^ (row & 7)) << 4));
            const int old = i - kABufs;
            if (old >= 0 && !wait(done + 8 * (old % kTcDone), old / kTcDone & 1)) break;
            tc_after_sync();
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t r[16];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint4 x = w[2 * c + j];
                    i8_decode(x.x, r[8 * j], r[8 * j + 1]);
                    i8_decode(x.y, r[8 * j + 2], r[8 * j + 3]);
                    i8_decode(x.z, r[8 * j + 4], r[8 * j + 5]);
                    i8_decode(x.w, r[8 * j + 6], r[8 * j + 7]);
                }
                tc_store16(tmem + lanes + kACols * a + 16 * c, r);
            }
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            tc_before_sync();
            __syncwarp();
            if (lane == 0) {
                wide_arrive(wide_at(a_full + 8 * a, 0));
                // not before the codes have been used (see gemm_w4_wide.cuh)
                tc_arrive(c_empty + 8 * s);
            }
        }
    } else if (warp >= 4) {
        // ------------------------------------------------------------ C
        op_wait_previous();
        const int quarter = warp & 3, set = warp < 8 ? 0 : 1;
        const uint32_t row = 32 * quarter + lane;
        const uint32_t at = d_cols + (static_cast<uint32_t>(32 * quarter) << 16);
        auto release = [&] {  // the sums have been read
            tc_before_sync();
            __syncwarp();
            if (lane == 0) wide_arrive(wide_at(d_empty, 0));
        };
        int i = 0;
        uint32_t runs = 0;
        bool ok = true;
        while (ok && i < n_units) {
            const int len = q.k_units - kb < n_units - i ? q.k_units - kb : n_units - i;
            const int64_t n = first_row() + row, m0 = first_token();
            const int tokens = static_cast<int>(p.M - m0 < q.tokens ? p.M - m0 : q.tokens);
            const bool whole = len == q.k_units;
            int end = len, more = 0;  // of the first run, units of the others
            if (len > kI8WideRun) {
                if (!wait(run_full, 0)) break;
                end = run_at[0];
                more = run_at[1];
            }
            // What the epilogue needs is here before the sums are: the MMAs of the next tile wait
            // for these to be read.
            const float bias = p.bias != nullptr && n < p.N ? p.bias[n] : 0.0f;
            const float sb = n < p.N ? p.sb[n] : 0.0f;
            float scales[kI8Tokens / 64];  // of this warp's tokens, 32 in each
#pragma unroll
            for (int g = 0; g < kI8Tokens / 64; ++g) {
                const int c = 64 * g + 32 * (lane >> 4) + 16 * set + (lane & 15);
                scales[g] = c < tokens ? p.sa[m0 + c] : 0.0f;
            }
            // those of the next 16 tokens, in lanes from `first` on
            int first = 0;
            auto next_scales = [&] {
                if (first == 16) {
                    const float f = scales[0];
#pragma unroll
                    for (int g = 0; g + 1 < kI8Tokens / 64; ++g) scales[g] = scales[g + 1];
                    scales[kI8Tokens / 64 - 1] = f;
                }
                first ^= 16;
            };
            int head = 0, tail = 0;  // of the clusters that share the tile
            if (!whole) {
                if (q.parts > 0) {
                    head = static_cast<int>(tile) * q.parts;
                    tail = head + q.parts - 1;
                } else {
                    head = static_cast<int>(tc_block_of(q.units, q.clusters, tile * q.k_units));
                    tail = static_cast<int>(tc_block_of(q.units, q.clusters, (tile + 1) * q.k_units - 1));
                }
            }
            // (of a whole tile a place of the cluster's own, not zeroed)
            const int place = whole ? q.places + cluster_no : q.by_tile ? static_cast<int>(tile) : head;
            int32_t* const sums = q.sums + int64_t{place * kWideCluster + rank} * q.tokens * kTcRows + row;
            uint32_t given = 0;  // of a whole tile: the tokens / 32 whose place has sums
            auto give = [&](int c, const uint32_t (&r)[16]) {
#pragma unroll
                for (int m = 0; m < 16; ++m)
                    asm volatile("red.relaxed.gpu.global.add.s32 [%0], %1;" ::"l"(sums + (c + m) * kTcRows),
                                 "r"(__float2int_rn(__uint_as_float(r[m])))
                                 : "memory");
            };
            for (; end < len; end += more) {  // a run that is not the last one
                // (a barrier of its own: a parity says nothing of a phase further off than one)
                if (!(ok = wait(d_full, runs++ & 1))) break;
                tc_after_sync();
                for (int c = 16 * set; c < tokens; c += 32) {
                    uint32_t r[16];
                    tc_load(at + c, r);
                    bool large = false;
#pragma unroll
                    for (int m = 0; m < 16; ++m) large = large || fabsf(__uint_as_float(r[m])) > kI8Keep;
                    if (!__any_sync(0xffffffffu, large)) continue;
                    if (whole && (given >> (c / 32) & 1) == 0) {
#pragma unroll
                        for (int m = 0; m < 16; ++m)
                            asm volatile("st.relaxed.gpu.global.s32 [%0], %1;" ::"l"(sums + (c + m) * kTcRows),
                                         "r"(__float2int_rn(__uint_as_float(r[m])))
                                         : "memory");
                        given |= 1u << (c / 32);
                    } else {
                        give(c, r);
                    }
#pragma unroll
                    for (int m = 0; m < 16; ++m) r[m] = 0;
                    tc_store16(at + c, r);
                }
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                release();
            }
            if (!ok || !(ok = wait(d_full, runs++ & 1))) break;
            tc_after_sync();
            if (16 * set >= tokens) release();  // (no tokens for this warp)
            for (int c = 16 * set; c < tokens; c += 32) {
                uint32_t r[16];
                __syncwarp();
                tc_load(at + c, r);
                if (c + 32 >= tokens) release();
                if (whole) {
                    float v[16];
#pragma unroll
                    for (int m = 0; m < 16; ++m) v[m] = __uint_as_float(r[m]);
                    if (given >> (c / 32) & 1) {
#pragma unroll
                        for (int m = 0; m < 16; ++m)
                            v[m] = static_cast<float>(i8_load(sums + (c + m) * kTcRows) + __float2int_rn(v[m]));
                    }
                    i8_wide_store<TC>(p, m0 + c, n, tokens - c, scales[0], first, sb, bias, v);
                    next_scales();
                } else {
                    give(c, r);
                }
            }
            if (!whole) {  // a share of a tile
                __syncwarp();
                uint32_t before = 0;
                if (lane == 0) {  // (its release and acquire are those of the warp, by the barriers around)
                    uint32_t* count = q.counters + 8 * (head * kWideCluster + rank) + 4 * set + quarter;
                    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;"
                                 : "=r"(before)
                                 : "l"(count)
                                 : "memory");
                }
                before = __shfl_sync(0xffffffffu, before, 0);
                __syncwarp();
                if (before == static_cast<uint32_t>(tail - head)) {
                    for (int c = 16 * set; c < tokens; c += 32) {
                        float v[16];
#pragma unroll
                        for (int m = 0; m < 16; ++m) v[m] = static_cast<float>(i8_load(sums + (c + m) * kTcRows));
                        __syncwarp();
                        i8_wide_store<TC>(p, m0 + c, n, tokens - c, scales[0], first, sb, bias, v);
                        next_scales();
                    }
                }
            }
            i += len;
            next_tile();
        }
    }
    tc_before_sync();
    __syncthreads();
    if (threadIdx.x == 0 && *dead != 0) atomicOr(q.timeouts, kOpTimeoutI8);
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
