// Products of up to 64 rows of A with 4-bit weights, on tcgen05: W·Aᵀ with W decoded
// into tensor memory.
//
// The weights are the MMA's A operand (128 rows of W by 128 k, a "unit"), and go
// there exactly: a thread owns a row, turns its words of 8 codes into pairs
// (c_i - z, c_i+4 - z) as in gemm_w4.cuh (fp16: nine instructions for 8 codes, bf16:
// eleven) and stores them with tcgen05.st; nothing decoded touches shared memory.  The
// rows of A ("tokens") are the B operand, laid out beforehand with each 8 values in the
// order of the pairs.  Every product is exact, the sums are fp32.
//
// The scales are per row of W and group of k, so a group's sum is an accumulator of its
// own: 128 / G of them per unit, each of NP columns (the tokens, padded), read back and
// added, times the row's scale, to the sums that a thread keeps in registers.
//
// Roles of a block's 20 warps, or 24 for 64 columns (all meet on mbarriers):
//   0      fetches codes, scales and zero points by TMA, kTcCodeStages units ahead
//   1      issues the MMAs of a unit, and one commit
//   2      fetches A by TMA
//   4-7    read the accumulators back (a quarter of the rows each), scale and sum,
//          and write C; of 64 columns warps 20-23 have the upper 32
//   8-19   decode, in three groups of four warps that take units in turn
// The blocks share all units (row block by row block, k inside) evenly.  Where a row
// block is shared, each block leaves its sums in the workspace, and the last one to
// come adds all of them, in the order of k: the same bits every time.
//
// What bounds it: the turn of a unit through its accumulator (issue, MMAs, wake-up, read
// back, release), about 0.4 us with 16 columns, where an SM could get the unit's codes in
// 0.19.  A wait costs 80 to 110 cycles even when there is nothing to wait for, so the MMA
// warp has one barrier for all that a unit needs.  Measured: 16384×8192, G = 128, 16 / 32 /
// 64 rows 28.8 / 32.8 / 41.4 us (2.5 / 2.1 / 1.7 TB/s; with three barriers per unit 31.0 /
// 34.3 / 45.4), G = 32 with 64 rows 52 us (one accumulator only).
#pragma once

#include "gemm_w4.cuh"

namespace tg {

// Depths of the rings, all divisors of kTcTurn: the MMA warp's loop is unrolled that far,
// and its addresses and parities are constants.
constexpr int kTcTurn = 8;
constexpr int kTcCodeStages = 8;
constexpr int kTcCodeBytes = 10240;   // codes 8192, scales ≤ 1024, zero points ≤ 512
constexpr int kTcScaleAt = 8192;
constexpr int kTcZeroAt = 9216;
constexpr int kTcXStages = 4;
constexpr int kTcABufs = 4;

template <int G, int NP>
struct TcShape {
    static constexpr int kGroups = kTcK / G;     // of k in a unit
    static constexpr int kDCols = NP * kGroups;  // accumulator columns of a unit
    static constexpr int kDBufs = 2 * kDCols <= 256 ? 2 : 1;
    static_assert(kTcXStages == kTcABufs, "one barrier for both");
    static_assert(64 * kTcABufs + kDBufs * kDCols <= 512, "tensor memory");
    static constexpr int kXBytes = NP * 256;     // two boxes of 64 k
    static constexpr int kCols = NP < 32 ? NP : 32;  // of a thread's sums
    static constexpr int kSets = NP / kCols;         // of summing warps
    static constexpr int kThreads = 32 * (16 + 4 * kSets);
    static constexpr int kSmem = 1024 + kTcXStages * kXBytes + kTcCodeStages * kTcCodeBytes + 512;
};

struct TcLaunch {
    W4Params p;
    uint64_t limit_ns;
    unsigned int* timeouts;  // set where a warp gives up on a wait
    int32_t inject;     // 1: block 0's first codes are left out (for tests of the limit)
    int64_t units;      // in all
    int32_t k_units;    // per row block
    float* slots;       // two per block: the sums of its first and last row block
    uint32_t* counters;  // eight per block
};

// A in the order of the decoded pairs, in rows of `ldo` (a multiple of 128), zero past
// column K: out[8q + (0 4 1 5 2 6 3 7)] <- a[8q + (0 .. 7)] read by place: 0 4 1 5 2 6 3 7.
__global__ void __launch_bounds__(256)
    tg_w4_order(const uint16_t* __restrict__ A, int64_t lda, int64_t M, int64_t K,
                uint16_t* __restrict__ out, int64_t ldo) {
    op_wait_previous();
    op_release_next();
    const int64_t c = int64_t{blockIdx.x} * 256 + threadIdx.x;
    if (8 * c >= ldo) return;
    const bool wide = (reinterpret_cast<uintptr_t>(A) & 15) == 0 && lda % 8 == 0 && 8 * c + 8 <= K;
    for (int64_t m = blockIdx.y; m < M; m += gridDim.y) {
        const uint16_t* a = A + m * lda;
        uint4 x;
        if (wide) {
            x = *reinterpret_cast<const uint4*>(a + 8 * c);
        } else {
            uint32_t h[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) h[i] = 8 * c + i < K ? a[8 * c + i] : 0;
            x = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
        }
        *reinterpret_cast<uint4*>(out + m * ldo + 8 * c) =
            make_uint4(__byte_perm(x.x, x.z, 0x5410), __byte_perm(x.x, x.z, 0x7632),
                       __byte_perm(x.y, x.w, 0x5410), __byte_perm(x.y, x.w, 0x7632));
    }
}

// The MMAs of a unit and the commit that reports them to `bar`, issued by one lane of
// a converged warp.  In one block, with operands that are the same in all lanes: the
// addresses then stay in uniform registers.  (Eight blocks with an election each took
// about 1500 cycles per unit, four times the MMAs.)  d, a: columns of tensor memory, b: A's
// descriptor; every G / 16 MMAs the next group's accumulator, NP columns on.
template <int G, int NP>
__device__ __forceinline__ void tc_unit(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t bar) {
    constexpr int kBox = NP * 128 / 16;  // the second 64 k, in the descriptor's 16 bytes
    asm volatile(
        "{\n\t.reg .pred e, zero, one;\n\t.reg .b32 ak, dk;\n\t.reg .b64 bk;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 zero, 0, 0;\n\tsetp.eq.b32 one, 0, 0;\n\t"
        "add.u32 dk, %0, %5;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [dk], [%1], %2, %3, zero;\n\t"
        "add.u32 ak, %1, 8;\n\tadd.u64 bk, %2, 2;\n\tadd.u32 dk, %0, %6;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [dk], [ak], bk, %3, one;\n\t"
        "add.u32 ak, %1, 16;\n\tadd.u64 bk, %2, 4;\n\tadd.u32 dk, %0, %7;\n\t"
        "setp.ne.b32 zero, %14, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [dk], [ak], bk, %3, zero;\n\t"
        "add.u32 ak, %1, 24;\n\tadd.u64 bk, %2, 6;\n\tadd.u32 dk, %0, %8;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [dk], [ak], bk, %3, one;\n\t"
        "add.u32 ak, %1, 32;\n\tadd.u64 bk, %2, %13;\n\tadd.u32 dk, %0, %9;\n\t"
        "setp.ne.b32 zero, %15, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [dk], [ak], bk, %3, zero;\n\t"
        "add.u64 bk, bk, 2;\n\tadd.u32 ak, %1, 40;\n\tadd.u32 dk, %0, %10;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [dk], [ak], bk, %3, one;\n\t"
        "add.u64 bk, bk, 2;\n\tadd.u32 ak, %1, 48;\n\tadd.u32 dk, %0, %11;\n\t"
        "setp.ne.b32 zero, %14, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [dk], [ak], bk, %3, zero;\n\t"
        "add.u64 bk, bk, 2;\n\tadd.u32 ak, %1, 56;\n\tadd.u32 dk, %0, %12;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [dk], [ak], bk, %3, one;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%4];\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(bar), "n"(0), "n"(16 / G * NP), "n"(32 / G * NP),
        "n"(48 / G * NP), "n"(64 / G * NP), "n"(80 / G * NP), "n"(96 / G * NP), "n"(112 / G * NP),
        "n"(kBox), "n"(G > 32 ? 1 : 0), "n"(G > 64 ? 1 : 0)
        : "memory");
}
template <typename T, int G, int NP, bool ZERO>
__global__ void __launch_bounds__((TcShape<G, NP>::kThreads), 1)
    tg_gemm_w4_tc(const __grid_constant__ TcLaunch q, const __grid_constant__ CUtensorMap codes,
                  const __grid_constant__ CUtensorMap scales,
                  const __grid_constant__ CUtensorMap zeros, const __grid_constant__ CUtensorMap order) {
    using S = TcShape<G, NP>;
    extern __shared__ __align__(1024) unsigned char tc_dynamic[];
    const W4Params& p = q.p;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t base = (op_smem(tc_dynamic) + 1023) & ~1023u;
    unsigned char* const tc_shared = tc_dynamic + (base - op_smem(tc_dynamic));
    const uint32_t xs = base, cs = xs + kTcXStages * S::kXBytes;
    const uint32_t bars = cs + kTcCodeStages * kTcCodeBytes;
    const uint32_t c_full = bars, c_empty = c_full + 8 * kTcCodeStages;
    const uint32_t ready = c_empty + 8 * kTcCodeStages, done = ready + 8 * kTcABufs;
    unsigned char* after = tc_shared + (done + 8 * kTcDone - base);
    uint32_t* tmem_at = reinterpret_cast<uint32_t*>(after);
    volatile int* dead = reinterpret_cast<volatile int*>(after + 4);  // a wait ran out: reported at the end

    op_release_next();
    if (warp == 0 && lane == 0) {
        for (int i = 0; i < kTcCodeStages; ++i) {
            op_bar_init(c_full + 8 * i, 1);
            op_bar_init(c_empty + 8 * i, 4 + 4 * S::kSets);  // decoded, and summed up
        }
        // all that a unit's MMAs wait for: W decoded, A's copies, the accumulator read
        for (int i = 0; i < kTcABufs; ++i) op_bar_init(ready + 8 * i, 4 + 1 + 4 * S::kSets);
        for (int i = 0; i < kTcDone; ++i) op_bar_init(done + 8 * i, 1);
        op_bar_init_done();
        *dead = 0;
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                         op_smem(tmem_at))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    // all columns are this block's, so they begin at 0 (known here, the addresses below
    // are the same in all lanes for the compiler too)
    constexpr uint32_t tmem = 0;
    constexpr uint32_t d_cols = tmem + 64 * kTcABufs;

    const int64_t u0 = tc_first(q.units, gridDim.x, blockIdx.x);
    const int n_units = static_cast<int>(tc_first(q.units, gridDim.x, blockIdx.x + 1) - u0);
    int64_t row_block = u0 / q.k_units;
    int kb = static_cast<int>(u0 - row_block * q.k_units);
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
        if (++kb == q.k_units) kb = 0, ++row_block;
    };

    if (warp == 0) {
        // ------------------------------------------------------------ codes
        // The weights are not the ordering kernel's work, and that kernel let this one
        // start only after everything before it was done: no wait here.
        int issued = 0;
        for (int i = 0; i < n_units; ++i, next_unit()) {
            const int s = i % kTcCodeStages;
            const uint32_t old = (i / kTcCodeStages - 1) & 1;
            if (i >= kTcCodeStages && !wait(c_empty + 8 * s, old)) break;
            if (lane == 0) {
                const uint32_t to = cs + s * kTcCodeBytes, bar = c_full + 8 * s;
                const uint32_t n = static_cast<uint32_t>(row_block) * kTcRows;
                if (!(q.inject == 1 && blockIdx.x == 0 && i == 0)) {
                    op_bar_expect(bar, 8192 + (ZERO ? 384 : 256) * S::kGroups);
                    op_tma_2d(to, &codes, bar, kb * 64, n);
                    op_tma_2d(to + kTcScaleAt, &scales, bar, n, kb * S::kGroups);
                    if (ZERO) op_tma_2d(to + kTcZeroAt, &zeros, bar, n, kb * S::kGroups);
                }
            }
            issued = i + 1;
        }
        // copies under way have to land before the block ends
        for (int i = issued > kTcCodeStages ? issued - kTcCodeStages : 0; i < issued; ++i)
            if (lane == 0) op_bar_wait(c_full + 8 * (i % kTcCodeStages), i / kTcCodeStages & 1, kTcLandNs);
    } else if (warp == 2) {
        // ------------------------------------------------------------ A
        op_wait_previous();
        int issued = 0;
        for (int i = 0; i < n_units; ++i, next_unit()) {
            const int s = i % kTcXStages;
            const int old = i - kTcXStages;
            if (old >= 0 && !wait(done + 8 * (old % kTcDone), old / kTcDone & 1)) break;
            if (lane == 0) {
                const uint32_t to = xs + s * S::kXBytes, bar = ready + 8 * s;
                op_bar_expect(bar, S::kXBytes);
                op_tma_2d(to, &order, bar, kb * kTcK, 0);
                op_tma_2d(to + S::kXBytes / 2, &order, bar, kb * kTcK + 64, 0);
            }
            issued = i + 1;
        }
        // copies under way have to land before the block ends: with their units' MMAs
        bool ok = true;
        for (int i = issued > kTcXStages ? issued - kTcXStages : 0; ok && i < issued; ++i)
            if (lane == 0) ok = op_bar_wait(done + 8 * (i % kTcDone), i / kTcDone & 1, kTcLandNs);
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMAs
        constexpr uint32_t fmt = std::is_same<T, __half>::value ? 0u : 1u;
        constexpr uint32_t idesc = (1u << 4) | (fmt << 7) | (fmt << 10) | ((NP >> 3) << 17) | (8u << 24);
        int issued = 0;
        bool ok = true;
        for (int i0 = 0; ok && i0 < n_units; i0 += kTcTurn) {
#pragma unroll
            for (int j = 0; j < kTcTurn; ++j) {
                if (i0 + j >= n_units) break;
                const int a = j % kTcABufs, d = j % S::kDBufs;
                ok = wait(ready + 8 * a, j / kTcABufs & 1);
                if (!ok) break;
                tc_after_sync();
                tc_unit<G, NP>(d_cols + d * S::kDCols, tmem + 64 * a, tc_desc(xs + a * S::kXBytes), idesc,
                               done + 8 * j);
                issued = i0 + j + 1;
            }
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
            const int s = i % kTcCodeStages, a = i % kTcABufs;
            if (!wait(c_full + 8 * s, i / kTcCodeStages & 1)) break;
            const uint32_t at = cs + s * kTcCodeBytes;
            uint4 w[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) w[c] = tc_lds128(at + row * 64 + ((c ^ (row >> 1 & 3)) << 4));
            uint32_t z[S::kGroups];
#pragma unroll
            for (int c = 0; c < S::kGroups; ++c)
                z[c] = ZERO ? tc_shared[at - base + kTcZeroAt + c * kTcRows + row] & 15u : 8u;
            const int old = i - kTcABufs;
            if (old >= 0 && !wait(done + 8 * (old % kTcDone), old / kTcDone & 1)) break;
            tc_after_sync();
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const W4Decode<T> decode(z[c * 32 / G]);
                const uint32_t words[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
                uint32_t r[16];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t v[4];
                    decode(words[j], v);
#pragma unroll
                    for (int e = 0; e < 4; ++e) r[4 * j + e] = v[e];
                }
                tc_store16(tmem + lanes + 64 * a + 16 * c, r);
            }
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            tc_before_sync();
            __syncwarp();
            if (lane == 0) {
                tc_arrive(ready + 8 * a);
                // not before the codes have been used: with the arrival right behind the
                // loads, stages were refilled before these had taken effect
                tc_arrive(c_empty + 8 * s);
            }
        }
    } else if (warp >= 4) {
        // ------------------------------------------------------------ sums and C
        op_wait_previous();
        const int quarter = warp & 3;
        const uint32_t row = 32 * quarter + lane;
        const uint32_t lanes = static_cast<uint32_t>(32 * quarter) << 16;
        constexpr int NC = S::kCols;
        const int set = warp < 8 ? 0 : 1, m0 = set * NC;
        const int tokens = static_cast<int>(p.M) - m0;  // from this thread's first column on
        float sum[NC];
#pragma unroll
        for (int m = 0; m < NC; ++m) sum[m] = 0.0f;
        int kb0 = kb;  // first unit of the row block here
        if (lane == 0)  // the accumulators are empty at first
            for (int i = 0; i < S::kDBufs; ++i) tc_arrive(ready + 8 * i);
        for (int i = 0; i < n_units; ++i) {
            const int s = i % kTcCodeStages, d = i % S::kDBufs;
            // (the scales came with the codes, and those were decoded)
            if (!wait(done + 8 * (i % kTcDone), i / kTcDone & 1)) break;
            tc_after_sync();
            float scale[S::kGroups];
#pragma unroll
            for (int c = 0; c < S::kGroups; ++c)
                scale[c] = op_to_float(*reinterpret_cast<const T*>(
                    tc_shared + (cs - base) + s * kTcCodeBytes + kTcScaleAt + (c * kTcRows + row) * 2));
            const uint32_t at = d_cols + lanes + d * S::kDCols;
            if constexpr (NP == 16 && S::kGroups > 1) {  // two groups at a time
#pragma unroll
                for (int c = 0; c < S::kGroups; c += 2) {
                    uint32_t r[32];
                    tc_load(at + c * NP, r);
#pragma unroll
                    for (int m = 0; m < 16; ++m)
                        sum[m] = fmaf(scale[c + 1], __uint_as_float(r[16 + m]),
                                      fmaf(scale[c], __uint_as_float(r[m]), sum[m]));
                }
            } else {
#pragma unroll
                for (int c = 0; c < S::kGroups; ++c) {
                    uint32_t r[NC];
                    tc_load(at + c * NP + m0, r);
#pragma unroll
                    for (int m = 0; m < NC; ++m)
                        sum[m] = fmaf(scale[c], __uint_as_float(r[m]), sum[m]);
                }
            }
            tc_before_sync();
            __syncwarp();
            if (lane == 0) {
                tc_arrive(ready + 8 * ((i + S::kDBufs) % kTcABufs));
                tc_arrive(c_empty + 8 * s);  // the scales have been used, as the codes above
            }
            if (kb + 1 == q.k_units || i + 1 == n_units) {
                const int64_t n = row_block * kTcRows + row;
                bool last = true;
                int64_t head = blockIdx.x, tail = blockIdx.x;
                if (kb0 > 0 || kb + 1 < q.k_units) {  // a share of a row block
                    float* to = q.slots + (2 * int64_t{blockIdx.x} + (kb0 > 0 ? 0 : 1)) * NP * kTcRows +
                                m0 * kTcRows + row;
#pragma unroll
                    for (int m = 0; m < NC; ++m)
                        if (m < tokens) __stcg(to + m * kTcRows, sum[m]);
                    __threadfence();
                    __syncwarp();
                    head = tc_block_of(q.units, gridDim.x, row_block * q.k_units);
                    tail = tc_block_of(q.units, gridDim.x, (row_block + 1) * q.k_units - 1);
                    uint32_t before = 0;
                    if (lane == 0) {
                        uint32_t* count = q.counters + 8 * head + 4 * set + quarter;
                        asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;"
                                     : "=r"(before)
                                     : "l"(count)
                                     : "memory");
                        if (before == static_cast<uint32_t>(tail - head)) *count = 0;  // for the next launch
                    }
                    before = __shfl_sync(0xffffffffu, before, 0);
                    last = before == static_cast<uint32_t>(tail - head);
                    __threadfence();
                    if (last) {  // the head's share is in its second slot, the others' in their first
#pragma unroll
                        for (int m = 0; m < NC; ++m)
                            if (m < tokens)
                                sum[m] = __ldcg(q.slots + ((2 * head + 1) * NP + m0 + m) * kTcRows + row);
                        for (int64_t b = head + 1; b <= tail; ++b)
#pragma unroll
                            for (int m = 0; m < NC; ++m)
                                if (m < tokens)
                                    sum[m] += __ldcg(q.slots + (2 * b * NP + m0 + m) * kTcRows + row);
                    }
                }
                if (last && n < p.N) {
#pragma unroll
                    for (int m = 0; m < NC; ++m)
                        if (m < tokens) w4_store<T>(p, m0 + m, n, sum[m]);
                }
#pragma unroll
                for (int m = 0; m < NC; ++m) sum[m] = 0.0f;
                kb0 = 0;
            }
            next_unit();
        }
    }
    tc_before_sync();
    __syncthreads();
    if (threadIdx.x == 0 && *dead != 0) atomicOr(q.timeouts, kOpTimeoutW4);
    if (warp == 1) {
        tc_after_sync();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(*tmem_at)
                     : "memory");
    }
}

}  // namespace tg
