// Device helpers of the tcgen05 kernels that decode a weight into tensor memory
// (gemm_w4_tc.cuh, gemm_w4_wide.cuh, gemm_i8_wide.cuh): the division of units among blocks,
// tensor-memory accesses, descriptors, and the MMAs and copies of a pair of blocks.
#pragma once

#include "op_device.cuh"

namespace tg {

// What copies under way get to land before a block that gave up on them ends.
constexpr uint64_t kTcLandNs = 1000000000ull;

constexpr int kTcRows = 128;
constexpr int kTcK = 128;
constexpr int kTcGroups = 3;       // of decoding warps
constexpr int kTcDone = 8;            // barriers of finished units
constexpr int kWideCluster = 2;
constexpr int kWideThreads = 768;

__device__ __forceinline__ uint4 tc_lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(a));
    return v;
}
__device__ __forceinline__ void tc_cluster_sync() {
    asm volatile("barrier.cluster.arrive;\n\tbarrier.cluster.wait;" ::: "memory");
}

// First unit of block b, and the block that has unit u.
__host__ __device__ __forceinline__ int64_t tc_first(int64_t units, int64_t blocks, int64_t b) {
    const int64_t more = units % blocks;
    return units / blocks * b + (b < more ? b : more);
}
__device__ __forceinline__ int64_t tc_block_of(int64_t units, int64_t blocks, int64_t u) {
    const int64_t each = units / blocks, more = units % blocks;
    return u < more * (each + 1) ? u / (each + 1) : more + (u - more * (each + 1)) / each;
}

// 16 columns of this warp's lanes from registers.
__device__ __forceinline__ void tc_store16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
// 16 or 32 columns of this warp's lanes to registers.
__device__ __forceinline__ void tc_load(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tc_load(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
          "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]),
          "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tc_before_sync() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_after_sync() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// K-major rows of 64 16-bit values in 128-byte swizzle, 8-row groups 1 KB apart.
__device__ __forceinline__ uint64_t tc_desc(uint32_t saddr) {
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (1ull << 16) | (64ull << 32) |
           (1ull << 46) | (2ull << 61);
}

// Address of this block's `addr` in block `rank` of the pair.
__device__ __forceinline__ uint32_t wide_at(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void wide_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// A box to this block, its bytes to a barrier of either block.
__device__ __forceinline__ void wide_tma(uint32_t dst, const void* map, uint32_t bar, uint32_t x, uint32_t y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile"
        ".mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// The MMAs of a unit, then (LAST) the commits, to `done` and `free` of both blocks.  As
// tc_unit, with one accumulator; `box`: the second 64 k of b, in 16 bytes.
template <bool LAST>
__device__ __forceinline__ void wide_unit(uint32_t d, uint32_t a, uint64_t b, uint32_t box, uint32_t idesc,
                                          uint32_t add, uint32_t done, uint32_t free) {
    asm volatile(
        "{\n\t.reg .pred e, first, one, last;\n\t.reg .b32 ak;\n\t.reg .b64 bk, bx;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 first, %5, 0;\n\tsetp.eq.b32 one, 0, 0;\n\tsetp.ne.b32 last, %9, 0;\n\t"
        "and.pred last, last, e;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %4, first;\n\t"
        "add.u32 ak, %1, 8;\n\tadd.u64 bk, %2, 2;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [ak], bk, %4, one;\n\t"
        "add.u32 ak, %1, 16;\n\tadd.u64 bk, %2, 4;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [ak], bk, %4, one;\n\t"
        "add.u32 ak, %1, 24;\n\tadd.u64 bk, %2, 6;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [ak], bk, %4, one;\n\t"
        "cvt.u64.u32 bx, %3;\n\tadd.u64 bk, %2, bx;\n\tadd.u32 ak, %1, 32;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [ak], bk, %4, one;\n\t"
        "add.u64 bk, bk, 2;\n\tadd.u32 ak, %1, 40;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [ak], bk, %4, one;\n\t"
        "add.u64 bk, bk, 2;\n\tadd.u32 ak, %1, 48;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [ak], bk, %4, one;\n\t"
        "add.u64 bk, bk, 2;\n\tadd.u32 ak, %1, 56;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [ak], bk, %4, one;\n\t"
        "@last tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
        " [%6], %8;\n\t"
        "@last tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
        " [%7], %8;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(box), "r"(idesc), "r"(add), "r"(done), "r"(free),
        "h"(static_cast<uint16_t>(3)), "n"(LAST ? 1 : 0)
        : "memory");
}

// 16 sums of a share, which lie [token / 4][row][token % 4].
__device__ __forceinline__ void wide_load(const float* from, float (&v)[16]) {
#pragma unroll
    for (int m = 0; m < 16; m += 4) {
        const float4 f = __ldcg(reinterpret_cast<const float4*>(from + m * kTcRows));
        v[m] = f.x, v[m + 1] = f.y, v[m + 2] = f.z, v[m + 3] = f.w;
    }
}
// Reports all MMAs so far to a barrier of both blocks.
__device__ __forceinline__ void wide_commit(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
        " [%0], %1;\n\t}" ::"r"(bar),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}
// p + n, not before it is needed: sixteen addresses at once do not fit the registers.
template <typename P>
__device__ __forceinline__ P* wide_step(P* p, int64_t n) {
    P* r;
    asm volatile("add.s64 %0, %1, %2;" : "=l"(r) : "l"(p), "l"(n));
    return r;
}

}  // namespace tg
