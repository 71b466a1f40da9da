// The norms after and before a block, fused with the block's gate, its
// residual scale and the residual sum, and their gradient.
//
//   m = x · rx,  rx = 1 / sqrt(mean_c x² + eps)       o = m · wpost   (or o = x)
//   y = r + s · g ⊙ o                                  (the residual stream)
//   n = y · ry,  ry = 1 / sqrt(mean_c y² + eps)       h = n · wpre
//
// Gradient, with dy and dh given (means over the row's columns):
//   dn = dh · wpre            dy' = dy + ry (dn - n · mean(dn n))     dr = dy'
//   do' = s · dy'             dg = Σ do' ⊙ o over the rows of a gate
//   do = do' ⊙ g              dm = do · wpost
//   dx = rx (dm - m · mean(dm m))
//   dwpre = Σ_rows dh ⊙ n     dwpost = Σ_rows do ⊙ m
//
// Every value is held in fp32; x, r, y, h and the gradients are rounded once,
// when they are stored (h comes from the unrounded y).
#pragma once

#include "granules.h"
#include "op_device.cuh"

namespace tg {

struct NormParams {
    int64_t rows, cols;
    const void* x;
    int64_t ldx;
    const void* r;
    int64_t ldr;
    const float* wpost;
    const void* gate;
    int64_t ldg;
    int64_t rows_per_gate;
    const float* wpre;
    float scale, eps;
    // forward
    void* y;
    int64_t ldy;
    void* h;
    int64_t ldh;
};

struct NormGradParams {
    NormParams n;
    const void* dy;
    int64_t lddy;
    const void* dh;
    int64_t lddh;
    void* dx;
    int64_t lddx;
    void* dr;
    int64_t lddr;
    void* dgate;
    int64_t lddg;
    float* dwpost;
    float* dwpre;
    // partial sums: ws_post and ws_pre have a row per block, ws_gate a row per
    // piece (a block's rows of one gate); null where nothing is to be summed
    float* ws_post;
    float* ws_pre;
    float* ws_gate;
    int64_t gates;
    int32_t whole_gates;  // a block has all rows of its gates and writes dgate itself
};

// Sum over the block, in a fixed order; every thread gets it.  `red`: 33 floats.
__device__ __forceinline__ float norm_block_sum(float v, float* red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    const int warps = (blockDim.x + 31) / 32;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x / 32] = v;
    __syncthreads();
    if (threadIdx.x < 32) {
        float t = threadIdx.x < warps ? red[threadIdx.x] : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
        if (threadIdx.x == 0) red[32] = t;
    }
    __syncthreads();
    const float total = red[32];
    __syncthreads();
    return total;
}

// First row of block b of `blocks` that share `rows` rows.
__host__ __device__ __forceinline__ int64_t norm_first_row(int64_t rows, int64_t blocks,
                                                           int64_t b) {
    return rows / blocks * b + (rows % blocks < b ? rows % blocks : b);
}

// ------------------------------------------------------------------ rows in a ring
//
// A thread has 8·CH columns of a row.  VEC: runs of 8 neighbours, 16 bytes of a
// 16-bit type (every row 16-byte aligned, cols a multiple of 8); else columns
// blockDim.x apart, so that a warp's accesses are consecutive.
//
// A block takes consecutive rows.  The rows to come are fetched by cp.async into a
// ring in shared memory, so that their bytes are under way while a row is worked
// on.  VEC: a warp fetches just its own columns and needs no barrier for them; else
// the group fetches the 16-byte granules that hold the row, and reads single values
// out of them.  One gate's row for all rows lies beside the ring, others' come with theirs.
//
// Measured, 8192×4096: bf16 53 us (5.1 TB/s), with an fp32 stream 71 us (5.7 TB/s of the
// 6.8 that a copy reaches); unaligned rows are bound by the issue of single-value
// accesses: 1021×5119 fp16, a gate per row, 32 us.

// Two fp32 values, for the packed instructions (a row's arithmetic is issue-bound
// without them).
typedef unsigned long long F2;
__device__ __forceinline__ F2 f2(float a, float b) {
    F2 d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float2 f2_get(F2 a) {
    float2 d;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(a));
    return d;
}
__device__ __forceinline__ F2 f2_mul(F2 a, F2 b) {
    F2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ F2 f2_fma(F2 a, F2 b, F2 c) {
    F2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ float f2_sum(F2 a) {
    const float2 v = f2_get(a);
    return v.x + v.y;
}

// 32 bits of T (one or two values) to fp32.
template <typename T>
__device__ __forceinline__ F2 f2_unpack(uint32_t u) {
    if constexpr (sizeof(T) == 2) {
        const T* e = reinterpret_cast<const T*>(&u);
        return f2(op_to_float(e[0]), op_to_float(e[1]));
    }
    return 0;
}
template <typename T>
__device__ __forceinline__ uint32_t f2_pack(F2 a) {
    const float2 v = f2_get(a);
    alignas(4) const T e[2] = {op_round<T>(v.x), op_round<T>(v.y)};
    return *reinterpret_cast<const uint32_t*>(e);
}
template <>
__device__ __forceinline__ uint32_t f2_pack<__half>(F2 a) {
    const __half2 h = __float22half2_rn(f2_get(a));
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t f2_pack<__nv_bfloat16>(F2 a) {
    const __nv_bfloat162 h = __float22bfloat162_rn(f2_get(a));
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint64_t norm_pair(uint32_t lo, uint32_t hi) {
    return static_cast<uint64_t>(hi) << 32 | lo;
}

// 8 values of T from an aligned place (fp32: in global memory).
template <typename T>
__device__ __forceinline__ void norm_take(const void* src, F2 (&v)[4]) {
    if constexpr (sizeof(T) == 4) {
        float a, b, d, e, f, g, h, i;
        asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=f"(a), "=f"(b), "=f"(d), "=f"(e), "=f"(f), "=f"(g), "=f"(h), "=f"(i)
                     : "l"(src));
        v[0] = f2(a, b), v[1] = f2(d, e), v[2] = f2(f, g), v[3] = f2(h, i);
    } else {
        const uint4 u = *static_cast<const uint4*>(src);
        v[0] = f2_unpack<T>(u.x), v[1] = f2_unpack<T>(u.y);
        v[2] = f2_unpack<T>(u.z), v[3] = f2_unpack<T>(u.w);
    }
}

template <int CH, bool VEC>
struct NormCols {
    int tid, threads, cols;
    __device__ __forceinline__ int at(int ch, int i) const {
        return VEC ? (ch * threads + tid) * 8 + i : (ch * 8 + i) * threads + tid;
    }
    __device__ __forceinline__ bool has(int ch, int i) const { return at(ch, i) < cols; }
    // 8 values of a row in global memory (0 past the last column)
    template <typename T>
    __device__ __forceinline__ void load(const T* row, int ch, F2 (&v)[4]) const {
        if constexpr (VEC) {
            if (has(ch, 0)) {
                norm_take<T>(row + at(ch, 0), v);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = 0;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = f2(has(ch, 2 * i) ? op_to_float(row[at(ch, 2 * i)]) : 0.0f,
                          has(ch, 2 * i + 1) ? op_to_float(row[at(ch, 2 * i + 1)]) : 0.0f);
        }
    }
    template <typename T>
    __device__ __forceinline__ void store(T* row, int ch, const F2 (&v)[4]) const {
        if constexpr (VEC) {
            if (!has(ch, 0)) return;
            T* p = row + at(ch, 0);
            if constexpr (sizeof(T) == 4) {
                // 32 bytes at once: two halves would each fill half of every sector
                const float2 a = f2_get(v[0]), b = f2_get(v[1]), d = f2_get(v[2]), e = f2_get(v[3]);
                asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p),
                             "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(d.x), "f"(d.y), "f"(e.x),
                             "f"(e.y)
                             : "memory");
            } else {
                *reinterpret_cast<uint4*>(p) = make_uint4(f2_pack<T>(v[0]), f2_pack<T>(v[1]),
                                                          f2_pack<T>(v[2]), f2_pack<T>(v[3]));
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = f2_get(v[i]);
                if (has(ch, 2 * i)) row[at(ch, 2 * i)] = op_round<T>(f.x);
                if (has(ch, 2 * i + 1)) row[at(ch, 2 * i + 1)] = op_round<T>(f.y);
            }
        }
    }
};

__device__ __forceinline__ void norm_copy16(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void norm_copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void norm_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}

constexpr int kNormThreads = 512;  // of a block
constexpr int kNormSplit = 8;      // blocks that share a row, at most

// Until the oldest of the stages - 1 groups under way is there (2 to 4 stages).
__device__ __forceinline__ void norm_wait(int stages) {
    if (stages == 4)
        asm volatile("cp.async.wait_group 2;" ::: "memory");
    else if (stages == 3)
        asm volatile("cp.async.wait_group 1;" ::: "memory");
    else
        asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// The threads that share a row: `threads` (a multiple of 32, at most 512) of a
// block; a block has as many such groups as fit into 512 threads.
struct NormGroup {
    int index, count;  // of the block
    int tid, threads;
    float* red;        // 2 × 5 × 16 floats of the group, zero at first
    int turn;          // one sum's shares are still read when the next one's are written

    __device__ __forceinline__ void sync() const {
        if (threads == 32)
            __syncwarp();
        else
            asm volatile("bar.sync %0, %1;" ::"r"(index + 1), "r"(threads) : "memory");
    }
    // Sums over the group in a fixed order, for every thread of it.
    __device__ __forceinline__ float sum(float v) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (threads == 32) return v;
        float* r = red + turn * 80;
        turn ^= 1;
        if ((tid & 31) == 0) r[tid >> 5] = v;
        sync();
        v = r[tid & 15];
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    }
    // Five at once: the lanes share the first four out among themselves, 8 lanes
    // for each, so that 11 exchanges do instead of 25.
    __device__ __forceinline__ void sum5(float (&v)[5]) {
        const int lane = tid & 31;
        const bool b4 = lane & 16, b3 = lane & 8;
        float p = (b4 ? v[2] : v[0]) + __shfl_xor_sync(0xffffffffu, b4 ? v[0] : v[2], 16);
        float q = (b4 ? v[3] : v[1]) + __shfl_xor_sync(0xffffffffu, b4 ? v[1] : v[3], 16);
        float w = (b3 ? q : p) + __shfl_xor_sync(0xffffffffu, b3 ? p : q, 8);  // value lane / 8
        float u = v[4];
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) u += __shfl_xor_sync(0xffffffffu, u, o);
        if (threads > 32) {
            float* r = red + turn * 80;
            turn ^= 1;
            if ((lane & 7) == 0) r[(lane >> 3) * 16 + (tid >> 5)] = w;
            if (lane == 0) r[64 + (tid >> 5)] = u;
            sync();
            const float2 two = reinterpret_cast<const float2*>(r)[lane];
            w = two.x + two.y;
            u = r[64 + (lane & 15)];
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) u += __shfl_xor_sync(0xffffffffu, u, o);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = __shfl_sync(0xffffffffu, w, 8 * k);
        v[4] = u;
    }
};

// Bytes of a stage that a row of T takes: VEC, the threads' columns; else the row
// from the granule of its first byte on.
template <typename T, int CH, bool VEC>
__host__ __device__ constexpr int norm_stage_bytes(int threads, int64_t cols) {
    return VEC ? threads * CH * 8 * static_cast<int>(sizeof(T))
               : static_cast<int>((cols * static_cast<int>(sizeof(T)) + 30) / 16 * 16);
}

// One input that goes through the ring.  Row numbers and strides are 32-bit, their
// products 64-bit.
template <typename T, int CH, bool VEC>
struct NormInput {
    const T* base;         // null: absent
    uint32_t ld;           // elements
    unsigned char* place;  // in stage 0

    __device__ __forceinline__ const unsigned char* row_at(uint32_t row) const {
        return reinterpret_cast<const unsigned char*>(base) +
               static_cast<uint64_t>(row) * ld * sizeof(T);
    }
    // VEC: a 16-byte piece of the stage.  16-bit types: this thread's columns of chunk
    // ch.  fp32: a thread has two pieces of each chunk, and a warp fetches and clears
    // them in the order of memory (lane l the l-th and the l + 32-th), turned so that
    // the reads of both halves fall into all banks.
    static constexpr int kPieces = sizeof(T) / 2;
    __device__ __forceinline__ static int piece(const NormCols<CH, VEC>& c, int ch, int n) {
        if constexpr (kPieces == 1) return ch * c.threads + c.tid;
        return 2 * (ch * c.threads + (c.tid & ~31)) + (n ^ (n >> 3 & 1));
    }
    // first column of the h-th piece that this thread fetches of a chunk
    __device__ __forceinline__ static int piece_col(const NormCols<CH, VEC>& c, int ch, int h) {
        if constexpr (kPieces == 1) return (ch * c.threads + c.tid) * 8;
        return (ch * c.threads + (c.tid & ~31)) * 8 + ((c.tid & 31) + 32 * h) * 4;
    }

    __device__ __forceinline__ void start(const NormCols<CH, VEC>& c, const void* matrix, int64_t ld_,
                                          unsigned char* at, int stages, int stage_bytes) {
        base = static_cast<const T*>(matrix);
        ld = static_cast<uint32_t>(ld_);
        place = at;
        if (VEC && base != nullptr)  // columns past the last are 0, in every stage
#pragma unroll
            for (int ch = 0; ch < CH; ++ch)
#pragma unroll
                for (int h = 0; h < kPieces; ++h)
                    if (piece_col(c, ch, h) >= c.cols)
                        for (int s = 0; s < stages; ++s)
                            *reinterpret_cast<uint4*>(place + s * stage_bytes +
                                                      piece(c, ch, (c.tid & 31) + 32 * h) * 16) =
                                make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void fetch(const NormCols<CH, VEC>& c, int offset, uint32_t row) const {
        if (base == nullptr) return;
        const unsigned char* src = row_at(row);
        const uint32_t dst = static_cast<uint32_t>(__cvta_generic_to_shared(place)) + offset;
        if constexpr (VEC) {
#pragma unroll
            for (int ch = 0; ch < CH; ++ch)
#pragma unroll
                for (int h = 0; h < kPieces; ++h)
                    if (piece_col(c, ch, h) < c.cols)
                        norm_copy16(dst + piece(c, ch, (c.tid & 31) + 32 * h) * 16,
                                    src + piece_col(c, ch, h) * static_cast<int>(sizeof(T)));
        } else {
            // of the last granule, the row's bytes only; a first granule that begins
            // before the matrix does is read value by value
            const Granules g = granules(reinterpret_cast<uint64_t>(base),
                                        static_cast<uint64_t>(row) * ld * sizeof(T),
                                        c.cols * static_cast<int>(sizeof(T)));
            for (int b = c.tid * 16; b < g.end; b += c.threads * 16) {
                const int n = g.end - b < 16 ? g.end - b : 16;
                if (b == 0 && g.outside) {
                    for (int i = g.skip; i < n; i += static_cast<int>(sizeof(T)))
                        *reinterpret_cast<T*>(place + offset + i) =
                            *reinterpret_cast<const T*>(src - g.skip + i);
                } else {
                    norm_copy16(dst + b, src - g.skip + b, n);
                }
            }
        }
    }
    // 8 values of the row; `none` where the input is absent
    __device__ __forceinline__ void get(const NormCols<CH, VEC>& c, int offset, uint32_t row, int ch,
                                        F2 (&v)[4], float none = 0.0f) const {
        if (base == nullptr) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = f2(none, none);
            return;
        }
        const unsigned char* s = place + offset;
        if constexpr (VEC) {
            if constexpr (kPieces == 2) {
                const int n = 2 * (c.tid & 31);
                const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(s + piece(c, ch, n) * 16);
                const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(s + piece(c, ch, n + 1) * 16);
                v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
            } else {
                norm_take<T>(s + piece(c, ch, 0) * 16, v);
            }
        } else {
            const T* t = reinterpret_cast<const T*>(s + (reinterpret_cast<uintptr_t>(row_at(row)) & 15));
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = f2(c.has(ch, 2 * i) ? op_to_float(t[c.at(ch, 2 * i)]) : 0.0f,
                          c.has(ch, 2 * i + 1) ? op_to_float(t[c.at(ch, 2 * i + 1)]) : 0.0f);
        }
    }
};

// The gate goes through the ring with the rows, but for one that all rows share:
// that one lies behind the ring.
__device__ __forceinline__ uint32_t norm_gate_row(uint32_t row, uint32_t per) {
    return per == 1 ? row : row / per;
}

template <int CH, bool VEC>
__device__ __forceinline__ void norm_weight(const float* w, const NormCols<CH, VEC>& c, int ch,
                                            F2 (&v)[4]) {
    if (w != nullptr) {
        c.load(w, ch, v);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = f2(1.0f, 1.0f);
    }
}

__device__ __forceinline__ NormGroup norm_group(int threads, float* red, int red_floats) {
    for (int i = threadIdx.x; i < red_floats; i += blockDim.x) red[i] = 0.0f;
    __syncthreads();
    NormGroup g;
    g.threads = threads;
    g.count = blockDim.x / threads;
    g.index = threadIdx.x / threads;
    g.tid = threadIdx.x % threads;
    g.red = red + (threads > 32 ? g.index * 160 : 0);
    g.turn = 0;
    return g;
}

// `threads`: of a group.  The groups of a block take its rows in turn.
template <typename TX, typename TR, int CH, bool VEC>
__global__ void __launch_bounds__(kNormThreads, CH == 1 && VEC ? 2 : 1)
    tg_norm_residual_rows(const NormParams p, int threads, int stages, int stage_bytes) {
    extern __shared__ __align__(16) unsigned char norm_stage[];
    __shared__ __align__(16) float red[8 * 160];
    NormGroup g = norm_group(threads, red, 8 * 160);
    const NormCols<CH, VEC> c{g.tid, g.threads, static_cast<int>(p.cols)};
    const float inv = 1.0f / static_cast<float>(p.cols);
    const int rows = static_cast<int>(p.rows), per = static_cast<int>(p.rows_per_gate);
    const int row0 = static_cast<int>(norm_first_row(p.rows, gridDim.x, blockIdx.x)) + g.index;
    const int row1 = static_cast<int>(norm_first_row(p.rows, gridDim.x, blockIdx.x + 1));
    const int stride = g.count;
    unsigned char* mine = norm_stage + g.index * stages * stage_bytes;
    const int bx = norm_stage_bytes<TX, CH, VEC>(threads, p.cols);
    const int br = norm_stage_bytes<TR, CH, VEC>(threads, p.cols);
    const bool one_gate = per == rows;
    NormInput<TX, CH, VEC> in_x, in_g;
    NormInput<TR, CH, VEC> in_r;
    in_x.start(c, p.x, p.ldx, mine, stages, stage_bytes);
    in_r.start(c, p.r, p.ldr, mine + bx, stages, stage_bytes);
    if (one_gate)
        in_g.start(c, p.gate, p.ldg, norm_stage + g.count * stages * stage_bytes + g.index * bx, 1, 0);
    else
        in_g.start(c, p.gate, p.ldg, mine + bx + br, stages, stage_bytes);
    int to_fetch = row0;
    auto fetch = [&](int slot) {
        if (to_fetch < row1) {
            in_x.fetch(c, slot * stage_bytes, to_fetch);
            in_r.fetch(c, slot * stage_bytes, to_fetch);
            if (!one_gate) in_g.fetch(c, slot * stage_bytes, norm_gate_row(to_fetch, per));
        }
        to_fetch += stride;
        norm_commit();
    };
    op_release_next();
    op_wait_previous();
    if (one_gate) in_g.fetch(c, 0, 0);
    for (int s = 0; s < stages - 1; ++s) fetch(s);
    int slot = 0;
    for (int row = row0; row < row1; row += stride) {
        norm_wait(stages);
        if (VEC)
            __syncwarp();
        else
            g.sync();
        // the slot before this one is free: all who read its row have come here
        fetch(slot == 0 ? stages - 1 : slot - 1);
        const int at = slot * stage_bytes;
        F2 x[CH][4], y[CH][4];
#pragma unroll
        for (int ch = 0; ch < CH; ++ch) in_x.get(c, at, row, ch, x[ch]);
        float f = p.scale;
        if (p.wpost != nullptr) {
            F2 a = 0;
#pragma unroll
            for (int ch = 0; ch < CH; ++ch)
#pragma unroll
                for (int i = 0; i < 4; ++i) a = f2_fma(x[ch][i], x[ch][i], a);
            f *= rsqrtf(g.sum(f2_sum(a)) * inv + p.eps);
        }
        const F2 ff = f2(f, f);
        F2 a = 0;
#pragma unroll
        for (int ch = 0; ch < CH; ++ch) {
            if (p.wpost != nullptr) {
                F2 w[4];
                c.load(p.wpost, ch, w);
#pragma unroll
                for (int i = 0; i < 4; ++i) x[ch][i] = f2_mul(x[ch][i], w[i]);
            }
            if (in_g.base != nullptr) {
                F2 w[4];
                in_g.get(c, one_gate ? 0 : at, norm_gate_row(row, per), ch, w);
#pragma unroll
                for (int i = 0; i < 4; ++i) x[ch][i] = f2_mul(x[ch][i], w[i]);
            }
            in_r.get(c, at, row, ch, y[ch]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                y[ch][i] = f2_fma(ff, x[ch][i], y[ch][i]);
                a = f2_fma(y[ch][i], y[ch][i], a);
            }
            if (p.y != nullptr)
                c.store(static_cast<TR*>(p.y) + static_cast<uint64_t>(row) * static_cast<uint32_t>(p.ldy),
                        ch, y[ch]);
        }
        if (p.wpre != nullptr) {
            const float ry = rsqrtf(g.sum(f2_sum(a)) * inv + p.eps);
            const F2 rr = f2(ry, ry);
#pragma unroll
            for (int ch = 0; ch < CH; ++ch) {
                F2 w[4];
                c.load(p.wpre, ch, w);
#pragma unroll
                for (int i = 0; i < 4; ++i) y[ch][i] = f2_mul(f2_mul(y[ch][i], rr), w[i]);
                c.store(static_cast<TX*>(p.h) + static_cast<uint64_t>(row) * static_cast<uint32_t>(p.ldh),
                        ch, y[ch]);
            }
        }
        slot = slot + 1 == stages ? 0 : slot + 1;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

template <typename T>
__device__ __forceinline__ const void* norm_at(const void* p, int col) {
    return p != nullptr ? static_cast<const T*>(p) + col : nullptr;
}

// Sums of the blocks of a cluster, over distributed shared memory: each block's values go
// to every block with their bytes counted on its mbarrier.  By the rows' times an exchange
// takes some 0.65 us; with cluster barriers, whose release waits for the stores of the row
// before, 0.85 (2048×8192 bf16 92 us against 104).
template <bool MULTI>
struct NormPeers {
    __device__ __forceinline__ NormPeers(int, int, uint64_t, unsigned int*, bool) {}
    template <int N>
    __device__ __forceinline__ void add(float (&)[N]) {}
    __device__ __forceinline__ void end() {}
};
template <>
struct NormPeers<true> {
    float* values;  // [2][block of the cluster][8]
    uint32_t bars;  // [2]
    int rank, count;
    uint64_t limit_ns;
    unsigned int* timeouts;  // set where a wait for another block runs out
    bool silent;          // for tests of the limit: the first values are not sent
    bool lost = false;    // a wait ran out: reported; nothing more is sent or waited for
    int turn = 0;         // one exchange's values are still read when the next one's come
    uint32_t parity = 0;  // of both barriers

    __device__ __forceinline__ NormPeers(int rank, int count, uint64_t limit_ns, unsigned int* timeouts,
                                         bool silent)
        : rank(rank), count(count), limit_ns(limit_ns), timeouts(timeouts), silent(silent) {
        __shared__ __align__(16) float room[2 * kNormSplit * 8];
        __shared__ __align__(8) unsigned long long two[2];
        values = room;
        bars = op_smem(two);
        if (threadIdx.x == 0) {
            op_bar_init(bars, 1);
            op_bar_init(bars + 8, 1);
            op_bar_init_done();
        }
        sync();  // the other blocks' barriers are there
    }
    __device__ __forceinline__ static void sync() {
        asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
    }
    // The blocks' v (the same in all threads of a block): 8 places for each, until the next but
    // one exchange.
    template <int N>
    __device__ __forceinline__ const float* exchange(const float (&v)[N]) {
        float* all = values + turn * kNormSplit * 8;
        const uint32_t bar = bars + 8 * turn;
        if (threadIdx.x == 0 && !lost) op_bar_expect(bar, count * N * 4);
        if (static_cast<int>(threadIdx.x) < count && !silent && !lost) {  // a thread for each block
            uint32_t to, at;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                         : "=r"(to)
                         : "r"(op_smem(all + rank * 8)), "r"(threadIdx.x));
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(bar), "r"(threadIdx.x));
#pragma unroll
            for (int k = 0; k < N; ++k)
                asm volatile(
                    "st.async.shared::cluster.mbarrier::complete_tx::bytes.f32 [%0], %1, [%2];" ::"r"(to + 4 * k),
                    "f"(v[k]), "r"(at)
                    : "memory");
        }
        silent = false;
        if (!lost && !op_bar_wait(bar, parity, limit_ns)) {
            lost = true;
            atomicOr(timeouts, kOpTimeoutNorm);
        }
        turn ^= 1;
        if (turn == 0) parity ^= 1;
        return all;
    }
    // Their sums, in the order of the blocks.
    template <int N>
    __device__ __forceinline__ void add(float (&v)[N]) {
        const float* all = exchange(v);
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = all[k];
        for (int b = 1; b < count; ++b)
#pragma unroll
            for (int k = 0; k < N; ++k) v[k] += all[b * 8 + k];
    }
    // No block leaves while another's values may be on their way to it.
    __device__ __forceinline__ void end() { sync(); }
};

// Gradient.  A thread keeps its columns' sums over its rows in registers; a block
// joins its groups' sums in shared memory and writes one share.  Two reductions per
// row: with t = o·g (so y = r + s·t) first Σ x² for rx, then
//   Σ y², Σ dn·y, Σ t·dy, Σ t·dn, Σ t·y,
// for the rest is linear in these: with c = ry²·mean(dn·y),
//   dy' = dy + ry·(dn - c·y)   and   Σ dm·m = s·(Σ t·dy + ry·(Σ t·dn - c·Σ t·y)).
//
// whole_gates: a group takes all rows of its gates, and writes their gradients
// itself.  Else the groups of a block take its rows in turn, and the block's share
// of a gate's gradient is joined whenever a gate's rows end.
//
// Bound by latency, that of the reductions above all: one block of 512 threads on an SM (its
// registers hold the sums) issues 2.2 of 4 instructions a cycle.  8192×4096 bf16 112 us
// (3.6 TB/s), fp32 stream 132 us (4.6); 1021×5119 fp16, unaligned, a gate per row, 63 us;
// 2048×8192 and 2048×16000 bf16 91 and 192 us.
//
// MULTI: the `split` blocks of a cluster share their rows, `part` columns each (the last
// one the rest), and add up their sums: for rows of more columns than a block's threads
// have in registers (8 each; with 16 a thread's sums did not fit, and 2048 rows of 8192
// columns took 107 us).
template <typename TX, typename TR, bool VEC, bool MULTI>
__global__ void __launch_bounds__(kNormThreads)
    tg_norm_grad_rows(const NormGradParams q, int threads, int stages, int stage_bytes, int split,
                      int part, uint64_t limit_ns, unsigned int* timeouts, int inject) {
    constexpr int CH = 1;
    extern __shared__ __align__(16) unsigned char norm_stage[];
    __shared__ __align__(16) float red[8 * 160];
    const NormParams& p = q.n;
    NormGroup g = norm_group(threads, red, 8 * 160);
    const int rank = MULTI ? blockIdx.x % split : 0;
    const int64_t block = MULTI ? blockIdx.x / split : blockIdx.x;
    const int64_t blocks = MULTI ? gridDim.x / split : gridDim.x;
    const int c0 = MULTI ? rank * part : 0;  // first column here
    int cols = static_cast<int>(p.cols) - c0;
    if (MULTI && cols > part) cols = part;
    const NormCols<CH, VEC> c{g.tid, g.threads, cols};
    NormPeers<MULTI> peers(rank, split, limit_ns, timeouts, inject == 1 && blockIdx.x == 1);
    const float* const wpost = p.wpost != nullptr ? p.wpost + c0 : nullptr;
    const float* const wpre = p.wpre != nullptr ? p.wpre + c0 : nullptr;
    const float inv = 1.0f / static_cast<float>(p.cols);
    const int rows = static_cast<int>(p.rows), per = static_cast<int>(p.rows_per_gate);
    int row0, row1, stride = 1;
    if (q.whole_gates) {
        const int64_t groups = blocks * g.count;
        const int64_t i = block * g.count + g.index;
        row0 = static_cast<int>(norm_first_row(q.gates, groups, i)) * per;
        row1 = static_cast<int>(norm_first_row(q.gates, groups, i + 1)) * per;
    } else {
        row0 = static_cast<int>(norm_first_row(rows, blocks, block)) + g.index;
        row1 = static_cast<int>(norm_first_row(rows, blocks, block + 1));
        stride = g.count;
    }
    unsigned char* mine = norm_stage + g.index * stages * stage_bytes;
    unsigned char* behind = norm_stage + g.count * stages * stage_bytes;  // the ring
    const int bx = norm_stage_bytes<TX, CH, VEC>(threads, MULTI ? part : p.cols);
    const int br = norm_stage_bytes<TR, CH, VEC>(threads, MULTI ? part : p.cols);
    const bool one_gate = per == rows;
    NormInput<TX, CH, VEC> in_x, in_dh, in_g;
    NormInput<TR, CH, VEC> in_r, in_dy;
    in_x.start(c, norm_at<TX>(p.x, c0), p.ldx, mine, stages, stage_bytes);
    in_dh.start(c, norm_at<TX>(q.dh, c0), q.lddh, mine + bx, stages, stage_bytes);
    in_r.start(c, norm_at<TR>(p.r, c0), p.ldr, mine + 2 * bx, stages, stage_bytes);
    in_dy.start(c, norm_at<TR>(q.dy, c0), q.lddy, mine + 2 * bx + br, stages, stage_bytes);
    if (one_gate)
        in_g.start(c, norm_at<TX>(p.gate, c0), p.ldg, behind + g.index * bx, 1, 0);
    else
        in_g.start(c, norm_at<TX>(p.gate, c0), p.ldg, mine + 2 * (bx + br), stages, stage_bytes);
    int to_fetch = row0;
    auto fetch = [&](int slot) {
        if (to_fetch < row1) {
            const int at = slot * stage_bytes;
            in_x.fetch(c, at, to_fetch);
            in_dh.fetch(c, at, to_fetch);
            in_r.fetch(c, at, to_fetch);
            in_dy.fetch(c, at, to_fetch);
            if (!one_gate) in_g.fetch(c, at, norm_gate_row(to_fetch, per));
        }
        to_fetch += stride;
        norm_commit();
    };
    op_release_next();
    op_wait_previous();
    if (one_gate) in_g.fetch(c, 0, 0);
    for (int s = 0; s < stages - 1; ++s) fetch(s);

    F2 wo[4], wp[4];
    norm_weight<CH, VEC>(wpost, c, 0, wo);
    norm_weight<CH, VEC>(wpre, c, 0, wp);
    F2 sum_post[CH][4], sum_pre[CH][4], sum_gate[CH][4];
#pragma unroll
    for (int ch = 0; ch < CH; ++ch)
#pragma unroll
        for (int i = 0; i < 4; ++i) sum_post[ch][i] = sum_pre[ch][i] = sum_gate[ch][i] = 0;
    const F2 scale2 = f2(p.scale, p.scale);
    // Σ over the block's groups of a thread's columns, times factor, to `share`
    F2* all = reinterpret_cast<F2*>(behind + g.count * bx);
    auto join = [&](F2 (&v)[CH][4], float* share, float factor) {
        if (g.count > 1) {
            __syncthreads();
            if (g.index > 0)
#pragma unroll
                for (int ch = 0; ch < CH; ++ch)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        all[(((g.index - 1) * CH + ch) * 4 + i) * threads + g.tid] = v[ch][i];
            __syncthreads();
        }
        if (g.index > 0) return;
#pragma unroll
        for (int ch = 0; ch < CH; ++ch) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float2 t = f2_get(v[ch][i]);
                for (int k = 1; k < g.count; ++k) {
                    const float2 u = f2_get(all[(((k - 1) * CH + ch) * 4 + i) * threads + g.tid]);
                    t.x += u.x;
                    t.y += u.y;
                }
                v[ch][i] = f2(t.x * factor, t.y * factor);
            }
            c.store(share, ch, v[ch]);
        }
    };

    int slot = 0, row = row0;
    // a block's rows, or one gate's of them after another's
    for (int first = q.whole_gates ? row0 : row0 - g.index; first < row1;) {
        const int gate_no = q.ws_gate != nullptr ? first / per : 0;
        int end = row1;
        if (q.ws_gate != nullptr && row1 - first > per - (first - gate_no * per))
            end = (gate_no + 1) * per;
        for (; row < end; row += stride) {
            norm_wait(stages);
            if (VEC)
                __syncwarp();
            else
                g.sync();
            fetch(slot == 0 ? stages - 1 : slot - 1);
            const int at = slot * stage_bytes;
            const int gate_at = one_gate ? 0 : at;
            const uint32_t gate_row = norm_gate_row(row, per);

            F2 x[CH][4];
            float rx = 1.0f;
#pragma unroll
            for (int ch = 0; ch < CH; ++ch) in_x.get(c, at, row, ch, x[ch]);
            if (p.wpost != nullptr) {
                F2 a = 0;
#pragma unroll
                for (int ch = 0; ch < CH; ++ch)
#pragma unroll
                    for (int i = 0; i < 4; ++i) a = f2_fma(x[ch][i], x[ch][i], a);
                float v[1] = {g.sum(f2_sum(a))};
                peers.add(v);
                rx = rsqrtf(v[0] * inv + p.eps);
            }
            const F2 rx2 = f2(rx, rx);
#pragma unroll
            for (int ch = 0; ch < CH; ++ch)  // m from here on
#pragma unroll
                for (int i = 0; i < 4; ++i) x[ch][i] = f2_mul(x[ch][i], rx2);
            F2 y[4], dy[4], dh[4], gt[4];
            // a chunk's inputs, and y
            auto chunk = [&](int ch) {
                in_g.get(c, gate_at, gate_row, ch, gt, 1.0f);
                in_r.get(c, at, row, ch, y);
                in_dy.get(c, at, row, ch, dy);
                in_dh.get(c, at, row, ch, dh);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    y[i] = f2_fma(scale2, f2_mul(f2_mul(x[ch][i], wo[i]), gt[i]), y[i]);
            };
            float s[5];
            {
                F2 a[5] = {0, 0, 0, 0, 0};
#pragma unroll
                for (int ch = 0; ch < CH; ++ch) {
                    chunk(ch);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const F2 t = f2_mul(f2_mul(x[ch][i], wo[i]), gt[i]);
                        const F2 dn = f2_mul(dh[i], wp[i]);
                        a[0] = f2_fma(y[i], y[i], a[0]);
                        a[1] = f2_fma(dn, y[i], a[1]);
                        a[2] = f2_fma(t, dy[i], a[2]);
                        a[3] = f2_fma(t, dn, a[3]);
                        a[4] = f2_fma(t, y[i], a[4]);
                    }
                }
#pragma unroll
                for (int k = 0; k < 5; ++k) s[k] = f2_sum(a[k]);
            }
            g.sum5(s);
            peers.add(s);
            // Without dh nothing is taken of y, which need not be finite then.
            const bool has_dh = in_dh.base != nullptr;
            const float ry = has_dh ? rsqrtf(s[0] * inv + p.eps) : 0.0f;
            const float cy = has_dh ? ry * ry * s[1] * inv : 0.0f;
            const float td = has_dh ? s[2] + ry * (s[3] - cy * s[4]) : s[2];  // Σ t·dy'
            // -mean(dm·m) · rx: what dx gets of m
            const float cx = p.wpost != nullptr ? -rx * p.scale * inv * td : 0.0f;
            const float sx = rx * p.scale;
            const F2 ry2 = f2(ry, ry), cy2 = f2(-cy, -cy), cx2 = f2(cx, cx), sx2 = f2(sx, sx);
            const bool own_gate =
                q.dgate != nullptr && q.ws_gate == nullptr &&
                (row + stride >= row1 || norm_gate_row(row + stride, per) != gate_row);
            TX* out_x = static_cast<TX*>(q.dx) +
                        static_cast<uint64_t>(row) * static_cast<uint32_t>(q.lddx) + c0;
            TR* out_r = static_cast<TR*>(q.dr) +
                        static_cast<uint64_t>(row) * static_cast<uint32_t>(q.lddr) + c0;
#pragma unroll
            for (int ch = 0; ch < CH; ++ch) {
                F2 dx[4];
                if (has_dh)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        sum_pre[ch][i] = f2_fma(dh[i], f2_mul(y[i], ry2), sum_pre[ch][i]);
                        dy[i] = f2_fma(ry2, f2_fma(cy2, y[i], f2_mul(dh[i], wp[i])), dy[i]);
                    }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const F2 m = x[ch][i];
                    sum_gate[ch][i] = f2_fma(dy[i], f2_mul(m, wo[i]), sum_gate[ch][i]);
                    const F2 dg = f2_mul(dy[i], gt[i]);
                    sum_post[ch][i] = f2_fma(dg, m, sum_post[ch][i]);
                    dx[i] = f2_fma(f2_mul(dg, wo[i]), sx2, f2_mul(cx2, m));
                }
                if (q.dx != nullptr) c.store(out_x, ch, dx);
                if (q.dr != nullptr) c.store(out_r, ch, dy);
                if (own_gate) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) dx[i] = f2_mul(sum_gate[ch][i], scale2);
                    c.store(static_cast<TX*>(q.dgate) + gate_row * q.lddg + c0, ch, dx);
#pragma unroll
                    for (int i = 0; i < 4; ++i) sum_gate[ch][i] = 0;
                }
            }
            slot = slot + 1 == stages ? 0 : slot + 1;
        }
        if (q.ws_gate != nullptr) {
            join(sum_gate, q.ws_gate + (block + gate_no) * p.cols + c0, p.scale);
#pragma unroll
            for (int ch = 0; ch < CH; ++ch)
#pragma unroll
                for (int k = 0; k < 4; ++k) sum_gate[ch][k] = 0;
        }
        first = end;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (q.ws_post != nullptr) join(sum_post, q.ws_post + block * p.cols + c0, p.scale);
    if (q.ws_pre != nullptr) join(sum_pre, q.ws_pre + block * p.cols + c0, 1.0f);
    peers.end();
}

// ------------------------------------------------------------------ any width
//
// What the rings do not hold: a forward row of more than 16384 columns, or of fp32 values
// that do not fit twice; strides of 2^32 elements; 2^31 rows.  Values are read again for
// each pass, from L2 (2048×16000 bf16, gradient: 1.8 ms, 192 us by the rings).

// Row by row, the unrounded y of the row in shared memory.
template <typename TX, typename TR>
__global__ void __launch_bounds__(256) tg_norm_residual_simple(const NormParams p) {
    extern __shared__ float norm_buf[];
    __shared__ float red[33];
    op_release_next();
    op_wait_previous();
    const float inv = 1.0f / static_cast<float>(p.cols);
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const TX* x = static_cast<const TX*>(p.x) + row * p.ldx;
        const TR* r = p.r != nullptr ? static_cast<const TR*>(p.r) + row * p.ldr : nullptr;
        const TX* g = p.gate != nullptr
                          ? static_cast<const TX*>(p.gate) + row / p.rows_per_gate * p.ldg
                          : nullptr;
        float rx = 1.0f;
        if (p.wpost != nullptr) {
            float s = 0.0f;
            for (int64_t c = threadIdx.x; c < p.cols; c += blockDim.x) {
                const float v = op_to_float(x[c]);
                s += v * v;
            }
            rx = rsqrtf(norm_block_sum(s, red) * inv + p.eps);
        }
        float s = 0.0f;
        for (int64_t c = threadIdx.x; c < p.cols; c += blockDim.x) {
            float o = op_to_float(x[c]);
            if (p.wpost != nullptr) o = o * rx * p.wpost[c];
            if (g != nullptr) o *= op_to_float(g[c]);
            const float y = (r != nullptr ? op_to_float(r[c]) : 0.0f) + p.scale * o;
            if (p.y != nullptr) (static_cast<TR*>(p.y) + row * p.ldy)[c] = op_round<TR>(y);
            norm_buf[c] = y;
            s += y * y;
        }
        if (p.wpre == nullptr) continue;
        const float ry = rsqrtf(norm_block_sum(s, red) * inv + p.eps);
        for (int64_t c = threadIdx.x; c < p.cols; c += blockDim.x)
            (static_cast<TX*>(p.h) + row * p.ldh)[c] = op_round<TX>(norm_buf[c] * ry * p.wpre[c]);
    }
}

// The gradient, row by row; a block has consecutive rows and adds its share
// of the column sums to its rows of the workspace.
template <typename TX, typename TR>
__global__ void __launch_bounds__(256) tg_norm_grad_simple(const NormGradParams q) {
    extern __shared__ float norm_buf[];
    __shared__ float red[33];
    op_release_next();
    op_wait_previous();
    const NormParams& p = q.n;
    const float inv = 1.0f / static_cast<float>(p.cols);
    int64_t row0, row1;
    if (q.whole_gates) {
        row0 = norm_first_row(q.gates, gridDim.x, blockIdx.x) * p.rows_per_gate;
        row1 = norm_first_row(q.gates, gridDim.x, blockIdx.x + 1) * p.rows_per_gate;
    } else {
        row0 = norm_first_row(p.rows, gridDim.x, blockIdx.x);
        row1 = norm_first_row(p.rows, gridDim.x, blockIdx.x + 1);
    }
    float* wpost = q.ws_post != nullptr ? q.ws_post + blockIdx.x * p.cols : nullptr;
    float* wpre = q.ws_pre != nullptr ? q.ws_pre + blockIdx.x * p.cols : nullptr;
    for (int64_t row = row0; row < row1; ++row) {
        const TX* x = static_cast<const TX*>(p.x) + row * p.ldx;
        const TR* r = p.r != nullptr ? static_cast<const TR*>(p.r) + row * p.ldr : nullptr;
        const int64_t gi = p.gate != nullptr ? row / p.rows_per_gate : 0;
        const TX* g = p.gate != nullptr ? static_cast<const TX*>(p.gate) + gi * p.ldg : nullptr;
        const TR* dy = q.dy != nullptr ? static_cast<const TR*>(q.dy) + row * q.lddy : nullptr;
        const TX* dh = q.dh != nullptr ? static_cast<const TX*>(q.dh) + row * q.lddh : nullptr;
        float rx = 1.0f, ry = 0.0f, mean = 0.0f;
        if (p.wpost != nullptr) {
            float s = 0.0f;
            for (int64_t c = threadIdx.x; c < p.cols; c += blockDim.x) {
                const float v = op_to_float(x[c]);
                s += v * v;
            }
            rx = rsqrtf(norm_block_sum(s, red) * inv + p.eps);
        }
        if (dh != nullptr) {
            float s = 0.0f, t = 0.0f;
            for (int64_t c = threadIdx.x; c < p.cols; c += blockDim.x) {
                float o = op_to_float(x[c]);
                if (p.wpost != nullptr) o = o * rx * p.wpost[c];
                if (g != nullptr) o *= op_to_float(g[c]);
                const float y = (r != nullptr ? op_to_float(r[c]) : 0.0f) + p.scale * o;
                norm_buf[c] = y;
                s += y * y;
            }
            ry = rsqrtf(norm_block_sum(s, red) * inv + p.eps);
            for (int64_t c = threadIdx.x; c < p.cols; c += blockDim.x)
                t += op_to_float(dh[c]) * p.wpre[c] * norm_buf[c] * ry;
            mean = norm_block_sum(t, red) * inv;
        }
        // first row of this block's share of its gate, and the last
        const bool first = row == row0 || row % p.rows_per_gate == 0;
        const bool last = row + 1 == row1 || (row + 1) % p.rows_per_gate == 0;
        float* wgate = nullptr;
        if (q.ws_gate != nullptr)
            wgate = q.ws_gate + (q.whole_gates ? int64_t{blockIdx.x} : blockIdx.x + gi) * p.cols;
        float t = 0.0f;
        for (int64_t c = threadIdx.x; c < p.cols; c += blockDim.x) {
            float d = dy != nullptr ? op_to_float(dy[c]) : 0.0f;
            if (dh != nullptr) {
                const float v = op_to_float(dh[c]), n = norm_buf[c] * ry;
                if (wpre != nullptr) wpre[c] = (row == row0 ? 0.0f : wpre[c]) + v * n;
                d += ry * (v * p.wpre[c] - n * mean);
            }
            if (q.dr != nullptr) (static_cast<TR*>(q.dr) + row * q.lddr)[c] = op_round<TR>(d);
            d *= p.scale;
            const float xv = op_to_float(x[c]), m = xv * rx;
            if (g != nullptr) {
                const float o = p.wpost != nullptr ? m * p.wpost[c] : xv;
                if (q.dgate != nullptr) {
                    float a = d * o;
                    if (wgate != nullptr) {
                        a += first ? 0.0f : wgate[c];
                        wgate[c] = a;
                    }
                    if (last && (q.whole_gates || wgate == nullptr))
                        (static_cast<TX*>(q.dgate) + gi * q.lddg)[c] = op_round<TX>(a);
                }
                d *= op_to_float(g[c]);
            }
            if (p.wpost != nullptr) {
                if (wpost != nullptr) wpost[c] = (row == row0 ? 0.0f : wpost[c]) + d * m;
                d *= p.wpost[c];
                t += d * m;
            }
            norm_buf[c] = d;
        }
        if (p.wpost != nullptr) mean = norm_block_sum(t, red) * inv;
        if (q.dx != nullptr)
            for (int64_t c = threadIdx.x; c < p.cols; c += blockDim.x) {
                float d = norm_buf[c];
                if (p.wpost != nullptr) d = rx * (d - op_to_float(x[c]) * rx * mean);
                (static_cast<TX*>(q.dx) + row * q.lddx)[c] = op_round<TX>(d);
            }
    }
}

// The block that has row `row` of `rows` shared among `blocks`.
__device__ __forceinline__ int64_t norm_block_of(int64_t rows, int64_t blocks, int64_t row) {
    const uint32_t each = static_cast<uint32_t>(rows) / static_cast<uint32_t>(blocks);
    const uint32_t more = static_cast<uint32_t>(rows) - each * static_cast<uint32_t>(blocks);
    const uint32_t r = static_cast<uint32_t>(row);  // the first `more` blocks have one row more
    return r < more * (each + 1) ? r / (each + 1) : more + (r - more * (each + 1)) / each;
}

// The column sums of the blocks' shares, in the order of the blocks:
// blockIdx.y 0 and 1: dwpost and dwpre; 2 + i: gate i.  32 columns per block, 16
// warps with every 16th share each, 8 of them under way at a time.
template <typename TX>
__global__ void __launch_bounds__(512)
    tg_norm_grad_sum(const NormGradParams q, int64_t blocks, int64_t jobs) {
    __shared__ float part[16][33];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    op_release_next();
    op_wait_previous();
    const int64_t c = int64_t{blockIdx.x} * 32 + lane;
    for (int64_t job = blockIdx.y; job < jobs; job += gridDim.y) {
        const float* src = job == 0 ? q.ws_post : job == 1 ? q.ws_pre : q.ws_gate;
        if (src == nullptr) continue;
        int64_t lo = 0, hi = blocks;
        if (job >= 2) {  // gate i: slots block + i of the blocks that have its rows
            const int64_t i = job - 2, per = q.n.rows_per_gate;
            lo = norm_block_of(q.n.rows, blocks, i * per) + i;
            hi = norm_block_of(q.n.rows, blocks, (i + 1) * per - 1) + i + 1;
        }
        float s = 0.0f;
        if (c < q.n.cols) {
            for (int64_t k = lo + w; k < hi; k += 128) {
                float v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[i] = k + 16 * i < hi ? src[(k + 16 * i) * q.n.cols + c] : 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) s += v[i];
            }
        }
        part[w][lane] = s;
        __syncthreads();
        if (w == 0 && c < q.n.cols) {
#pragma unroll
            for (int k = 1; k < 16; ++k) s += part[k][lane];
            if (job == 0)
                q.dwpost[c] = s;
            else if (job == 1)
                q.dwpre[c] = s;
            else
                (static_cast<TX*>(q.dgate) + (job - 2) * q.lddg)[c] = op_round<TX>(s);
        }
        __syncthreads();
    }
}

}  // namespace tg
