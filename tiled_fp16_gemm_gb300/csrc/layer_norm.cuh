// Layer norm with the residual sum before it, its rows as 8-bit codes, and its gradient.
//
//   v = x + r  (the residual stream; y = v)     mu = mean_c v
//   s = 1 / sqrt(mean_c (v - mu)² + eps)        n = (v - mu) · s        h = n · w + b
//
// Codes of a row z (of h, or of x itself):
//   scale = max_c |z| / 127,   code = z / scale to the nearest whole number, ties to even.
//
// Gradient, with dy and dh given (means over the row's columns):
//   dn = dh · w        dv = dy + s (dn - mean(dn) - n · mean(dn n))        dx = dr = dv
//   dw = Σ_rows dh ⊙ n        db = Σ_rows dh
//
// Every value is held in fp32 (the mean too: the squares are taken of v - mu, so that a mean
// far from zero costs no digits); outputs are rounded once, when they are stored, and h comes
// from the unrounded v.
#pragma once

#include <type_traits>

#include "norm.cuh"

namespace tg {

struct LayerNormParams {
    int64_t rows, cols;
    const void* x;
    int64_t ldx;
    const void* r;
    int64_t ldr;
    const float* w;
    const float* b;
    float eps;
    // forward
    void* y;
    int64_t ldy;
    void* h;  // of x's type, or codes
    int64_t ldh;
    float* scale;  // of the codes' rows
};

struct LayerNormGradParams {
    LayerNormParams n;
    const void* dy;
    int64_t lddy;
    const void* dh;
    int64_t lddh;
    void* dx;
    int64_t lddx;
    void* dr;
    int64_t lddr;
    float* dw;
    float* db;
    // the blocks' shares of the column sums, a row per block; null where not wanted
    float* ws_w;
    float* ws_b;
};

// What a launch makes of a row: h, the codes of h, or the codes of x (no norm).
enum : int { kLnH = 0, kLnCodes = 1, kLnRaw = 2 };

// ------------------------------------------------------------------ codes

__device__ __forceinline__ F2 f2_add(F2 a, F2 b) {
    F2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

constexpr uint32_t kLnInf = 0x7f800000u;

// The scale of a row whose largest |value| has these bits.  With a NaN or an infinity among
// the values (as bits, both are the largest) no scale can stand for the row: it is NaN.
__device__ __forceinline__ float ln_scale(uint32_t largest) {
    return largest >= kLnInf ? __uint_as_float(0x7fc00000u) : __fdiv_rn(__uint_as_float(largest), 127.0f);
}
// Codes of a row with this scale: value / scale to the nearest, exactly.  The product with the
// reciprocal is off by 2^-22 of it at most, so it rounds to the right whole number or, near a
// half, to one beside it; what is left over, value - q · scale, is exact in fp32 and tells
// which.  Numbers are rounded by adding 1.5·2^23 (the conversions run at an eighth of the rate),
// which leaves the code in the low byte.
struct LnCoder {
    float scale, inv, half;
    bool plain;  // a scale whose reciprocal is an fp32 number, and codes within ±127 by themselves
    static constexpr float kRound = 12582912.0f;
    __device__ __forceinline__ explicit LnCoder(float s) {
        scale = s;
        half = 0.5f * s;
        plain = s >= 1e-30f;
        inv = __frcp_rn(s);
    }
    // Any row: zeros (or values so small that their scale is 0) and one without a scale have
    // codes 0; small scales are taken 2^100 times, and the least are so coarse that ±127 is passed.
    __device__ __noinline__ static uint32_t any(float value, float scale) {
        if (!(scale > 0.0f)) return 0;
        if (scale < 1e-30f) value *= 1.2676506e30f, scale *= 1.2676506e30f;
        float t = fmaf(value, __frcp_rn(scale), kRound);
        const float rest = fmaf(kRound - t, scale, value), twice = 2.0f * fabsf(rest);
        if (twice > scale || (twice == scale && (__float_as_uint(t) & 1) != 0)) t += rest > 0.0f ? 1.0f : -1.0f;
        return __float_as_uint(fminf(fmaxf(t, kRound - 127.0f), kRound + 127.0f));
    }
    // Eight at once; each code in the low byte.
    __device__ __forceinline__ void codes(const F2 (&v)[4], uint32_t (&code)[8]) const {
        bool again = !plain;
        if (plain) {
            const F2 inv2 = f2(inv, inv), round2 = f2(kRound, kRound), less2 = f2(-scale, -scale);
            const F2 back2 = f2(-kRound, -kRound);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const F2 t = f2_fma(v[i], inv2, round2);
                const float2 rest = f2_get(f2_fma(f2_add(t, back2), less2, v[i]));
                again = again || fabsf(rest.x) >= half || fabsf(rest.y) >= half;
                const float2 w = f2_get(t);
                code[2 * i] = __float_as_uint(w.x);
                code[2 * i + 1] = __float_as_uint(w.y);
            }
        }
        if (again) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 w = f2_get(v[i]);
                code[2 * i] = any(w.x, scale);
                code[2 * i + 1] = any(w.y, scale);
            }
        }
    }
};

// The larger of three sizes; NaN where one is.
__device__ __forceinline__ float ln_most(float a, float b, float c) {
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Largest of the block's values, for every thread.  `red`: 33 words.
__device__ __forceinline__ uint32_t ln_block_max(uint32_t v, uint32_t* red) {
    v = __reduce_max_sync(0xffffffffu, v);
    const int warps = (blockDim.x + 31) / 32;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x / 32] = v;
    __syncthreads();
    if (threadIdx.x < 32) {
        v = __reduce_max_sync(0xffffffffu, threadIdx.x < warps ? red[threadIdx.x] : 0u);
        if (threadIdx.x == 0) red[32] = v;
    }
    __syncthreads();
    v = red[32];
    __syncthreads();
    return v;
}

// ------------------------------------------------------------------ rows in registers
//
// A row's values stay in the registers of the threads that share it, 8·CH columns each
// (LnCols): one warp, or for longer rows (and few of them) a block.
//
// One barrier for the statistics, whatever the values: a warp takes the mean m_u of its own
// columns first, and its sums of d = v - m_u and of d².  From the warps' (m_u, Σd, Σd²) and counts
// n_u follow, with nothing but differences of means added up,
//   mu - m_0 = Σ_u (n_u (m_u - m_0) + Σd) / cols
//   Σ (v - mu)² = Σ_u (Σd² + 2 g_u Σd + n_u g_u²),   g_u = m_u - mu
// so neither a mean far from zero nor warps with different means cost digits.
//
// Measured, calls back to back on inputs in turn: 8192×4096 bf16 on an fp32 stream 60 us (6.7 TB/s), bf16 47 us, its codes 59 and 49 us; rows of
// x as codes 17 us; 600×16384 bf16 16.1 us; 8192×1536 19 us; unaligned, 1021×5119 13 us, 4096×767 10 us;
// one row of 4096 2.1 us.  Bound by memory on the fp32 stream; else by the way of a row from its loads to
// its stores, with five rows of 4096 on an SM (96 registers).  The weights' reads, from L1, are some 4 us
// of 60.  A warp or block has one row and is done: a loop over rows kept weights and addresses in
// registers that the row needs (8192×1536 22.6 us, rows of x as codes 21).  Registers hold a row in all
// classes but runs of eight and unaligned runs of four with 640 or 1024 threads, which spill 12 to 20 bytes.
// Tried: the next rows fetched ahead by cp.async (2048×8192 29 us instead of 33, 2048×16384 88
// instead of 57) or to L2 (slower everywhere), a warp per row of 4096 (spills, 83 us), a thread's
// columns a block apart (addresses in registers, 80 us), runs of 4 or 2 neighbours instead of 8 (bf16
// 57 and 63 us).

// One over the deviation, from Σ (v - mean)².
__device__ __forceinline__ float ln_scale_of(float squares, float inv, float eps) {
    const float s = rsqrtf(fmaxf(squares, 0.0f) * inv + eps);
    return squares == squares ? s : squares;  // (fmaxf turns a NaN into 0)
}

__device__ __forceinline__ float ln_warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Two 16-bit values of a word.
template <typename T>
__device__ __forceinline__ F2 ln_pair(uint32_t u) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        return f2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    } else {
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&u));
        return f2(v.x, v.y);
    }
}
// 8 values of a row that are read once.
template <typename T>
__device__ __forceinline__ void ln_take(const T* src, F2 (&v)[4]) {
    if constexpr (sizeof(T) == 4) {
        float a, b, d, e, f, g, h, i;
        asm volatile("ld.global.L1::no_allocate.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=f"(a), "=f"(b), "=f"(d), "=f"(e), "=f"(f), "=f"(g), "=f"(h), "=f"(i)
                     : "l"(src));
        v[0] = f2(a, b), v[1] = f2(d, e), v[2] = f2(f, g), v[3] = f2(h, i);
    } else {
        uint4 u;
        asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                     : "l"(src));
        v[0] = ln_pair<T>(u.x), v[1] = ln_pair<T>(u.y), v[2] = ln_pair<T>(u.z), v[3] = ln_pair<T>(u.w);
    }
}
// 8·CH·32 consecutive columns of a row for each of its warps, so that a thread's lie at fixed
// distances.  VEC: a thread has CH runs of 8 neighbours (every row on 8 elements, cols a multiple
// of 8); else every 32nd column.
//
// ALL: the warp has all of its columns, and nothing is asked of single ones.  Then the loads of
// a row leave one after another (8192×4096 bf16 48 us, 52 with each asked for; 600×16384 17.7 and
// 20.6), and unaligned rows do not spend as much time on the questions as on their values.
template <int CH, bool VEC>
struct LnCols {
    int first, cols;  // this thread's first column
    bool all;
    __device__ __forceinline__ LnCols(int cols, int warp, int lane)
        : first(warp * 256 * CH + (VEC ? 8 : 1) * lane), cols(cols), all((warp + 1) * 256 * CH <= cols) {}
    // f(ALL): a branch around all loads of a row at once, for the results of those inside a branch
    // are waited for at its end
    template <typename F>
    __device__ __forceinline__ void either(F f) const {
        if (all)
            f(std::true_type{});
        else
            f(std::false_type{});
    }
    __device__ __forceinline__ static constexpr int at(int ch, int i) { return VEC ? 256 * ch + i : 32 * (8 * ch + i); }
    template <bool ALL = false>
    __device__ __forceinline__ bool has(int ch, int i) const {
        return ALL || first < cols - at(ch, VEC ? 0 : i);
    }
    // `row` is at this thread's first column, here and below
    template <bool ALL, typename T>
    __device__ __forceinline__ void load(const T* row, int ch, F2 (&v)[4]) const {
        if constexpr (VEC) {
            if (has<ALL>(ch, 0)) {
                ln_take<T>(row + at(ch, 0), v);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = 0;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = f2(has<ALL>(ch, 2 * i) ? op_to_float(row[at(ch, 2 * i)]) : 0.0f,
                          has<ALL>(ch, 2 * i + 1) ? op_to_float(row[at(ch, 2 * i + 1)]) : 0.0f);
        }
    }
    // of a weight, which other rows read too; `none` where there is no weight
    template <bool ALL>
    __device__ __forceinline__ void weight(const float* row, int ch, F2 (&v)[4], float none) const {
        if (row == nullptr) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = f2(none, none);
        } else if constexpr (VEC) {
            if (has<ALL>(ch, 0)) norm_take<float>(row + at(ch, 0), v);
        } else {
            load<ALL>(row, ch, v);
        }
    }
    template <bool ALL = false, typename T>
    __device__ __forceinline__ void store(T* row, int ch, const F2 (&v)[4]) const {
        if constexpr (VEC) {
            if (!has<ALL>(ch, 0)) return;
            T* p = row + at(ch, 0);
            if constexpr (sizeof(T) == 4) {
                const float2 a = f2_get(v[0]), b = f2_get(v[1]), d = f2_get(v[2]), e = f2_get(v[3]);
                asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(a.x),
                             "f"(a.y), "f"(b.x), "f"(b.y), "f"(d.x), "f"(d.y), "f"(e.x), "f"(e.y)
                             : "memory");
            } else {
                *reinterpret_cast<uint4*>(p) =
                    make_uint4(f2_pack<T>(v[0]), f2_pack<T>(v[1]), f2_pack<T>(v[2]), f2_pack<T>(v[3]));
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = f2_get(v[i]);
                if (has<ALL>(ch, 2 * i)) row[at(ch, 2 * i)] = op_round<T>(f.x);
                if (has<ALL>(ch, 2 * i + 1)) row[at(ch, 2 * i + 1)] = op_round<T>(f.y);
            }
        }
    }
    // v - m, and 0 where there is no column
    template <bool ALL = false>
    __device__ __forceinline__ void less(int ch, float m, F2 (&v)[4]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = f2_add(v[i], f2(has<ALL>(ch, 2 * i) ? -m : 0.0f, has<ALL>(ch, 2 * i + 1) ? -m : 0.0f));
    }
};

// `threads`: of a row, 32 (a block has a row for each warp) or all of the block.  SM: of an SM, what
// registers are for.
template <typename TX, typename TR, int CH, bool VEC, int MODE, int SM>
__global__ void __launch_bounds__(SM, 1)
    tg_layer_norm_rows(const LayerNormParams p, int threads) {
    __shared__ float stat[3][32];  // of the warps: mean, Σd, Σd²
    __shared__ uint32_t most[32];
    const int lane = threadIdx.x & 31, cols = static_cast<int>(p.cols);
    const bool alone = threads == 32;
    const int warp = alone ? 0 : threadIdx.x >> 5, warps = threads >> 5;
    const int group = alone ? threadIdx.x >> 5 : 0, groups = alone ? blockDim.x >> 5 : 1;
    const LnCols<CH, VEC> c(cols, warp, lane);
    const float inv = 1.0f / static_cast<float>(cols);
    // lane u: columns of warp u
    const float count = lane < warps ? static_cast<float>(min(cols - 256 * CH * lane, 256 * CH)) : 0.0f;
    const float mine = __shfl_sync(0xffffffffu, count, warp);
    const float mine_inv = mine > 0.0f ? 1.0f / mine : 0.0f;
    op_release_next();
    op_wait_previous();
    const int64_t row = int64_t{blockIdx.x} * groups + group;
    if (row >= p.rows) return;
    // The weights come with the row where the SMs hold all rows at once (64×8192 3.0 us, 3.25 without;
    // 2048×512 3.0, 3.3); else rows on an SM take turns, and registers count for more.
    constexpr bool kEarly = MODE != kLnRaw && SM == 512 && CH <= 2;
    auto here = [&](const float* all) { return all != nullptr ? all + c.first : nullptr; };
    F2 v[CH][4], w_row[kEarly ? CH : 1][4], b_row[kEarly ? CH : 1][4];
    c.either([&](auto whole) {
        constexpr bool ALL = decltype(whole)::value;
        const TX* x = static_cast<const TX*>(p.x) + row * p.ldx + c.first;
#pragma unroll
        for (int ch = 0; ch < CH; ++ch) c.template load<ALL>(x, ch, v[ch]);
        if constexpr (kEarly) {
#pragma unroll
            for (int ch = 0; ch < CH; ++ch) {
                c.template weight<ALL>(here(p.w), ch, w_row[ch], 1.0f);
                c.template weight<ALL>(here(p.b), ch, b_row[ch], 0.0f);
            }
        }
        if (MODE == kLnRaw || p.r == nullptr) return;
        const TR* rr = static_cast<const TR*>(p.r) + row * p.ldr + c.first;
        F2 r[CH][4];
#pragma unroll
        for (int ch = 0; ch < CH; ++ch) c.template load<ALL>(rr, ch, r[ch]);
#pragma unroll
        for (int ch = 0; ch < CH; ++ch)
#pragma unroll
            for (int i = 0; i < 4; ++i) v[ch][i] = f2_add(v[ch][i], r[ch][i]);
        if (p.y == nullptr) return;
        TR* y = static_cast<TR*>(p.y) + row * p.ldy + c.first;
#pragma unroll
        for (int ch = 0; ch < CH; ++ch) c.template store<ALL>(y, ch, v[ch]);
    });
    if (MODE != kLnRaw) {
        if (MODE == kLnH && p.h == nullptr) return;
        F2 a = 0;
#pragma unroll
        for (int ch = 0; ch < CH; ++ch)
#pragma unroll
            for (int i = 0; i < 4; ++i) a = f2_add(a, v[ch][i]);
        const float m = ln_warp_sum(f2_sum(a)) * mine_inv;
        F2 b = 0;
        a = 0;
        c.either([&](auto whole) {
#pragma unroll
            for (int ch = 0; ch < CH; ++ch) c.template less<decltype(whole)::value>(ch, m, v[ch]);
        });
#pragma unroll
        for (int ch = 0; ch < CH; ++ch) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a = f2_add(a, v[ch][i]);
                b = f2_fma(v[ch][i], v[ch][i], b);
            }
        }
        // both at once: the lower lanes take Σd, the upper ones Σd²
        const float a1 = f2_sum(a), b1 = f2_sum(b);
        float w = (lane < 16 ? a1 : b1) + __shfl_xor_sync(0xffffffffu, lane < 16 ? b1 : a1, 16);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
        float off, var;  // mu - m, Σ (v - mu)²
        if (alone) {
            const float s1 = __shfl_sync(0xffffffffu, w, 0);
            off = s1 * inv;
            var = __shfl_sync(0xffffffffu, w, 16) - off * s1;
        } else {
            if (lane == 0) {
                stat[0][warp] = m;
                stat[1][warp] = w;
            }
            if (lane == 16) stat[2][warp] = w;
            __syncthreads();
            const bool has = lane < warps;
            const float m0 = stat[0][0];
            const float mu = has ? stat[0][lane] - m0 : 0.0f;
            const float s1 = has ? stat[1][lane] : 0.0f;
            const float shift = ln_warp_sum(fmaf(count, mu, s1)) * inv;  // mu - m_0
            const float gu = mu - shift;
            var = ln_warp_sum(has ? fmaf(gu, fmaf(count, gu, 2.0f * s1), stat[2][lane]) : 0.0f);
            off = shift - (m - m0);
        }
        const float s = ln_scale_of(var, inv, p.eps);
        const F2 s2 = f2(s, s), o2 = f2(-off, -off);
        TX* h = static_cast<TX*>(p.h) + row * p.ldh + c.first;
        c.either([&](auto whole) {
            constexpr bool ALL = decltype(whole)::value;
#pragma unroll
            for (int ch = 0; ch < CH; ++ch) {
                const int at = kEarly ? ch : 0;
                if constexpr (!kEarly) {
                    c.template weight<ALL>(here(p.w), ch, w_row[0], 1.0f);
                    c.template weight<ALL>(here(p.b), ch, b_row[0], 0.0f);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    v[ch][i] = f2_fma(f2_mul(f2_add(v[ch][i], o2), s2), w_row[at][i], b_row[at][i]);
                if (MODE == kLnH) c.template store<ALL>(h, ch, v[ch]);
            }
        });
    }
    if constexpr (MODE != kLnH) {
        float size = 0.0f;
        c.either([&](auto whole) {
            constexpr bool ALL = decltype(whole)::value;
#pragma unroll
            for (int ch = 0; ch < CH; ++ch)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = f2_get(v[ch][i]);
                    size = ln_most(size, c.template has<ALL>(ch, 2 * i) ? f.x : 0.0f,
                                   c.template has<ALL>(ch, 2 * i + 1) ? f.y : 0.0f);
                }
        });
        uint32_t u = __reduce_max_sync(0xffffffffu, __float_as_uint(size) & 0x7fffffffu);
        if (!alone) {
            if (lane == 0) most[warp] = u;
            __syncthreads();
            u = __reduce_max_sync(0xffffffffu, lane < warps ? most[lane] : 0u);
        }
        const float scale = ln_scale(u);
        if (lane == 0 && warp == 0) p.scale[row] = scale;
        const LnCoder coder(scale);
        int8_t* to = static_cast<int8_t*>(p.h) + row * p.ldh + c.first;
#pragma unroll
        for (int ch = 0; ch < CH; ++ch) {
            uint32_t code[8];
            coder.codes(v[ch], code);
            if constexpr (VEC) {
                if (c.has(ch, 0)) {
                    uint2 w;
                    w.x = __byte_perm(__byte_perm(code[0], code[1], 0x0040),
                                      __byte_perm(code[2], code[3], 0x0040), 0x5410);
                    w.y = __byte_perm(__byte_perm(code[4], code[5], 0x0040),
                                      __byte_perm(code[6], code[7], 0x0040), 0x5410);
                    *reinterpret_cast<uint2*>(to + c.at(ch, 0)) = w;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (c.has(ch, i)) to[c.at(ch, i)] = static_cast<int8_t>(code[i]);
            }
        }
    }
}

// ------------------------------------------------------------------ the gradient of rows in a ring
//
// A thread has 16 columns of every row that its warps take, and keeps their sums (of dw and db) in
// registers, and their weights.  The rows come through a ring in shared memory, a part of it for
// each warp, by cp.async: x, r and dh are read for the row's sums, dh and dy again for the results.
// The statistics are those of tg_layer_norm_rows, with two sums more in the same exchange,
//   Σ dn   and   Σ dn (v - mu) = Σ_u (Σ dn d + g_u Σ dn).
// A block of 16 warps has as many groups of warps as rows fit beside one another; at the end it
// joins their sums and writes one share.
//
// MULTI: the `split` blocks of a cluster share their rows, `part` columns each, and exchange
// their means and sums: for rows of more columns than a block's threads have in registers.
//
// Measured, in bf16 with a residual: 8192×4096 66 us (6.1 TB/s), on an fp32 stream 107 us; 8192×1024 23
// us, 2048×8192 40 us, 600×16384 34 us; unaligned, 2050×1537 on an fp32 stream 21 us, 1021×5119 27 us;
// 256×1024 5.9 us (in fp16 without a residual 5.1).
// The column sums (a block's share, the second launch) are 2 to 5 us of each.  Aligned rows are bound
// by memory, unaligned ones by the issue of single-value accesses, rows that blocks share by their
// exchanges.  (The groups' sums joined by the first group alone, one sum after the other: 2 us more.)

constexpr int kLnGradWarps = 16;
constexpr int kLnGradCols = 512;  // of a warp
constexpr int kLnGradStages = 2;

// One input's place in the ring.  VEC: fp32 values are fetched in the order of memory (lane l the
// l-th and the l + 32-th 16 bytes of 256 columns), so that each fetch takes whole sectors, and lie
// turned so that the reads of both halves fall into all banks.  Else the 16-byte granules that
// hold the warp's columns are fetched, and single values read out of them.
template <typename T, bool VEC>
struct LnInput {
    using Cols = LnCols<2, VEC>;
    static constexpr int kPieces = sizeof(T) / 2;
    static constexpr int kBytes = kLnGradCols * static_cast<int>(sizeof(T)) + (VEC ? 0 : 16);
    const T* base;  // at the block's first column; null: absent
    int64_t ld;
    unsigned char* place;  // of this warp, in stage 0
    int first;             // column of the warp

    __device__ __forceinline__ static int piece(int n) { return kPieces == 1 ? n : n ^ (n >> 3 & 1); }
    __device__ __forceinline__ void fetch(const Cols& c, int offset, int64_t row, int lane) const {
        if (base == nullptr) return;
        const T* src = base + row * ld + first;
        const uint32_t to = op_smem(place + offset);
        if constexpr (VEC) {
#pragma unroll
            for (int ch = 0; ch < 2; ++ch)
#pragma unroll
                for (int h = 0; h < kPieces; ++h) {
                    const int n = lane + 32 * h, col = 256 * ch + n * (8 / kPieces);
                    if (first + col < c.cols) norm_copy16(to + ch * 512 * kPieces + 16 * piece(n), src + col);
                }
        } else {
            const int cols = min(c.cols - first, kLnGradCols);
            if (cols <= 0) return;
            const Granules g = granules(reinterpret_cast<uint64_t>(base),
                                        static_cast<uint64_t>((row * ld + first) * static_cast<int64_t>(sizeof(T))),
                                        cols * static_cast<int>(sizeof(T)));
            const unsigned char* at = reinterpret_cast<const unsigned char*>(src) - g.skip;
            for (int b = 16 * lane; b < g.end; b += 512) {
                const int n = g.end - b < 16 ? g.end - b : 16;
                if (b == 0 && g.outside) {
                    for (int i = g.skip; i < n; i += static_cast<int>(sizeof(T)))
                        *reinterpret_cast<T*>(place + offset + i) = *reinterpret_cast<const T*>(at + i);
                } else {
                    norm_copy16(to + b, at + b, n);
                }
            }
        }
    }
    template <bool ALL>
    __device__ __forceinline__ void get(const Cols& c, int offset, int64_t row, int ch, int lane, F2 (&v)[4]) const {
        const unsigned char* s = place + offset;
        if (base == nullptr || (VEC && !c.template has<ALL>(ch, 0))) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = 0;
        } else if constexpr (!VEC) {
            const T* t = reinterpret_cast<const T*>(
                             s + (reinterpret_cast<uintptr_t>(base + row * ld + first) & 15)) + lane;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = f2(c.template has<ALL>(ch, 2 * i) ? op_to_float(t[c.at(ch, 2 * i)]) : 0.0f,
                          c.template has<ALL>(ch, 2 * i + 1) ? op_to_float(t[c.at(ch, 2 * i + 1)]) : 0.0f);
        } else if constexpr (kPieces == 2) {
            s += ch * 1024;
            const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(s + 16 * piece(2 * lane));
            const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(s + 16 * piece(2 * lane + 1));
            v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
        } else {
            const uint4 u = *reinterpret_cast<const uint4*>(s + ch * 512 + 16 * lane);
            v[0] = ln_pair<T>(u.x), v[1] = ln_pair<T>(u.y), v[2] = ln_pair<T>(u.z), v[3] = ln_pair<T>(u.w);
        }
    }
};

// `warps`: of a group.  Shared memory: the warps' rings, and at the end the groups' sums.
template <typename TX, typename TR, bool VEC, bool MULTI>
__global__ void __launch_bounds__(32 * kLnGradWarps, 1)
    tg_layer_norm_grad_rows(const LayerNormGradParams q, int warps, int split, int part, uint64_t limit_ns,
                            unsigned int* timeouts, int inject) {
    constexpr int CH = 2;
    extern __shared__ __align__(16) unsigned char ln_ring[];
    // [turn][m, Σd, Σd², Σdn, Σdn·d][warp]: one row's are read while the next one's come
    __shared__ float red[2][5][kLnGradWarps];
    const LayerNormParams& p = q.n;
    const int lane = threadIdx.x & 31, all_warps = blockDim.x >> 5;
    const int group = (threadIdx.x >> 5) / warps, warp = (threadIdx.x >> 5) - group * warps;
    const int groups = all_warps / warps;
    const int rank = MULTI ? blockIdx.x % split : 0;
    const int64_t block = MULTI ? blockIdx.x / split : blockIdx.x;
    const int64_t blocks = MULTI ? gridDim.x / split : gridDim.x;
    const int c0 = MULTI ? rank * part : 0;  // first column here
    const int cols = MULTI ? min(static_cast<int>(p.cols) - c0, part) : static_cast<int>(p.cols);
    const LnCols<CH, VEC> c(cols, warp, lane);
    NormPeers<MULTI> peers(rank, split, limit_ns, timeouts, inject == 1 && blockIdx.x == 1);
    const float inv = 1.0f / static_cast<float>(p.cols);
    // lane u (and u + 16): columns of warp u
    const int u = lane & 15;
    const float count = u < warps ? static_cast<float>(max(min(cols - kLnGradCols * u, kLnGradCols), 0)) : 0.0f;
    const float mine = __shfl_sync(0xffffffffu, count, warp);
    const float mine_inv = mine > 0.0f ? 1.0f / mine : 0.0f;
    const float here_inv = MULTI ? 1.0f / static_cast<float>(cols) : inv;

    constexpr int bx = LnInput<TX, VEC>::kBytes, br = LnInput<TR, VEC>::kBytes, kStage = 2 * (bx + br);
    unsigned char* const place = ln_ring + (threadIdx.x >> 5) * kLnGradStages * kStage;
    const int first = warp * kLnGradCols;
    const LnInput<TX, VEC> in_x{static_cast<const TX*>(norm_at<TX>(p.x, c0)), p.ldx, place, first};
    const LnInput<TX, VEC> in_dh{static_cast<const TX*>(norm_at<TX>(q.dh, c0)), q.lddh, place + bx, first};
    const LnInput<TR, VEC> in_r{static_cast<const TR*>(norm_at<TR>(p.r, c0)), p.ldr, place + 2 * bx, first};
    const LnInput<TR, VEC> in_dy{static_cast<const TR*>(norm_at<TR>(q.dy, c0)), q.lddy, place + 2 * bx + br, first};
    const bool has_dh = in_dh.base != nullptr;
    const int64_t step = blocks * groups;
    int64_t row = block * groups + group, next = row;
    auto fetch = [&](int offset) {
        if (next < p.rows) {
            if (has_dh) {
                in_x.fetch(c, offset, next, lane);
                in_r.fetch(c, offset, next, lane);
                in_dh.fetch(c, offset, next, lane);
            }
            in_dy.fetch(c, offset, next, lane);
        }
        next += step;
        norm_commit();
    };
    op_release_next();
    op_wait_previous();
    for (int i = 0; i < kLnGradStages; ++i) fetch(i * kStage);
    F2 w[CH][4], sum_w[CH][4], sum_b[CH][4];
#pragma unroll
    for (int ch = 0; ch < CH; ++ch) {
        c.template weight<false>(p.w != nullptr ? p.w + c0 + c.first : nullptr, ch, w[ch], 1.0f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (!c.has(ch, 2 * i)) w[ch][i] = 0;
            sum_w[ch][i] = sum_b[ch][i] = 0;
        }
    }

    static_assert(kLnGradStages == 2, "a row's stage is its turn");
    c.either([&](auto whole) {  // (the barrier inside counts warps, wherever they are in the code)
        constexpr bool ALL = decltype(whole)::value;
        for (int turn = 0; row < p.rows; row += step, turn ^= 1) {
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            __syncwarp();
            const int at = turn * kStage;
            F2 v[CH][4];
            float s = 0.0f, off = 0.0f, m1 = 0.0f, m2 = 0.0f;  // off: mu - m
            if (has_dh) {
                F2 a = 0;
#pragma unroll
                for (int ch = 0; ch < CH; ++ch) {
                    in_x.template get<ALL>(c, at, row, ch, lane, v[ch]);
                    if (in_r.base != nullptr) {
                        F2 r[4];
                        in_r.template get<ALL>(c, at, row, ch, lane, r);
#pragma unroll
                        for (int i = 0; i < 4; ++i) v[ch][i] = f2_add(v[ch][i], r[i]);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) a = f2_add(a, v[ch][i]);
                }
                const float m = ln_warp_sum(f2_sum(a)) * mine_inv;
                F2 b[4] = {0, 0, 0, 0};
#pragma unroll
                for (int ch = 0; ch < CH; ++ch) {
                    F2 dh[4];
                    in_dh.template get<ALL>(c, at, row, ch, lane, dh);
                    c.template less<ALL>(ch, m, v[ch]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const F2 dn = f2_mul(dh[i], w[ch][i]);
                        b[0] = f2_add(b[0], v[ch][i]);
                        b[1] = f2_fma(v[ch][i], v[ch][i], b[1]);
                        b[2] = f2_add(b[2], dn);
                        b[3] = f2_fma(dn, v[ch][i], b[3]);
                    }
                }
                // Four sums at once: 8 lanes for each.
                const bool b4 = lane & 16, b3 = lane & 8;
                const float s0 = f2_sum(b[0]), s1 = f2_sum(b[1]), s2 = f2_sum(b[2]), s3 = f2_sum(b[3]);
                const float e = (b4 ? s2 : s0) + __shfl_xor_sync(0xffffffffu, b4 ? s0 : s2, 16);
                const float f = (b4 ? s3 : s1) + __shfl_xor_sync(0xffffffffu, b4 ? s1 : s3, 16);
                float t = (b3 ? f : e) + __shfl_xor_sync(0xffffffffu, b3 ? e : f, 8);  // sum lane / 8
#pragma unroll
                for (int o = 4; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
                // of the block: base and mean - base, Σ (v - mean)², Σ dn, Σ dn (v - mean)
                float base, rest, var, p1, p2;
                if (warps == 1) {
                    const float d1 = __shfl_sync(0xffffffffu, t, 0), d2 = __shfl_sync(0xffffffffu, t, 8);
                    base = m;
                    rest = d1 * here_inv;
                    var = d2 - rest * d1;
                    p1 = __shfl_sync(0xffffffffu, t, 16);
                    p2 = __shfl_sync(0xffffffffu, t, 24) - rest * p1;
                    off = rest;
                } else {
                    float* r = &red[turn][0][group * warps];
                    if ((lane & 7) == 0) r[(1 + (lane >> 3)) * kLnGradWarps + warp] = t;
                    if (lane == 0) r[warp] = m;
                    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(32 * warps) : "memory");
                    const bool has = u < warps;
                    const float m0 = r[0];
                    const float mu = has ? r[u] - m0 : 0.0f, d1 = has ? r[kLnGradWarps + u] : 0.0f;
                    const float dn = has ? r[3 * kLnGradWarps + u] : 0.0f;
                    // the lower lanes take one sum, the upper ones another
                    float z = b4 ? dn : fmaf(count, mu, d1);
#pragma unroll
                    for (int o = 8; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
                    const float shift = __shfl_sync(0xffffffffu, z, 0) * here_inv;
                    p1 = __shfl_sync(0xffffffffu, z, 16);
                    const float gu = mu - shift;
                    z = !has ? 0.0f
                        : b4 ? fmaf(gu, dn, r[4 * kLnGradWarps + u])
                             : fmaf(gu, fmaf(count, gu, 2.0f * d1), r[2 * kLnGradWarps + u]);
#pragma unroll
                    for (int o = 8; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
                    var = __shfl_sync(0xffffffffu, z, 0);
                    p2 = __shfl_sync(0xffffffffu, z, 16);
                    off = shift - (m - m0);
                    base = m0;
                    rest = shift;
                }
                if constexpr (MULTI) {
                    // (the block's mean in two parts: far from zero it loses in one what counts)
                    const float send[5] = {base, rest, var, p1, p2};
                    const float* got = peers.exchange(send);
                    const float from = got[0];
                    auto above = [&](int b) { return got[8 * b] - from + got[8 * b + 1]; };  // from
                    auto columns = [&](int b) {
                        return static_cast<float>(min(static_cast<int>(p.cols) - b * part, part));
                    };
                    float shift = 0.0f;
                    for (int b = 0; b < split; ++b) shift = fmaf(columns(b), above(b), shift);
                    shift *= inv;
                    var = p1 = p2 = 0.0f;
                    for (int b = 0; b < split; ++b) {
                        const float g = above(b) - shift;
                        var += fmaf(columns(b) * g, g, got[8 * b + 2]);
                        p1 += got[8 * b + 3];
                        p2 += fmaf(g, got[8 * b + 3], got[8 * b + 4]);
                    }
                    off += shift - (base - from + rest);
                }
                s = ln_scale_of(var, inv, p.eps);
                m1 = p1 * inv;
                m2 = p2 * inv * s;
            }
            const F2 s2 = f2(s, s), o2 = f2(-off, -off), m1n = f2(-m1, -m1), m2n = f2(-m2, -m2);
#pragma unroll
            for (int ch = 0; ch < CH; ++ch) {
                F2 d[4];
                in_dy.template get<ALL>(c, at, row, ch, lane, d);
                if (has_dh) {
                    F2 dh[4];
                    in_dh.template get<ALL>(c, at, row, ch, lane, dh);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const F2 n = f2_mul(f2_add(v[ch][i], o2), s2);
                        sum_b[ch][i] = f2_add(sum_b[ch][i], dh[i]);
                        sum_w[ch][i] = f2_fma(dh[i], n, sum_w[ch][i]);
                        d[i] = f2_fma(s2, f2_fma(n, m2n, f2_fma(dh[i], w[ch][i], m1n)), d[i]);
                    }
                }
                if (q.dx != nullptr) c.template store<ALL>(static_cast<TX*>(q.dx) + row * q.lddx + c0 + c.first, ch, d);
                if (q.dr != nullptr) c.template store<ALL>(static_cast<TR*>(q.dr) + row * q.lddr + c0 + c.first, ch, d);
            }
            __syncwarp();  // all lanes have read the stage, which is filled again
            fetch(at);
        }
    });
    asm volatile("cp.async.wait_group 0;" ::: "memory");

    // The groups' sums, in their order, to the block's share.
    float* const share_w = q.ws_w != nullptr ? q.ws_w + block * p.cols + c0 : nullptr;
    float* const share_b = q.ws_b != nullptr ? q.ws_b + block * p.cols + c0 : nullptr;
    if (groups == 1) {
#pragma unroll
        for (int ch = 0; ch < CH; ++ch) {
            if (share_w != nullptr) c.store(share_w + c.first, ch, sum_w[ch]);
            if (share_b != nullptr) c.store(share_b + c.first, ch, sum_b[ch]);
        }
    } else if (share_w != nullptr || share_b != nullptr) {
        // (4 KB of each warp, whose ring had 8)
        float* const all = reinterpret_cast<float*>(ln_ring);
        const int width = kLnGradCols * warps;
        __syncthreads();  // all have read their rings
        auto keep = [&](float* to, int ch, const F2 (&v)[4]) {
            if constexpr (VEC) {
                ulonglong2* at = reinterpret_cast<ulonglong2*>(to + c.at(ch, 0));
                at[0] = make_ulonglong2(v[0], v[1]);
                at[1] = make_ulonglong2(v[2], v[3]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = f2_get(v[i]);
                    to[c.at(ch, 2 * i)] = f.x;
                    to[c.at(ch, 2 * i + 1)] = f.y;
                }
            }
        };
#pragma unroll
        for (int ch = 0; ch < CH; ++ch) {
            keep(all + 2 * group * width + c.first, ch, sum_w[ch]);
            keep(all + (2 * group + 1) * width + c.first, ch, sum_b[ch]);
        }
        __syncthreads();
        const int threads = blockDim.x;
        for (int which = share_w != nullptr ? 0 : 1; which < (share_b != nullptr ? 2 : 1); ++which) {
            float* const share = which == 0 ? share_w : share_b;
            for (int col = threadIdx.x; col < cols; col += 4 * threads) {  // four under way at a time
                const float* at = all + which * width + col;
                float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                for (int g = 0; g < groups; ++g, at += 2 * width)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (col + k * threads < cols) sum[k] += at[k * threads];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (col + k * threads < cols) share[col + k * threads] = sum[k];
            }
        }
    }
    peers.end();
}

// ------------------------------------------------------------------ any width and stride
//
// A row per block and turn; values are read again for each pass, from L2.  The second pass takes the
// differences from the first one's mean, and with them what that lacks.

template <typename TX, typename TR, int MODE>
__global__ void __launch_bounds__(256) tg_layer_norm_simple(const LayerNormParams p) {
    __shared__ float red[33];
    op_release_next();
    op_wait_previous();
    const float inv = 1.0f / static_cast<float>(p.cols);
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const TX* x = static_cast<const TX*>(p.x) + row * p.ldx;
        const TR* r = p.r != nullptr ? static_cast<const TR*>(p.r) + row * p.ldr : nullptr;
        auto value = [&](int64_t c) {
            const float v = op_to_float(x[c]);
            return r != nullptr ? v + op_to_float(r[c]) : v;
        };
        float m = 0.0f, off = 0.0f, s = 1.0f;  // the mean is m + off
        if (MODE != kLnRaw) {
            float a = 0.0f, b = 0.0f;
            for (int64_t c = threadIdx.x; c < p.cols; c += blockDim.x) a += value(c);
            m = norm_block_sum(a, red) * inv;
            a = 0.0f;
            for (int64_t c = threadIdx.x; c < p.cols; c += blockDim.x) {
                const float d = value(c) - m;
                a += d;
                b += d * d;
            }
            a = norm_block_sum(a, red);
            off = a * inv;
            s = ln_scale_of(norm_block_sum(b, red) - off * a, inv, p.eps);
        }
        auto normed = [&](float v, int64_t c) {
            if (MODE == kLnRaw) return v;
            const float n = (v - m - off) * s;
            return fmaf(n, p.w != nullptr ? p.w[c] : 1.0f, p.b != nullptr ? p.b[c] : 0.0f);
        };
        float scale = 0.0f;
        if (MODE != kLnH) {
            uint32_t most = 0;
            for (int64_t c = threadIdx.x; c < p.cols; c += blockDim.x) {
                const uint32_t u = __float_as_uint(normed(value(c), c)) & 0x7fffffffu;
                most = u > most ? u : most;
            }
            scale = ln_scale(ln_block_max(most, reinterpret_cast<uint32_t*>(red)));
            if (threadIdx.x == 0) p.scale[row] = scale;
        }
        // (the last look at r: y may take its place)
        for (int64_t c = threadIdx.x; c < p.cols; c += blockDim.x) {
            const float v = value(c), h = normed(v, c);
            if (MODE == kLnH) {
                if (p.h != nullptr) (static_cast<TX*>(p.h) + row * p.ldh)[c] = op_round<TX>(h);
            } else {
                (static_cast<int8_t*>(p.h) + row * p.ldh)[c] = static_cast<int8_t>(LnCoder::any(h, scale));
            }
            if (p.y != nullptr) (static_cast<TR*>(p.y) + row * p.ldy)[c] = op_round<TR>(v);
        }
    }
}

// The gradient, row by row; a block has consecutive rows and adds its share of the column
// sums to its rows of the workspace.
template <typename TX, typename TR>
__global__ void __launch_bounds__(256) tg_layer_norm_grad_simple(const LayerNormGradParams q) {
    __shared__ float red[33];
    op_release_next();
    op_wait_previous();
    const LayerNormParams& p = q.n;
    const float inv = 1.0f / static_cast<float>(p.cols);
    const int64_t row0 = norm_first_row(p.rows, gridDim.x, blockIdx.x);
    const int64_t row1 = norm_first_row(p.rows, gridDim.x, blockIdx.x + 1);
    float* ww = q.ws_w != nullptr ? q.ws_w + blockIdx.x * p.cols : nullptr;
    float* wb = q.ws_b != nullptr ? q.ws_b + blockIdx.x * p.cols : nullptr;
    for (int64_t row = row0; row < row1; ++row) {
        const TX* x = static_cast<const TX*>(p.x) + row * p.ldx;
        const TR* r = p.r != nullptr ? static_cast<const TR*>(p.r) + row * p.ldr : nullptr;
        const TR* dy = q.dy != nullptr ? static_cast<const TR*>(q.dy) + row * q.lddy : nullptr;
        const TX* dh = q.dh != nullptr ? static_cast<const TX*>(q.dh) + row * q.lddh : nullptr;
        auto value = [&](int64_t c) {
            const float v = op_to_float(x[c]);
            return r != nullptr ? v + op_to_float(r[c]) : v;
        };
        auto dn_at = [&](int64_t c) {
            const float d = op_to_float(dh[c]);
            return p.w != nullptr ? d * p.w[c] : d;
        };
        float m = 0.0f, off = 0.0f, s = 0.0f, m1 = 0.0f, m2 = 0.0f;  // the mean is m + off
        if (dh != nullptr) {  // else nothing is taken of v, which need not be finite then
            float a = 0.0f, a2 = 0.0f, b = 0.0f, d = 0.0f;
            for (int64_t c = threadIdx.x; c < p.cols; c += blockDim.x) a += value(c);
            m = norm_block_sum(a, red) * inv;
            a = 0.0f;
            for (int64_t c = threadIdx.x; c < p.cols; c += blockDim.x) {
                const float u = value(c) - m, dn = dn_at(c);
                a += u;
                a2 += u * u;
                b += dn;
                d += dn * u;
            }
            a = norm_block_sum(a, red);
            off = a * inv;
            s = ln_scale_of(norm_block_sum(a2, red) - off * a, inv, p.eps);
            b = norm_block_sum(b, red);
            m1 = b * inv;
            m2 = (norm_block_sum(d, red) - off * b) * inv * s;
        }
        for (int64_t c = threadIdx.x; c < p.cols; c += blockDim.x) {
            float d = dy != nullptr ? op_to_float(dy[c]) : 0.0f;
            if (dh != nullptr) {
                const float n = (value(c) - m - off) * s;
                d += s * (dn_at(c) - m1 - n * m2);
                if (ww != nullptr) ww[c] = (row == row0 ? 0.0f : ww[c]) + op_to_float(dh[c]) * n;
                if (wb != nullptr) wb[c] = (row == row0 ? 0.0f : wb[c]) + op_to_float(dh[c]);
            }
            if (q.dx != nullptr) (static_cast<TX*>(q.dx) + row * q.lddx)[c] = op_round<TX>(d);
            if (q.dr != nullptr) (static_cast<TR*>(q.dr) + row * q.lddr)[c] = op_round<TR>(d);
        }
    }
}

// The column sums of the blocks' shares, in a fixed order: blockIdx.y 0: dw, 1: db.  32·G columns
// per block, 32 warps with every 32nd share each, 8 values of a thread under way at a time.  (16
// warps with every 16th share, and 64-bit addresses: 2 us more.)
constexpr int kLnSumAhead = 8;
constexpr int kLnSumShares = 32 * kLnSumAhead;  // under way at once, with G = 1
template <int G>
__global__ void __launch_bounds__(1024) tg_layer_norm_grad_sum(const LayerNormGradParams q, int blocks) {
    constexpr int kAhead = kLnSumAhead / G;
    __shared__ float part[32][32 * G + 1];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, cols = static_cast<int>(q.n.cols);
    const int c0 = blockIdx.x * 32 * G, here = cols - c0 - lane;  // columns from this thread's first on
    const float* src = blockIdx.y == 0 ? q.ws_w : q.ws_b;
    op_release_next();
    op_wait_previous();
    if (src == nullptr) return;
    float s[G];
#pragma unroll
    for (int g = 0; g < G; ++g) s[g] = 0.0f;
    const float* at = src + (w * cols + c0 + lane);  // (42 million elements at most)
    const int step = 32 * cols;
    for (int k = w; k < blocks; k += 32 * kAhead, at += kAhead * step) {
        float v[kAhead][G];
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
#pragma unroll
            for (int g = 0; g < G; ++g) {
                v[i][g] = 0.0f;
                if (k + 32 * i < blocks && 32 * g < here) v[i][g] = at[i * step + 32 * g];
            }
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
#pragma unroll
            for (int g = 0; g < G; ++g) s[g] += v[i][g];
    }
#pragma unroll
    for (int g = 0; g < G; ++g) part[w][32 * g + lane] = s[g];
    __syncthreads();
    // warp w: columns w, w + 32, ... of them
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const float sum = ln_warp_sum(part[lane][32 * g + w]);
        const int c = c0 + 32 * g + w;
        if (lane == 0 && c < cols) (blockIdx.y == 0 ? q.dw : q.db)[c] = sum;
    }
}

}  // namespace tg
