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

constexpr uint32_t kLnInf = 0x7f800000u;

// The scale of a row whose largest |value| has these bits.  With a NaN or an infinity among
// the values (as bits, both are the largest) no scale can stand for the row: it is NaN.
__device__ __forceinline__ float ln_scale(uint32_t largest) {
    return largest >= kLnInf ? __uint_as_float(0x7fc00000u) : __fdiv_rn(__uint_as_float(largest), 127.0f);
}
// For ln_code: what value and scale are multiplied by (a power of two; 1 but for scales whose
// reciprocal would leave fp32), and the reciprocal.  A row of zeros (or of values so small that
// their scale is 0), and one without a scale, has codes 0.
struct LnCoder {
    float up, scale, inv;
    __device__ __forceinline__ explicit LnCoder(float s) {
        up = s < 1e-30f ? 1.2676506e30f : 1.0f;  // 2^100
        scale = s * up;
        inv = s > 0.0f ? __frcp_rn(scale) : 0.0f;
    }
    // value / scale to the nearest, exactly: the product with the reciprocal is off by 2^-22 of
    // it at most, so it rounds to the right whole number or, near a half, to one beside it; what
    // is left over, value - q · scale, is exact in fp32 and tells which.
    __device__ __forceinline__ int code(float value) const {
        if (!(inv > 0.0f)) return 0;
        value *= up;
        float q = rintf(value * inv);
        const float rest = fmaf(-q, scale, value), twice = 2.0f * fabsf(rest);
        const bool odd = (__float2int_rn(q) & 1) != 0;
        if (twice > scale || (twice == scale && odd)) q += rest > 0.0f ? 1.0f : -1.0f;
        return __float2int_rn(fminf(fmaxf(q, -127.0f), 127.0f));  // (the least scales are coarse)
    }
};

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

// ------------------------------------------------------------------ any width and stride
//
// A row per block and turn; values are read again for each pass, from L2.

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
        float mean = 0.0f, s = 1.0f;
        if (MODE != kLnRaw) {
            float a = 0.0f;
            for (int64_t c = threadIdx.x; c < p.cols; c += blockDim.x) a += value(c);
            mean = norm_block_sum(a, red) * inv;
            a = 0.0f;
            for (int64_t c = threadIdx.x; c < p.cols; c += blockDim.x) {
                const float d = value(c) - mean;
                a += d * d;
            }
            s = rsqrtf(norm_block_sum(a, red) * inv + p.eps);
        }
        auto normed = [&](float v, int64_t c) {
            if (MODE == kLnRaw) return v;
            const float n = (v - mean) * s;
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
        const LnCoder coder(scale);
        // (the last look at r: y may take its place)
        for (int64_t c = threadIdx.x; c < p.cols; c += blockDim.x) {
            const float v = value(c), h = normed(v, c);
            if (MODE == kLnH) {
                if (p.h != nullptr) (static_cast<TX*>(p.h) + row * p.ldh)[c] = op_round<TX>(h);
            } else {
                (static_cast<int8_t*>(p.h) + row * p.ldh)[c] = static_cast<int8_t>(coder.code(h));
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
        float mean = 0.0f, s = 0.0f, m1 = 0.0f, m2 = 0.0f;
        if (dh != nullptr) {  // else nothing is taken of v, which need not be finite then
            float a = 0.0f, b = 0.0f, d = 0.0f;
            for (int64_t c = threadIdx.x; c < p.cols; c += blockDim.x) a += value(c);
            mean = norm_block_sum(a, red) * inv;
            a = 0.0f;
            for (int64_t c = threadIdx.x; c < p.cols; c += blockDim.x) {
                const float u = value(c) - mean, dn = dn_at(c);
                a += u * u;
                b += dn;
                d += dn * u;
            }
            s = rsqrtf(norm_block_sum(a, red) * inv + p.eps);
            m1 = norm_block_sum(b, red) * inv;
            m2 = norm_block_sum(d, red) * inv * s;
        }
        for (int64_t c = threadIdx.x; c < p.cols; c += blockDim.x) {
            float d = dy != nullptr ? op_to_float(dy[c]) : 0.0f;
            if (dh != nullptr) {
                const float n = (value(c) - mean) * s;
                d += s * (dn_at(c) - m1 - n * m2);
                if (ww != nullptr) ww[c] = (row == row0 ? 0.0f : ww[c]) + op_to_float(dh[c]) * n;
                if (wb != nullptr) wb[c] = (row == row0 ? 0.0f : wb[c]) + op_to_float(dh[c]);
            }
            if (q.dx != nullptr) (static_cast<TX*>(q.dx) + row * q.lddx)[c] = op_round<TX>(d);
            if (q.dr != nullptr) (static_cast<TR*>(q.dr) + row * q.lddr)[c] = op_round<TR>(d);
        }
    }
}

// The column sums of the blocks' shares, in the order of the blocks: blockIdx.y 0: dw, 1: db.
// 32 columns per block, 16 warps with every 16th share each, 8 of them under way at a time.
__global__ void __launch_bounds__(512) tg_layer_norm_grad_sum(const LayerNormGradParams q, int64_t blocks) {
    __shared__ float part[16][33];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    op_release_next();
    op_wait_previous();
    const int64_t c = int64_t{blockIdx.x} * 32 + lane;
    const float* src = blockIdx.y == 0 ? q.ws_w : q.ws_b;
    if (src == nullptr) return;
    float s = 0.0f;
    if (c < q.n.cols) {
        for (int64_t k = w; k < blocks; k += 128) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = k + 16 * i < blocks ? src[(k + 16 * i) * q.n.cols + c] : 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) s += v[i];
        }
    }
    part[w][lane] = s;
    __syncthreads();
    if (w == 0 && c < q.n.cols) {
#pragma unroll
        for (int k = 1; k < 16; ++k) s += part[k][lane];
        (blockIdx.y == 0 ? q.dw : q.db)[c] = s;
    }
}

}  // namespace tg
