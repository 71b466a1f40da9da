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

// Row by row, the unrounded y of the row in shared memory.
template <typename TX, typename TR>
__global__ void __launch_bounds__(256) tg_norm_residual_simple(const NormParams p) {
    extern __shared__ float norm_buf[];
    __shared__ float red[33];
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

// The column sums of the blocks' shares, in the order of the blocks:
// blockIdx.y 0 and 1: dwpost and dwpre; 2 + i: gate i.
template <typename TX>
__global__ void __launch_bounds__(256)
    tg_norm_grad_sum(const NormGradParams q, int64_t blocks) {
    __shared__ float part[8][33];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int64_t c = int64_t{blockIdx.x} * 32 + lane;
    for (int64_t job = blockIdx.y; job < 2 + q.gates; job += gridDim.y) {
        const float* src = job == 0 ? q.ws_post : job == 1 ? q.ws_pre : q.ws_gate;
        if (src == nullptr || (job >= 2 && q.whole_gates)) continue;
        int64_t lo = 0, hi = blocks;
        if (job >= 2) {  // the pieces of gate i: slots block + i of the blocks that have its rows
            const int64_t i = job - 2, per = q.n.rows_per_gate;
            int64_t a = 0, b = blocks - 1;
            while (norm_first_row(q.n.rows, blocks, a + 1) <= i * per) ++a;
            while (norm_first_row(q.n.rows, blocks, b) >= (i + 1) * per) --b;
            lo = a + i;
            hi = b + i + 1;
        }
        float s = 0.0f;
        if (c < q.n.cols)
            for (int64_t k = lo + w; k < hi; k += 8) s += src[k * q.n.cols + c];
        part[w][lane] = s;
        __syncthreads();
        if (w == 0 && c < q.n.cols) {
            for (int k = 1; k < 8; ++k) s += part[k][lane];
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
