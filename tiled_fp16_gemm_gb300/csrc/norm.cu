// tg_norm_residual and tg_norm_residual_backward (include/tgemm.h): argument
// checks, workspace and launches.  The kernels and the formulas: norm.cuh.
#include <cstring>

#include "norm.cuh"
#include "op_host.h"

namespace {

using tg::NormGradParams;
using tg::NormParams;

constexpr int64_t kMaxCols = 32768;  // a row's fp32 values have to fit in shared memory

tg::OpWorkspace g_workspace;  // column sums of the gradient

int elem_bytes(int32_t dtype) { return dtype == TG_DTYPE_F32 ? 4 : 2; }

bool misaligned(const void* p, int bytes) {
    return (reinterpret_cast<uintptr_t>(p) & static_cast<uintptr_t>(bytes - 1)) != 0;
}

// One matrix argument: present or not, its stride, its alignment.
tg_status_t check_matrix(const void* p, int64_t ld, int64_t cols, int32_t dtype) {
    if (p == nullptr) return TG_OK;
    if (ld < cols) return TG_ERR_INVALID_VALUE;
    return misaligned(p, elem_bytes(dtype)) ? TG_ERR_MISALIGNED : TG_OK;
}

// The arguments that the forward and the backward call share.
tg_status_t check_norm(const tg_norm_t* a, NormParams* p) {
    if (a == nullptr) return TG_ERR_INVALID_VALUE;
    if (a->dtype != TG_DTYPE_F16 && a->dtype != TG_DTYPE_BF16 && a->dtype != TG_DTYPE_F32)
        return TG_ERR_INVALID_VALUE;
    if (a->stream_dtype != a->dtype && a->stream_dtype != TG_DTYPE_F32) return TG_ERR_INVALID_VALUE;
    if (a->rows < 0 || a->rows > tg::kOpMaxDim || a->cols < 0 || a->cols > kMaxCols)
        return TG_ERR_INVALID_VALUE;
    if (!(a->eps >= 0.0f)) return TG_ERR_INVALID_VALUE;
    if (a->gate != nullptr &&
        (a->gate_rows < 1 || (a->rows > 0 && (a->gate_rows > a->rows || a->rows % a->gate_rows != 0))))
        return TG_ERR_INVALID_VALUE;
    if (a->rows > 0 && a->cols > 0 && a->x == nullptr) return TG_ERR_INVALID_VALUE;
    tg_status_t st;
    if ((st = check_matrix(a->x, a->ldx, a->cols, a->dtype)) != TG_OK) return st;
    if ((st = check_matrix(a->residual, a->ldr, a->cols, a->stream_dtype)) != TG_OK) return st;
    if ((st = check_matrix(a->gate, a->ldg, a->cols, a->dtype)) != TG_OK) return st;
    if (misaligned(a->post_weight, 4) || misaligned(a->pre_weight, 4)) return TG_ERR_MISALIGNED;
    std::memset(p, 0, sizeof(*p));
    p->rows = a->rows;
    p->cols = a->cols;
    p->x = a->x;
    p->ldx = a->ldx;
    p->r = a->residual;
    p->ldr = a->ldr;
    p->wpost = a->post_weight;
    p->gate = a->gate;
    p->ldg = a->ldg;
    p->rows_per_gate = a->gate != nullptr && a->rows > 0 ? a->rows / a->gate_rows : 1;
    p->wpre = a->pre_weight;
    p->scale = a->scale;
    p->eps = a->eps;
    return TG_OK;
}

// f<TX, TR>() for the call's types.
template <typename F>
tg_status_t with_types(const tg_norm_t& a, F f) {
    const bool wide = a.stream_dtype == TG_DTYPE_F32;
    if (a.dtype == TG_DTYPE_F32) return f(float{}, float{});
    if (a.dtype == TG_DTYPE_F16) return wide ? f(__half{}, float{}) : f(__half{}, __half{});
    return wide ? f(__nv_bfloat16{}, float{}) : f(__nv_bfloat16{}, __nv_bfloat16{});
}

tg_status_t launched() {
    if (cudaGetLastError() != cudaSuccess) return TG_ERR_LAUNCH;
    return TG_OK;
}

template <typename Kernel>
bool allow_smem(Kernel k, size_t bytes) {
    if (bytes <= 48 * 1024) return true;
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(bytes)) == cudaSuccess)
        return true;
    cudaGetLastError();
    return false;
}

}  // namespace

extern "C" {

tg_status_t tg_norm_residual(const tg_norm_t* a, void* y, int64_t ldy, void* h, int64_t ldh,
                             void* stream) {
    NormParams p;
    tg_status_t st = check_norm(a, &p);
    if (st != TG_OK) return st;
    if ((h != nullptr) != (a->pre_weight != nullptr) && a->rows > 0 && a->cols > 0)
        return TG_ERR_INVALID_VALUE;
    if ((st = check_matrix(y, ldy, a->cols, a->stream_dtype)) != TG_OK) return st;
    if ((st = check_matrix(h, ldh, a->cols, a->dtype)) != TG_OK) return st;
    if (a->rows == 0 || a->cols == 0 || (y == nullptr && h == nullptr)) return TG_OK;
    p.y = y;
    p.ldy = ldy;
    p.h = h;
    p.ldh = ldh;
    tg::OpDevice dev;
    if ((st = tg::op_device(&dev)) != TG_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return with_types(*a, [&](auto tx, auto tr) {
        auto kernel = tg::tg_norm_residual_simple<decltype(tx), decltype(tr)>;
        const size_t smem = static_cast<size_t>(p.cols) * 4;
        if (!allow_smem(kernel, smem)) return TG_ERR_LAUNCH;
        const int64_t grid = p.rows < 8 * dev.num_sms ? p.rows : 8 * dev.num_sms;
        kernel<<<static_cast<unsigned>(grid), 256, smem, s>>>(p);
        return launched();
    });
}

tg_status_t tg_norm_residual_backward(const tg_norm_t* a, const tg_norm_grad_t* b, void* stream) {
    NormGradParams q;
    std::memset(&q, 0, sizeof(q));
    if (b == nullptr) return TG_ERR_INVALID_VALUE;
    tg_status_t st = check_norm(a, &q.n);
    if (st != TG_OK) return st;
    if (b->dh != nullptr && a->pre_weight == nullptr) return TG_ERR_INVALID_VALUE;
    if ((b->dgate != nullptr && a->gate == nullptr) ||
        (b->dpost_weight != nullptr && a->post_weight == nullptr) ||
        (b->dpre_weight != nullptr && a->pre_weight == nullptr))
        return TG_ERR_INVALID_VALUE;
    if ((st = check_matrix(b->dy, b->lddy, a->cols, a->stream_dtype)) != TG_OK) return st;
    if ((st = check_matrix(b->dh, b->lddh, a->cols, a->dtype)) != TG_OK) return st;
    if ((st = check_matrix(b->dx, b->lddx, a->cols, a->dtype)) != TG_OK) return st;
    if ((st = check_matrix(b->dresidual, b->lddr, a->cols, a->stream_dtype)) != TG_OK) return st;
    if ((st = check_matrix(b->dgate, b->lddg, a->cols, a->dtype)) != TG_OK) return st;
    if (misaligned(b->dpost_weight, 4) || misaligned(b->dpre_weight, 4)) return TG_ERR_MISALIGNED;
    if (a->cols == 0) return TG_OK;
    tg::OpDevice dev;
    if ((st = tg::op_device(&dev)) != TG_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    q.dy = b->dy;
    q.lddy = b->lddy;
    q.dh = b->dh;
    q.lddh = b->lddh;
    q.dx = b->dx;
    q.lddx = b->lddx;
    q.dr = b->dresidual;
    q.lddr = b->lddr;
    q.dgate = b->dgate;
    q.lddg = b->lddg;
    q.dwpost = b->dpost_weight;
    q.dwpre = b->dpre_weight;
    q.gates = a->gate != nullptr ? a->gate_rows : 0;
    const int64_t cols = a->cols;
    // Sums over no rows are zero (a pre_weight whose norm has no dh too).
    auto zero = [&](void* p, int64_t ld, int64_t rows, int bytes) {
        if (p != nullptr && cudaMemset2DAsync(p, static_cast<size_t>(ld) * bytes, 0,
                                              static_cast<size_t>(cols) * bytes,
                                              static_cast<size_t>(rows), s) != cudaSuccess) {
            cudaGetLastError();
            st = TG_ERR_LAUNCH;
        }
    };
    if (a->rows == 0) {
        zero(q.dwpost, cols, 1, 4);
        zero(q.dwpre, cols, 1, 4);
        zero(q.dgate, q.lddg, q.gates, elem_bytes(a->dtype));
        return st;
    }
    if (q.dh == nullptr) {
        zero(q.dwpre, cols, 1, 4);
        q.dwpre = nullptr;
        if (st != TG_OK) return st;
    }
    const int64_t most = 2 * dev.num_sms;
    int64_t blocks = a->rows < most ? a->rows : most;
    // Many gates: a block takes whole gates.  Few: it takes rows, and the
    // blocks' shares of a gate are summed afterwards.
    const bool gate_sums = q.dgate != nullptr && q.n.rows_per_gate > 1;
    if (gate_sums && q.gates >= 2 * blocks) q.whole_gates = 1;
    const int64_t gate_slots = !gate_sums ? 0 : q.whole_gates ? blocks : blocks + q.gates;
    const int64_t slots = (q.dwpost != nullptr ? blocks : 0) + (q.dwpre != nullptr ? blocks : 0) +
                          gate_slots;
    if (slots > 0) {
        void* ws = nullptr;
        if ((st = g_workspace.get(dev.dev, s, static_cast<size_t>(slots * cols) * 4, &ws)) != TG_OK)
            return st;
        float* next = static_cast<float*>(ws);
        if (q.dwpost != nullptr) q.ws_post = next, next += blocks * cols;
        if (q.dwpre != nullptr) q.ws_pre = next, next += blocks * cols;
        if (gate_slots > 0) q.ws_gate = next;
    }
    return with_types(*a, [&](auto tx, auto tr) {
        auto kernel = tg::tg_norm_grad_simple<decltype(tx), decltype(tr)>;
        const size_t smem = static_cast<size_t>(cols) * 4;
        if (!allow_smem(kernel, smem)) return TG_ERR_LAUNCH;
        kernel<<<static_cast<unsigned>(blocks), 256, smem, s>>>(q);
        if (slots > 0) {
            const int64_t jobs = 2 + (q.whole_gates ? 0 : q.gates);
            const dim3 grid(static_cast<unsigned>((cols + 31) / 32),
                            static_cast<unsigned>(jobs < 1024 ? jobs : 1024));
            tg::tg_norm_grad_sum<decltype(tx)><<<grid, 256, 0, s>>>(q, blocks);
        }
        return launched();
    });
}

}  // extern "C"
