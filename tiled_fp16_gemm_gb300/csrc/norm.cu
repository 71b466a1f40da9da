// tg_norm_residual and tg_norm_residual_backward (include/tgemm.h): argument
// checks, workspace and launches.  The kernels and the formulas: norm.cuh.
#include <cstring>
#include <type_traits>

#include "norm_host.h"

namespace {

using tg::allow_smem;
using tg::check_matrix;
using tg::elem_bytes;
using tg::known_clusters;
using tg::launch;
using tg::misaligned;
using tg::narrow;
using tg::NormGradParams;
using tg::NormParams;
using tg::plan_rows;
using tg::RowPlan;
using tg::wide;

template <int N>
using Int = std::integral_constant<int, N>;

constexpr int64_t kMaxCols = 32768;  // a row's fp32 values have to fit in shared memory

tg::OpWorkspace g_workspace;  // column sums of the gradient

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
    if ((st = check_matrix(a->x, a->ldx, a->cols, elem_bytes(a->dtype))) != TG_OK) return st;
    if ((st = check_matrix(a->residual, a->ldr, a->cols, elem_bytes(a->stream_dtype))) != TG_OK) return st;
    if ((st = check_matrix(a->gate, a->ldg, a->cols, elem_bytes(a->dtype))) != TG_OK) return st;
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

}  // namespace

static tg_status_t norm_residual(const tg_norm_t* a, void* y, int64_t ldy, void* h, int64_t ldh,
                                 void* stream) {
    NormParams p;
    tg_status_t st = check_norm(a, &p);
    if (st != TG_OK) return st;
    if ((h != nullptr) != (a->pre_weight != nullptr) && a->rows > 0 && a->cols > 0)
        return TG_ERR_INVALID_VALUE;
    if ((st = check_matrix(y, ldy, a->cols, elem_bytes(a->stream_dtype))) != TG_OK) return st;
    if ((st = check_matrix(h, ldh, a->cols, elem_bytes(a->dtype))) != TG_OK) return st;
    if (a->rows == 0 || a->cols == 0 || (y == nullptr && h == nullptr)) return TG_OK;
    p.y = y;
    p.ldy = ldy;
    p.h = h;
    p.ldh = ldh;
    tg::OpDevice dev;
    if ((st = tg::op_device(&dev)) != TG_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return with_types(*a, [&](auto tx, auto tr) {
        using TX = decltype(tx);
        using TR = decltype(tr);
        // whether a thread may read and write 8 neighbouring columns at a time
        const bool vec = p.cols % 8 == 0 && wide(p.x, p.ldx, sizeof(TX)) &&
                         wide(p.r, p.ldr, sizeof(TR)) && wide(p.gate, p.ldg, sizeof(TX)) &&
                         wide(p.wpost, 0, 4) && wide(p.wpre, 0, 4) &&
                         wide(p.y, p.ldy, sizeof(TR)) && wide(p.h, p.ldh, sizeof(TX));
        RowPlan r;
        auto plan = [&](auto ch, auto v) {
            constexpr int CH = decltype(ch)::value;
            constexpr bool VEC = decltype(v)::value;
            const int threads = static_cast<int>((p.cols + 256 * CH - 1) / (256 * CH)) * 32;
            const int bx = tg::norm_stage_bytes<TX, CH, VEC>(threads, p.cols);
            const int stage = bx + tg::norm_stage_bytes<TR, CH, VEC>(threads, p.cols);
            const bool one_gate = p.rows_per_gate == p.rows;
            const int gate = p.gate != nullptr ? bx : 0;
            return threads <= tg::kNormThreads && narrow(p.ldx, p.ldr, p.ldg, p.ldy, p.ldh) &&
                   plan_rows(p.rows, threads, stage + (one_gate ? 0 : gate), one_gate ? gate : 0,
                             CH == 1 && VEC ? 2 : 1, dev.num_sms, &r);
        };
        auto run = [&](auto kernel) {
            if (!allow_smem(kernel, dev.dev)) return TG_ERR_LAUNCH;
            const int64_t most = int64_t{r.per_sm} * dev.num_sms;
            const int64_t blocks = (p.rows + r.groups - 1) / r.groups;
            return launch(kernel, dim3(static_cast<unsigned>(blocks < most ? blocks : most)),
                          r.threads * r.groups, r.smem, 1, s, p, r.threads, r.stages, r.stage_bytes);
        };
        if (vec) {
            if (plan(Int<1>{}, std::true_type{})) return run(tg::tg_norm_residual_rows<TX, TR, 1, true>);
            if (plan(Int<2>{}, std::true_type{})) return run(tg::tg_norm_residual_rows<TX, TR, 2, true>);
            if (plan(Int<4>{}, std::true_type{})) return run(tg::tg_norm_residual_rows<TX, TR, 4, true>);
        } else {
            if (plan(Int<1>{}, std::false_type{})) return run(tg::tg_norm_residual_rows<TX, TR, 1, false>);
            if (plan(Int<2>{}, std::false_type{})) return run(tg::tg_norm_residual_rows<TX, TR, 2, false>);
            if (plan(Int<4>{}, std::false_type{})) return run(tg::tg_norm_residual_rows<TX, TR, 4, false>);
        }
        auto kernel = tg::tg_norm_residual_simple<TX, TR>;
        const size_t smem = static_cast<size_t>(p.cols) * 4;
        if (!allow_smem(kernel, dev.dev)) return TG_ERR_LAUNCH;
        const int64_t grid = p.rows < 8 * dev.num_sms ? p.rows : 8 * dev.num_sms;
        return launch(kernel, dim3(static_cast<unsigned>(grid)), 256, smem, 1, s, p);
    });
}

static tg_status_t norm_residual_backward(const tg_norm_t* a, const tg_norm_grad_t* b, void* stream) {
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
    if ((st = check_matrix(b->dy, b->lddy, a->cols, elem_bytes(a->stream_dtype))) != TG_OK) return st;
    if ((st = check_matrix(b->dh, b->lddh, a->cols, elem_bytes(a->dtype))) != TG_OK) return st;
    if ((st = check_matrix(b->dx, b->lddx, a->cols, elem_bytes(a->dtype))) != TG_OK) return st;
    if ((st = check_matrix(b->dresidual, b->lddr, a->cols, elem_bytes(a->stream_dtype))) != TG_OK) return st;
    if ((st = check_matrix(b->dgate, b->lddg, a->cols, elem_bytes(a->dtype))) != TG_OK) return st;
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
    return with_types(*a, [&](auto tx, auto tr) {
        using TX = decltype(tx);
        using TR = decltype(tr);
        const void* in[4] = {q.n.x, q.n.r, q.dy, q.dh};
        const int64_t ld[4] = {q.n.ldx, q.n.ldr, q.lddy, q.lddh};
        const int elem[4] = {sizeof(TX), sizeof(TR), sizeof(TR), sizeof(TX)};
        bool vec = cols % 8 == 0 && wide(q.n.wpost, 0, 4) && wide(q.n.wpre, 0, 4) &&
                   wide(q.n.gate, q.n.ldg, sizeof(TX)) && wide(q.dx, q.lddx, sizeof(TX)) &&
                   wide(q.dr, q.lddr, sizeof(TR)) && wide(q.dgate, q.lddg, sizeof(TX)) &&
                   wide(q.dwpost, 0, 4) && wide(q.dwpre, 0, 4);
        for (int k = 0; k < 4; ++k) vec = vec && wide(in[k], ld[k], elem[k]);
        RowPlan r;
        // 8 columns of a thread; longer rows on the blocks of a cluster
        int split = 1;
        while (split < tg::kNormSplit && cols > int64_t{split} * 8 * tg::kNormThreads) split *= 2;
        const int part = split == 1 ? static_cast<int>(cols)
                                    : static_cast<int>((cols + 8 * split - 1) / (8 * split)) * 8;
        auto plan = [&](auto v) {
            constexpr bool VEC = decltype(v)::value;
            const int threads = (part + 255) / 256 * 32;
            const int bx = tg::norm_stage_bytes<TX, 1, VEC>(threads, part);
            const int stage = 2 * (bx + tg::norm_stage_bytes<TR, 1, VEC>(threads, part));
            const bool one_gate = q.n.rows_per_gate == a->rows;
            const int gate = q.n.gate != nullptr ? bx : 0;
            const int join = threads * 32;  // a group's column sums
            // (the groups of a block would take rows in turn: one, where blocks share rows)
            return narrow(q.n.ldx, q.n.ldr, q.n.ldg, q.lddx, q.lddr) &&
                   narrow(q.lddy, q.lddh, 0, 0, 0) && (split == 1 || threads > tg::kNormThreads / 2) &&
                   plan_rows(a->rows, threads, stage + (one_gate ? 0 : gate),
                             bx + (tg::kNormThreads / threads > 1 ? join : 0), 1, dev.num_sms, &r);
        };
        const bool ring = vec ? plan(std::true_type{}) : plan(std::false_type{});
        int64_t most = ring ? dev.num_sms : 2 * dev.num_sms;
        if (ring && split > 1) {
            const auto kernel = vec ? tg::tg_norm_grad_rows<TX, TR, true, true>
                                    : tg::tg_norm_grad_rows<TX, TR, false, true>;
            if (!allow_smem(kernel, dev.dev)) return TG_ERR_LAUNCH;
            most = known_clusters(kernel, split, r.threads, r.smem, dev);
            if (most < 1) return TG_ERR_LAUNCH;
        }
        const int64_t wanted = ring ? (a->rows + r.groups - 1) / r.groups : a->rows;
        const int64_t blocks = wanted < most ? wanted : most;
        // Many gates: a block takes whole gates.  Few: it takes rows, and the
        // blocks' shares of a gate are summed afterwards.
        const bool gate_sums = q.dgate != nullptr && q.n.rows_per_gate > 1;
        if (gate_sums && q.gates >= 2 * blocks) q.whole_gates = 1;
        // (a thread of the row kernels sums its whole gates in registers)
        const int64_t gate_slots = !gate_sums                ? 0
                                   : !q.whole_gates ? blocks + q.gates
                                   : ring           ? 0
                                                    : blocks;
        const int64_t slots = (q.dwpost != nullptr ? blocks : 0) +
                              (q.dwpre != nullptr ? blocks : 0) + gate_slots;
        tg::OpWorkspace::Hold hold;  // until the shares' sums are launched
        if (slots > 0) {
            void* ws = nullptr;
            st = g_workspace.get(dev.dev, s, static_cast<size_t>(slots * cols) * 4, &ws, &hold);
            if (st != TG_OK) return st;
            float* next = static_cast<float*>(ws);
            if (q.dwpost != nullptr) q.ws_post = next, next += blocks * cols;
            if (q.dwpre != nullptr) q.ws_pre = next, next += blocks * cols;
            if (gate_slots > 0) q.ws_gate = next;
        }
        const dim3 grid(static_cast<unsigned>(ring ? blocks * split : blocks));
        if (ring) {
            auto run = [&](auto kernel) {
                if (!allow_smem(kernel, dev.dev)) return TG_ERR_LAUNCH;
                return launch(kernel, grid, r.threads * r.groups, r.smem, split, s, q, r.threads, r.stages,
                              r.stage_bytes, split, part, tg::op_wait_limit_ns(), dev.timeouts,
                              split > 1 ? tg::op_take_inject() : 0);
            };
            if (split > 1)
                st = vec ? run(tg::tg_norm_grad_rows<TX, TR, true, true>)
                         : run(tg::tg_norm_grad_rows<TX, TR, false, true>);
            else
                st = vec ? run(tg::tg_norm_grad_rows<TX, TR, true, false>)
                         : run(tg::tg_norm_grad_rows<TX, TR, false, false>);
        } else {
            auto kernel = tg::tg_norm_grad_simple<TX, TR>;
            const size_t smem = static_cast<size_t>(cols) * 4;
            if (!allow_smem(kernel, dev.dev)) return TG_ERR_LAUNCH;
            st = launch(kernel, grid, 256, smem, 1, s, q);
        }
        if (st != TG_OK || slots == 0) return st;
        const int64_t jobs = 2 + (gate_sums && !q.whole_gates ? q.gates : 0);
        return launch(tg::tg_norm_grad_sum<TX>,
                      dim3(static_cast<unsigned>((cols + 31) / 32),
                           static_cast<unsigned>(jobs < 1024 ? jobs : 1024)),
                      512, 0, 1, s, q, blocks, jobs);
    });
}

extern "C" {

tg_status_t tg_norm_residual(const tg_norm_t* a, void* y, int64_t ldy, void* h, int64_t ldh,
                             void* stream) {
    return tg::op_entry([&] { return norm_residual(a, y, ldy, h, ldh, stream); });
}

tg_status_t tg_norm_residual_backward(const tg_norm_t* a, const tg_norm_grad_t* b, void* stream) {
    return tg::op_entry([&] { return norm_residual_backward(a, b, stream); });
}

}  // extern "C"
