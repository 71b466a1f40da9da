// tg_layer_norm, tg_layer_norm_i8, tg_quantize_rows and tg_layer_norm_backward
// (include/tgemm.h): argument checks, workspace and launches.  The kernels and the formulas:
// layer_norm.cuh.
#include <cstring>
#include <type_traits>

#include "layer_norm.cuh"
#include "norm_host.h"

namespace {

using tg::allow_smem;
using tg::check_matrix;
using tg::elem_bytes;
using tg::known_clusters;
using tg::kRingBytes;
using tg::launch;
using tg::LayerNormGradParams;
using tg::LayerNormParams;
using tg::misaligned;
using tg::wide;

constexpr int64_t kMaxCols = 131071;   // codes of a row: whole sums of gemm_i8 fit 32 bits
constexpr int64_t kGradBlocks = 320;   // that share the column sums, at most

tg::OpWorkspace g_workspace;  // column sums of the gradient, where the caller has none

// The arguments that all calls share.
tg_status_t check_norm(const tg_layer_norm_t* a, LayerNormParams* p) {
    if (a == nullptr) return TG_ERR_INVALID_VALUE;
    if (a->dtype != TG_DTYPE_F16 && a->dtype != TG_DTYPE_BF16 && a->dtype != TG_DTYPE_F32)
        return TG_ERR_INVALID_VALUE;
    if (a->stream_dtype != a->dtype && a->stream_dtype != TG_DTYPE_F32) return TG_ERR_INVALID_VALUE;
    if (a->rows < 0 || a->rows > tg::kOpMaxDim || a->cols < 0 || a->cols > kMaxCols)
        return TG_ERR_INVALID_VALUE;
    if (!(a->eps >= 0.0f)) return TG_ERR_INVALID_VALUE;
    if (a->rows > 0 && a->cols > 0 && a->x == nullptr) return TG_ERR_INVALID_VALUE;
    tg_status_t st;
    if ((st = check_matrix(a->x, a->ldx, a->cols, elem_bytes(a->dtype))) != TG_OK) return st;
    if ((st = check_matrix(a->residual, a->ldr, a->cols, elem_bytes(a->stream_dtype))) != TG_OK) return st;
    if (misaligned(a->weight, 4) || misaligned(a->bias, 4)) return TG_ERR_MISALIGNED;
    std::memset(p, 0, sizeof(*p));
    p->rows = a->rows;
    p->cols = a->cols;
    p->x = a->x;
    p->ldx = a->ldx;
    p->r = a->residual;
    p->ldr = a->ldr;
    p->w = a->weight;
    p->b = a->bias;
    p->eps = a->eps;
    return TG_OK;
}

// f<TX, TR>() for the call's types.
template <typename F>
tg_status_t with_types(int32_t dtype, int32_t stream_dtype, F f) {
    const bool wide = stream_dtype == TG_DTYPE_F32;
    if (dtype == TG_DTYPE_F32) return f(float{}, float{});
    if (dtype == TG_DTYPE_F16) return wide ? f(__half{}, float{}) : f(__half{}, __half{});
    return wide ? f(__nv_bfloat16{}, float{}) : f(__nv_bfloat16{}, __nv_bfloat16{});
}

template <int N>
using Int = std::integral_constant<int, N>;

// Rows in registers where they fit: of the widths of a thread's share (8·CH columns) the largest
// that leaves no SM without warps.
template <typename TX, typename TR, int MODE>
tg_status_t launch_rows(const LayerNormParams& p, const tg::OpDevice& dev, cudaStream_t s) {
    // whether a thread may read and write 8 neighbouring columns at a time
    const int out = MODE == tg::kLnH ? sizeof(TX) : 1;
    const bool vec = p.cols % 8 == 0 && wide(p.x, p.ldx, sizeof(TX)) && wide(p.r, p.ldr, sizeof(TR)) &&
                     wide(p.w, 0, 4) && wide(p.b, 0, 4) && wide(p.y, p.ldy, sizeof(TR)) && wide(p.h, p.ldh, out);
    const int64_t cols = p.cols;
    auto warps = [&](int ch) { return (cols + 256 * ch - 1) / (256 * ch); };  // of a row
    auto run = [&](auto ch, auto v, auto sm) {
        constexpr int CH = decltype(ch)::value;
        const int threads = static_cast<int>(warps(CH)) * 32;
        const int64_t each = (p.rows + dev.num_sms - 1) / dev.num_sms;
        const int64_t groups = threads > 32 ? 1 : each < 4 ? each : 4;  // rows of a block
        const int64_t blocks = (p.rows + groups - 1) / groups;
        return launch(tg::tg_layer_norm_rows<TX, TR, CH, decltype(v)::value, MODE, decltype(sm)::value>,
                      dim3(static_cast<unsigned>(blocks)), static_cast<int>(threads * groups), 0, 1, s, p, threads);
    };
    // whether the SMs hold all rows with 512 threads each
    auto few = [&](int n) { return p.rows * warps(n) * 32 <= 512 * int64_t{dev.num_sms}; };
    // (16 warps of four runs leave an SM one block; few rows gain: 152×16384 6.7 us, 8.1 with eight)
    auto fits = [&](int n) { return warps(n) <= (vec && n == 4 && !few(4) ? 12 : 16); };
    int ch = !vec || fits(4) ? 4 : 8;
    while (ch > 1 && (cols <= 128 * ch || (p.rows * warps(ch) < 8 * dev.num_sms && fits(ch / 2)))) ch /= 2;
    // Threads of an SM, for which a kernel's registers are: in rows of four runs 640, of eight 512; else
    // 1024, and 512 where that holds all rows, whose weights come with them (16×1024 1.9 us, 2.1 without;
    // 64×8192 2.95, 3.25).
    if (vec && fits(ch)) {
        // Warps that have all of their columns (2050×1536 8.2 us with three of 512, 8.8 with two of
        // 1024; 1200×768 4.3 and 4.7), where an SM does not hold fewer rows for it, or holds all
        // (700×3584 6.2 us with four of 1024, 8.3 with seven of 512 in two waves).
        auto held = [&](int n) { return (n > 2 ? 640 : 1024) / (32 * warps(n)); };  // rows, of an SM
        while ((ch == 4 || ch == 2) && cols % (256 * ch) != 0 && cols % (128 * ch) == 0 && fits(ch / 2) &&
               (held(ch / 2) >= held(ch) || p.rows <= held(ch / 2) * dev.num_sms))
            ch /= 2;
        std::true_type v;
        if (ch == 1) return few(1) ? run(Int<1>{}, v, Int<512>{}) : run(Int<1>{}, v, Int<1024>{});
        if (ch == 2) return few(2) ? run(Int<2>{}, v, Int<512>{}) : run(Int<2>{}, v, Int<1024>{});
        return ch == 4 ? run(Int<4>{}, v, Int<640>{}) : run(Int<8>{}, v, Int<512>{});
    }
    if (!vec && warps(4) <= 32) {
        std::false_type v;
        if (warps(ch) > 16) return run(Int<4>{}, v, Int<1024>{});  // (registers do not hold all)
        if (ch == 1) return few(1) ? run(Int<1>{}, v, Int<512>{}) : run(Int<1>{}, v, Int<1024>{});
        if (ch == 2) return few(2) ? run(Int<2>{}, v, Int<512>{}) : run(Int<2>{}, v, Int<1024>{});
        // (640 where an SM then has a block more: 1021×5119 12.9 us, 14.7 with 512; 700×9999 17.3, 22.6)
        return warps(4) <= 10 ? run(Int<4>{}, v, Int<640>{}) : run(Int<4>{}, v, Int<512>{});
    }
    const int64_t most = 8 * int64_t{dev.num_sms};
    return launch(tg::tg_layer_norm_simple<TX, TR, MODE>,
                  dim3(static_cast<unsigned>(p.rows < most ? p.rows : most)), 256, 0, 1, s, p);
}

// y, and h or the codes of a norm.
tg_status_t forward(const tg_layer_norm_t* a, void* y, int64_t ldy, void* h, int64_t ldh, float* scale,
                    bool codes, void* stream) {
    LayerNormParams p;
    tg_status_t st = check_norm(a, &p);
    if (st != TG_OK) return st;
    if (y != nullptr && a->residual == nullptr) return TG_ERR_INVALID_VALUE;
    if ((st = check_matrix(y, ldy, a->cols, elem_bytes(a->stream_dtype))) != TG_OK) return st;
    if ((st = check_matrix(h, ldh, a->cols, codes ? 1 : elem_bytes(a->dtype))) != TG_OK) return st;
    if (codes && misaligned(scale, 4)) return TG_ERR_MISALIGNED;
    if (a->rows == 0 || a->cols == 0) return TG_OK;
    if (codes ? h == nullptr || scale == nullptr : h == nullptr && y == nullptr) return TG_ERR_INVALID_VALUE;
    p.y = y;
    p.ldy = ldy;
    p.h = h;
    p.ldh = ldh;
    p.scale = scale;
    tg::OpDevice dev;
    if ((st = tg::op_device(&dev)) != TG_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return with_types(a->dtype, a->stream_dtype, [&](auto tx, auto tr) {
        using TX = decltype(tx);
        using TR = decltype(tr);
        return codes ? launch_rows<TX, TR, tg::kLnCodes>(p, dev, s) : launch_rows<TX, TR, tg::kLnH>(p, dev, s);
    });
}

tg_status_t quantize(int32_t dtype, const void* x, int64_t ldx, int8_t* codes, int64_t ldc, float* scale,
                     int64_t rows, int64_t cols, void* stream) {
    tg_layer_norm_t a;
    std::memset(&a, 0, sizeof(a));
    a.dtype = a.stream_dtype = dtype;
    a.rows = rows;
    a.cols = cols;
    a.x = x;
    a.ldx = ldx;
    LayerNormParams p;
    tg_status_t st = check_norm(&a, &p);
    if (st != TG_OK) return st;
    if ((st = check_matrix(codes, ldc, cols, 1)) != TG_OK) return st;
    if (misaligned(scale, 4)) return TG_ERR_MISALIGNED;
    if (rows == 0 || cols == 0) return TG_OK;
    if (codes == nullptr || scale == nullptr) return TG_ERR_INVALID_VALUE;
    p.h = codes;
    p.ldh = ldc;
    p.scale = scale;
    tg::OpDevice dev;
    if ((st = tg::op_device(&dev)) != TG_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return with_types(dtype, dtype, [&](auto tx, auto) {
        using TX = decltype(tx);
        return launch_rows<TX, TX, tg::kLnRaw>(p, dev, s);
    });
}

int64_t grad_workspace(int64_t rows, int64_t cols) {
    return (rows < kGradBlocks ? rows : kGradBlocks) * cols * 8;
}

tg_status_t backward(const tg_layer_norm_t* a, const tg_layer_norm_grad_t* b, void* stream) {
    LayerNormGradParams q;
    std::memset(&q, 0, sizeof(q));
    if (b == nullptr) return TG_ERR_INVALID_VALUE;
    tg_status_t st = check_norm(a, &q.n);
    if (st != TG_OK) return st;
    const int bx = elem_bytes(a->dtype), br = elem_bytes(a->stream_dtype);
    if (b->dresidual != nullptr && a->residual == nullptr) return TG_ERR_INVALID_VALUE;
    if (b->dweight != nullptr && a->weight == nullptr) return TG_ERR_INVALID_VALUE;
    if ((st = check_matrix(b->dy, b->lddy, a->cols, br)) != TG_OK) return st;
    if ((st = check_matrix(b->dh, b->lddh, a->cols, bx)) != TG_OK) return st;
    if ((st = check_matrix(b->dx, b->lddx, a->cols, bx)) != TG_OK) return st;
    if ((st = check_matrix(b->dresidual, b->lddr, a->cols, br)) != TG_OK) return st;
    if (misaligned(b->dweight, 4) || misaligned(b->dbias, 4) || misaligned(b->workspace, 256))
        return TG_ERR_MISALIGNED;
    if (b->workspace != nullptr && b->workspace_bytes < grad_workspace(a->rows, a->cols))
        return TG_ERR_INVALID_VALUE;
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
    q.dw = b->dweight;
    q.db = b->dbias;
    const int64_t cols = a->cols;
    if (a->rows == 0 || q.dh == nullptr) {  // sums of nothing
        for (float* sum : {q.dw, q.db})
            if (sum != nullptr && cudaMemsetAsync(sum, 0, static_cast<size_t>(cols) * 4, s) != cudaSuccess) {
                cudaGetLastError();
                return TG_ERR_LAUNCH;
            }
        q.dw = q.db = nullptr;
    }
    if (a->rows == 0 || (q.dx == nullptr && q.dr == nullptr && q.dw == nullptr && q.db == nullptr)) return TG_OK;
    return with_types(a->dtype, a->stream_dtype, [&](auto tx, auto tr) {
        using TX = decltype(tx);
        using TR = decltype(tr);
        const void* in[4] = {q.n.x, q.n.r, q.dy, q.dh};
        const int64_t ld[4] = {q.n.ldx, q.n.ldr, q.lddy, q.lddh};
        const int elem[4] = {sizeof(TX), sizeof(TR), sizeof(TR), sizeof(TX)};
        bool vec = cols % 8 == 0 && wide(q.n.w, 0, 4) && wide(q.dx, q.lddx, sizeof(TX)) &&
                   wide(q.dr, q.lddr, sizeof(TR));
        for (int k = 0; k < 4; ++k) vec = vec && wide(in[k], ld[k], elem[k]);
        // A warp has 512 columns, a block as many warps as their rings fit; longer rows lie on the
        // blocks of a cluster.
        const int ring = 2 * tg::kLnGradStages * (vec ? tg::LnInput<TX, true>::kBytes + tg::LnInput<TR, true>::kBytes
                                                      : tg::LnInput<TX, false>::kBytes + tg::LnInput<TR, false>::kBytes);
        const int fit = kRingBytes / ring < tg::kLnGradWarps ? kRingBytes / ring : tg::kLnGradWarps;
        int split = 1;
        while (split <= tg::kNormSplit && cols > int64_t{split} * fit * tg::kLnGradCols) split *= 2;
        const bool rows_ring = split <= tg::kNormSplit;
        const int part = split == 1 ? static_cast<int>(cols)
                                    : static_cast<int>((cols + 8 * split - 1) / (8 * split)) * 8;
        const int warps = (part + tg::kLnGradCols - 1) / tg::kLnGradCols;  // of a row
        int groups = 1;
        int64_t most = 2 * dev.num_sms;
        if (rows_ring) {
            const int64_t each = (a->rows + dev.num_sms - 1) / dev.num_sms;
            groups = split > 1 ? 1 : fit / warps < each ? fit / warps : static_cast<int>(each);
            most = dev.num_sms;
            // Two rows of an SM in two blocks, not in two groups of a block, while the second launch has
            // all shares under way at once.  us, groups / blocks, in bf16: 160×1024 5.9 / 4.8, 224×512 4.9 /
            // 4.5, 256×1024 6.3 / 5.2, 256×1536 6.4 / 5.9, 224×2560 6.7 / 6.6, 256×4096 8.2 / 7.9; past
            // that number 257×1024 6.3 / 6.6, 304×1024 6.2 / 7.3, 257×4096 8.2 / 9.3.
            if (groups == 2 && each == 2 && a->rows <= tg::kLnSumShares) groups = 1, most = 2 * dev.num_sms;
        }
        const size_t smem = static_cast<size_t>(ring) * groups * warps;
        if (rows_ring && split > 1) {
            const auto kernel = vec ? tg::tg_layer_norm_grad_rows<TX, TR, true, true>
                                    : tg::tg_layer_norm_grad_rows<TX, TR, false, true>;
            if (!allow_smem(kernel, dev.dev)) return TG_ERR_LAUNCH;
            most = known_clusters(kernel, split, 32 * warps, smem, dev);
            if (most < 1) return TG_ERR_LAUNCH;
        }
        if (most > kGradBlocks) most = kGradBlocks;
        const int64_t wanted = (a->rows + groups - 1) / groups;
        const int64_t blocks = wanted < most ? wanted : most;
        tg::OpWorkspace::Hold hold;  // until the shares' sums are launched
        if (q.dw != nullptr || q.db != nullptr) {
            void* ws = b->workspace;
            if (ws == nullptr) {
                st = g_workspace.get(dev.dev, s, static_cast<size_t>(grad_workspace(a->rows, cols)), &ws, &hold);
                if (st != TG_OK) return st;
            }
            float* next = static_cast<float*>(ws);
            if (q.dw != nullptr) q.ws_w = next, next += blocks * cols;
            if (q.db != nullptr) q.ws_b = next;
        }
        auto run = [&](auto kernel) {
            if (!allow_smem(kernel, dev.dev)) return TG_ERR_LAUNCH;
            return launch(kernel, dim3(static_cast<unsigned>(blocks * split)), 32 * warps * groups, smem, split, s, q,
                          warps, split, part, tg::op_wait_limit_ns(), dev.timeouts,
                          split > 1 ? tg::op_take_inject() : 0);
        };
        if (!rows_ring)
            st = launch(tg::tg_layer_norm_grad_simple<TX, TR>, dim3(static_cast<unsigned>(blocks)), 256, 0, 1, s, q);
        else if (split > 1)
            st = vec ? run(tg::tg_layer_norm_grad_rows<TX, TR, true, true>)
                     : run(tg::tg_layer_norm_grad_rows<TX, TR, false, true>);
        else
            st = vec ? run(tg::tg_layer_norm_grad_rows<TX, TR, true, false>)
                     : run(tg::tg_layer_norm_grad_rows<TX, TR, false, false>);
        if (st != TG_OK || (q.dw == nullptr && q.db == nullptr)) return st;
        // long rows: fewer and wider blocks (50×16384 11.0 us, 13.8 with 32 columns; 500×12001 37.6, 39.4;
        // up to 9000 columns there is no difference)
        auto sum = [&](auto kernel, int columns) {
            return launch(kernel, dim3(static_cast<unsigned>((cols + columns - 1) / columns), 2), 1024, 0, 1, s, q,
                          blocks);
        };
        return cols <= 64 * dev.num_sms ? sum(tg::tg_layer_norm_grad_sum<1>, 32)
                                        : sum(tg::tg_layer_norm_grad_sum<4>, 128);
    });
}

}  // namespace

extern "C" {

tg_status_t tg_layer_norm(const tg_layer_norm_t* a, void* y, int64_t ldy, void* h, int64_t ldh, void* stream) {
    return tg::op_entry([&] { return forward(a, y, ldy, h, ldh, nullptr, false, stream); });
}

tg_status_t tg_layer_norm_i8(const tg_layer_norm_t* a, void* y, int64_t ldy, int8_t* codes, int64_t ldc,
                             float* scale, void* stream) {
    return tg::op_entry([&] { return forward(a, y, ldy, codes, ldc, scale, true, stream); });
}

tg_status_t tg_quantize_rows(int32_t dtype, const void* x, int64_t ldx, int8_t* codes, int64_t ldc, float* scale,
                             int64_t rows, int64_t cols, void* stream) {
    return tg::op_entry([&] { return quantize(dtype, x, ldx, codes, ldc, scale, rows, cols, stream); });
}

int64_t tg_layer_norm_backward_workspace(int64_t rows, int64_t cols) {
    return rows < 0 || cols < 0 || rows > tg::kOpMaxDim || cols > kMaxCols ? -1 : grad_workspace(rows, cols);
}

tg_status_t tg_layer_norm_backward(const tg_layer_norm_t* a, const tg_layer_norm_grad_t* b, void* stream) {
    return tg::op_entry([&] { return backward(a, b, stream); });
}

}  // extern "C"
