// tg_gemm_i8 (include/tgemm.h): argument checks and launches.  The kernels and the
// formulas: gemm_i8.cuh.
#include <cstring>

#include "gemm_i8.cuh"
#include "op_host.h"

namespace {

using tg::I8Params;

constexpr int64_t kMaxK = 131071;  // 2^17 - 1: a sum of K products of -128 · -128 fits 32 bits

bool misaligned(const void* p, unsigned bytes) {
    return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0;
}

// One launch with dependent launch allowed.
template <typename... Args, typename... Given>
tg_status_t launch(void (*kernel)(Args...), dim3 grid, int threads, size_t smem, cudaStream_t s,
                   Given... given) {
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, static_cast<Args>(given)...) != cudaSuccess) {
        cudaGetLastError();
        return TG_ERR_LAUNCH;
    }
    return TG_OK;
}

template <typename TC>
tg_status_t launch_type(const I8Params& p, const tg::OpDevice& dev, cudaStream_t s) {
    const int64_t blocks = (p.M * p.N + 7) / 8, most = 8 * int64_t{dev.num_sms};
    return launch(tg::tg_gemm_i8_simple<TC>, dim3(static_cast<unsigned>(blocks < most ? blocks : most)), 256, 0, s,
                  p);
}

int64_t workspace_bytes(int64_t M, int64_t N, int64_t K) { return 0 * M * N * K; }

tg_status_t gemm_i8(const int8_t* A, int64_t lda, const float* sa, const int8_t* B, int64_t ldb,
                    const float* sb, void* C, int64_t ldc, int64_t M, int64_t N, int64_t K,
                    const tg_epilogue_ex_t* epi, void* workspace, int64_t bytes, void* stream) {
    tg_epilogue_ex_t x;
    std::memset(&x, 0, sizeof(x));
    x.activation = TG_EPI_NONE;
    x.out_dtype = TG_DTYPE_F16;
    if (epi != nullptr) x = *epi;
    if (x.out_dtype != TG_DTYPE_F16 && x.out_dtype != TG_DTYPE_BF16 && x.out_dtype != TG_DTYPE_F32)
        return TG_ERR_INVALID_VALUE;
    if (x.activation != TG_EPI_NONE && x.activation != TG_EPI_RELU) return TG_ERR_INVALID_VALUE;
    if (M < 0 || N < 0 || K < 0 || M > tg::kOpMaxDim || N > tg::kOpMaxDim || K > kMaxK)
        return TG_ERR_INVALID_VALUE;
    if (M == 0 || N == 0) return TG_OK;
    if (C == nullptr || ldc < N || (x.residual != nullptr && x.ldr < N)) return TG_ERR_INVALID_VALUE;
    const unsigned out = x.out_dtype == TG_DTYPE_F32 ? 4 : 2;
    if (misaligned(C, out) || misaligned(x.bias, 4) || misaligned(x.residual, out) || misaligned(workspace, 256))
        return TG_ERR_MISALIGNED;
    if (sa == nullptr || sb == nullptr) return TG_ERR_INVALID_VALUE;
    if (misaligned(sa, 4) || misaligned(sb, 4)) return TG_ERR_MISALIGNED;
    if (K > 0) {
        if (A == nullptr || B == nullptr || lda < K || ldb < K) return TG_ERR_INVALID_VALUE;
        if (misaligned(B, 16) || ldb % 16 != 0) return TG_ERR_MISALIGNED;
    }
    if (workspace != nullptr && bytes < workspace_bytes(M, N, K)) return TG_ERR_INVALID_VALUE;
    tg::OpDevice dev;
    tg_status_t st = tg::op_device(&dev);
    if (st != TG_OK) return st;
    I8Params p;
    std::memset(&p, 0, sizeof(p));
    p.A = A;
    p.lda = lda;
    p.sa = sa;
    p.B = B;
    p.ldb = ldb;
    p.sb = sb;
    p.C = C;
    p.ldc = ldc;
    p.bias = x.bias;
    p.resid = x.residual;
    p.ldr = x.ldr;
    p.M = M;
    p.N = N;
    p.K = K;
    p.relu = x.activation == TG_EPI_RELU ? 1 : 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (x.out_dtype == TG_DTYPE_F32) return launch_type<float>(p, dev, s);
    return x.out_dtype == TG_DTYPE_F16 ? launch_type<__half>(p, dev, s) : launch_type<__nv_bfloat16>(p, dev, s);
}

}  // namespace

extern "C" {

int64_t tg_gemm_i8_workspace(int64_t M, int64_t N, int64_t K) {
    return M < 0 || N < 0 || K < 0 || M > tg::kOpMaxDim || N > tg::kOpMaxDim || K > kMaxK ? -1
                                                                                          : workspace_bytes(M, N, K);
}

tg_status_t tg_gemm_i8(const int8_t* A, int64_t lda, const float* Ascale, const int8_t* B, int64_t ldb,
                       const float* Bscale, void* C, int64_t ldc, int64_t M, int64_t N, int64_t K,
                       const tg_epilogue_ex_t* epi, void* workspace, int64_t workspace_bytes, void* stream) {
    return tg::op_entry([&] {
        return gemm_i8(A, lda, Ascale, B, ldb, Bscale, C, ldc, M, N, K, epi, workspace, workspace_bytes, stream);
    });
}

}  // extern "C"
