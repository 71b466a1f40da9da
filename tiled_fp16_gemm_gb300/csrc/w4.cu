// tg_gemm_w4 (include/tgemm.h): argument checks and launches.  The kernels
// and the formulas: gemm_w4.cuh.
#include <cstring>

#include "gemm_w4.cuh"
#include "op_host.h"

namespace {

using tg::W4Params;

tg::OpWorkspace g_workspace;  // 16-bit weights of the dense path

bool misaligned(const void* p, unsigned bytes) {
    return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0;
}

// Above this many rows of A the weights are decoded to 16 bits once and the
// dense GEMM runs on them.
constexpr int64_t kDenseRows = 64;

template <typename T>
tg_status_t launch_dense(int32_t in_dtype, const W4Params& p, const tg_epilogue_ex_t& x,
                         const tg::OpDevice& dev, cudaStream_t s) {
    const int64_t ldo = (p.N + 7) / 8 * 8;
    void* ws = nullptr;
    tg_status_t st = g_workspace.get(dev.dev, s, static_cast<size_t>(p.K * ldo) * 2, &ws);
    if (st != TG_OK) return st;
    const int64_t tiles = (p.K + 127) / 128 * ((p.N + 63) / 64);
    const int64_t grid = tiles < 8 * dev.num_sms ? tiles : 8 * dev.num_sms;
    tg::tg_w4_dequant<T><<<static_cast<unsigned>(grid), 256, 0, s>>>(p, static_cast<T*>(ws), ldo);
    if (cudaGetLastError() != cudaSuccess) return TG_ERR_LAUNCH;
    return tg_gemm_ex(in_dtype, p.A, ws, p.C, p.M, p.N, p.K, p.lda, ldo, p.ldc, &x, s);
}

template <typename T>
tg_status_t launch_rows(const W4Params& p, const tg::OpDevice& dev, cudaStream_t s) {
    const int64_t jobs = (p.M + 7) / 8 * p.N;
    const int64_t blocks = (jobs + 7) / 8;
    const int64_t grid = blocks < 8 * dev.num_sms ? blocks : 8 * dev.num_sms;
    tg::tg_gemm_w4_simple<T><<<static_cast<unsigned>(grid), 256, 0, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? TG_OK : TG_ERR_LAUNCH;
}

}  // namespace

extern "C" tg_status_t tg_gemm_w4(int32_t in_dtype, const void* A, const void* Bq,
                                  const void* Bscale, const void* Bzero, void* C, int64_t M,
                                  int64_t N, int64_t K, int32_t group, int64_t lda, int64_t ldbq,
                                  int64_t ldbs, int64_t ldbz, int64_t ldc,
                                  const tg_epilogue_ex_t* epi, void* stream) {
    tg_epilogue_ex_t x;
    if (epi != nullptr) {
        x = *epi;
    } else {
        std::memset(&x, 0, sizeof(x));
        x.activation = TG_EPI_NONE;
        x.out_dtype = in_dtype;
    }
    if (in_dtype != TG_DTYPE_F16 && in_dtype != TG_DTYPE_BF16) return TG_ERR_INVALID_VALUE;
    if (x.out_dtype != in_dtype && x.out_dtype != TG_DTYPE_F32) return TG_ERR_INVALID_VALUE;
    if (x.activation != TG_EPI_NONE && x.activation != TG_EPI_RELU) return TG_ERR_INVALID_VALUE;
    if (group != 32 && group != 64 && group != 128) return TG_ERR_INVALID_VALUE;
    if (M < 0 || N < 0 || K < 0 || M > tg::kOpMaxDim || N > tg::kOpMaxDim || K > tg::kOpMaxDim)
        return TG_ERR_INVALID_VALUE;
    if (M == 0 || N == 0) return TG_OK;
    if (C == nullptr || ldc < N || (x.residual != nullptr && x.ldr < N))
        return TG_ERR_INVALID_VALUE;
    if (misaligned(C, x.out_dtype == TG_DTYPE_F32 ? 4 : 2) || misaligned(x.bias, 4) ||
        misaligned(x.residual, 2))
        return TG_ERR_MISALIGNED;
    if (K > 0) {
        if (A == nullptr || Bq == nullptr || Bscale == nullptr || lda < K || ldbq < (K + 1) / 2 ||
            ldbs < N || (Bzero != nullptr && ldbz < N))
            return TG_ERR_INVALID_VALUE;
        if (misaligned(A, 2) || misaligned(Bq, 16) || misaligned(Bscale, 16) ||
            misaligned(Bzero, 16) || ldbq % 16 != 0 || ldbs % 8 != 0 ||
            (Bzero != nullptr && ldbz % 16 != 0))
            return TG_ERR_MISALIGNED;
    }
    tg::OpDevice dev;
    tg_status_t st = tg::op_device(&dev);
    if (st != TG_OK) return st;
    if (K == 0)  // the product is +0: only the epilogue remains
        return tg_gemm_ex(in_dtype, nullptr, nullptr, C, M, N, 0, 0, 0, ldc, &x, stream);
    W4Params p;
    std::memset(&p, 0, sizeof(p));
    p.A = A;
    p.lda = lda;
    p.Bq = static_cast<const uint8_t*>(Bq);
    p.ldbq = ldbq;
    p.scale = Bscale;
    p.lds = ldbs;
    p.zero = static_cast<const uint8_t*>(Bzero);
    p.ldz = ldbz;
    p.C = C;
    p.ldc = ldc;
    p.bias = x.bias;
    p.resid = x.residual;
    p.ldr = x.ldr;
    p.M = M;
    p.N = N;
    p.K = K;
    p.group = group;
    p.relu = x.activation == TG_EPI_RELU ? 1 : 0;
    p.out_f32 = x.out_dtype == TG_DTYPE_F32 ? 1 : 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (M > kDenseRows)
        return in_dtype == TG_DTYPE_BF16 ? launch_dense<__nv_bfloat16>(in_dtype, p, x, dev, s)
                                         : launch_dense<__half>(in_dtype, p, x, dev, s);
    return in_dtype == TG_DTYPE_BF16 ? launch_rows<__nv_bfloat16>(p, dev, s)
                                     : launch_rows<__half>(p, dev, s);
}
