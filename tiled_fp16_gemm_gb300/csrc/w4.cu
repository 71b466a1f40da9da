// tg_gemm_w4 (include/tgemm.h): argument checks and launches.  The kernels
// and the formulas: gemm_w4.cuh.
#include <cstring>
#include <set>

#include "gemm_w4.cuh"
#include "gemm_w4_tc.cuh"
#include "gemm_w4_wide.cuh"
#include "op_host.h"

namespace {

using tg::W4Params;

tg::OpWorkspace g_workspace;  // 16-bit weights of the dense path
// Of tg_gemm_w4_tc and tg_gemm_w4_wide: counters, sums of shares, A in order.  The counters'
// place is the same for every shape: each launch leaves them at zero for the stream's next.
constexpr int64_t kCounterBytes = 64 * 1024;
tg::OpWorkspace g_tc(kCounterBytes);

bool misaligned(const void* p, unsigned bytes) {
    return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0;
}

template <typename T>
tg_status_t launch_dense(int32_t in_dtype, const W4Params& p, const tg_epilogue_ex_t& x,
                         const tg::OpDevice& dev, cudaStream_t s) {
    const int64_t ldo = (p.N + 7) / 8 * 8;
    void* ws = nullptr;
    tg::OpWorkspace::Hold hold;  // until the product is launched
    tg_status_t st = g_workspace.get(dev.dev, s, static_cast<size_t>(p.K * ldo) * 2, &ws, &hold);
    if (st != TG_OK) return st;
    const int64_t tiles = (p.K + 127) / 128 * ((p.N + 63) / 64);
    const int64_t grid = tiles < 8 * dev.num_sms ? tiles : 8 * dev.num_sms;
    tg::tg_w4_dequant<T><<<static_cast<unsigned>(grid), 256, 0, s>>>(p, static_cast<T*>(ws), ldo);
    if (cudaGetLastError() != cudaSuccess) return TG_ERR_LAUNCH;
    return tg_gemm_ex(in_dtype, p.A, ws, p.C, p.M, p.N, p.K, p.lda, ldo, p.ldc, &x, s);
}

// One launch with dependent launch allowed, in clusters of `cluster` blocks.
template <typename... Args, typename... Given>
tg_status_t launch(void (*kernel)(Args...), dim3 grid, int threads, size_t smem, int cluster,
                   cudaStream_t s, Given... given) {
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, kernel, static_cast<Args>(given)...) != cudaSuccess) {
        cudaGetLastError();
        return TG_ERR_LAUNCH;
    }
    return TG_OK;
}

constexpr int kSmem = 226 * 1024;

// Shared memory of a block, or more than there is.
template <int G, int NT>
int64_t w4_smem_bytes(tg::W4Launch* q) {
    using Step = tg::W4Step<G>;
    const int64_t slice = (q->steps + q->cluster - 1) / q->cluster + 1;  // k steps of a block
    const int64_t x = (slice * tg::kW4K * q->tokens * 2 + 511) / 512 * 512;
    const int64_t join = q->wk > 1 ? int64_t{q->wn} * (q->wk - 1) * 1024 * NT : 0;
    const int64_t res = q->cluster > 1 ? int64_t{q->rounds} * q->wn * q->tokens * tg::kW4Rows * 4 : 0;
    for (q->stages = 4; q->stages >= 2; --q->stages) {
        const int64_t all = tg::kW4Warps * 32 + x + tg::kW4Warps * q->stages * int64_t{Step::kBytes} + join + res;
        if (all <= kSmem) {
            q->x_bytes = static_cast<int32_t>(x);
            q->join_bytes = static_cast<int32_t>(join);
            return all;
        }
    }
    return kSmem + 1;
}

// Clusters of `size` blocks that the device holds at once.
template <typename Kernel>
int max_clusters(Kernel kernel, int size, int threads, size_t smem, const tg::OpDevice& dev) {
    if (size == 1) return dev.num_sms;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = static_cast<unsigned>(size);
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3(static_cast<unsigned>(size * (dev.num_sms / size)));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return n;
}

// NT: tokens / 8.
template <typename T, int G, int NT, bool ZERO>
tg_status_t launch_tiles(const W4Params& p, const tg::OpDevice& dev, cudaStream_t s) {
    auto kernel = tg::tg_gemm_w4<T, G, NT, ZERO>;
    struct Limits {
        std::once_flag once;
        bool ok = false;
        int clusters[4] = {};  // of 1, 2, 4, 8 blocks
    };
    static Limits limits[tg::kOpMaxDevices];
    Limits& lim = limits[dev.dev];
    std::call_once(lim.once, [&] {
        lim.ok = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) ==
                 cudaSuccess;
        for (int i = 0; i < 4; ++i) lim.clusters[i] = max_clusters(kernel, 1 << i, tg::kW4Threads, kSmem, dev);
        cudaGetLastError();
    });
    if (!lim.ok) return TG_ERR_LAUNCH;

    tg::W4Launch q, best;
    std::memset(&q, 0, sizeof(q));
    q.p = p;
    q.tokens = static_cast<int32_t>(p.M < 8 * NT ? p.M : 8 * NT);
    int64_t by_m = (p.M + q.tokens - 1) / q.tokens;
    q.steps = static_cast<int32_t>((p.K + tg::kW4K - 1) / tg::kW4K);
    q.tiles = static_cast<int32_t>((p.N + tg::kW4Rows - 1) / tg::kW4Rows);
    // The shape with the least time, in steps of a warp: a block takes rounds of
    // tiles; a round costs its steps and a join, a block the fetch of A and, with a
    // cluster, the last join.
    double least = 1e300;
    int64_t smem = 0;
    for (; q.tokens >= 1 && least > 1e299; q.tokens /= 2) {  // k too long for so many tokens: fewer
        by_m = (p.M + q.tokens - 1) / q.tokens;
        for (int i = 0; i < 4; ++i) {
            q.cluster = 1 << i;
            if (q.cluster > q.steps) break;
            if (lim.clusters[i] < 1) continue;
            for (q.wk = 1; q.wk <= 16; q.wk *= 2) {
                q.wn = tg::kW4Warps / q.wk;
                const int64_t jobs = (q.tiles + q.wn - 1) / q.wn;
                int64_t clusters = lim.clusters[i];
                if (clusters > jobs) clusters = jobs;
                q.rounds = static_cast<int32_t>((jobs + clusters - 1) / clusters);
                q.clusters = static_cast<int32_t>((jobs + q.rounds - 1) / q.rounds);
                const int64_t bytes = w4_smem_bytes<G, NT>(&q);
                if (bytes > kSmem) continue;
                const int64_t slice = (q.steps + q.cluster - 1) / q.cluster;
                const int64_t each = (slice + q.wk - 1) / q.wk;
                const double waves = static_cast<double>(
                    (q.clusters * by_m + lim.clusters[i] - 1) / lim.clusters[i]);
                const double time =
                    waves * (q.rounds * (each + (q.wk > 1 ? 0.5 + 0.1 * q.wk * NT : 0.3)) +
                             0.01 * slice * q.tokens + (q.cluster > 1 ? 3.0 : 0.0) +
                             (q.stages < 4 ? 2.0 * (4 - q.stages) : 0.0));
                if (time < least) least = time, best = q, smem = bytes;
            }
        }
    }
    if (least > 1e299) {
        const int64_t blocks = ((p.M + 7) / 8 * p.N + 7) / 8;
        const int64_t most = 8 * dev.num_sms;
        return launch(tg::tg_gemm_w4_simple<T>,
                      dim3(static_cast<unsigned>(blocks < most ? blocks : most)), 256, 0, 1, s, p);
    }
    by_m = (p.M + best.tokens - 1) / best.tokens;
    best.limit_ns = tg::op_wait_limit_ns();
    best.timeouts = dev.timeouts;
    best.inject = tg::op_take_inject();
    using Step = tg::W4Step<G>;
    constexpr CUtensorMapDataType type =
        std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const uint64_t groups = (p.K + G - 1) / G;
    CUtensorMap codes, scales, zeros;
    if (!tg::op_map_2d(&codes, p.Bq, CU_TENSOR_MAP_DATA_TYPE_UINT8, (p.K + 1) / 2, p.N, p.ldbq,
                       tg::kW4K / 2, tg::kW4Rows, CU_TENSOR_MAP_SWIZZLE_64B) ||
        !tg::op_map_2d(&scales, p.scale, type, p.N, groups, p.lds * 2, tg::kW4Rows, Step::kGroups,
                       CU_TENSOR_MAP_SWIZZLE_NONE))
        return TG_ERR_LAUNCH;
    zeros = scales;
    if (ZERO && !tg::op_map_2d(&zeros, p.zero, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.N, groups, p.ldz,
                               tg::kW4Rows, Step::kGroups, CU_TENSOR_MAP_SWIZZLE_NONE))
        return TG_ERR_LAUNCH;
    return launch(kernel,
                  dim3(static_cast<unsigned>(best.clusters * best.cluster), static_cast<unsigned>(by_m)),
                  tg::kW4Threads, static_cast<size_t>(smem), best.cluster, s, best, codes, scales, zeros);
}

// Opts a kernel into its shared memory, once per device.
template <typename Kernel>
bool allow_smem(Kernel kernel, int bytes, int dev) {
    static std::mutex m;
    static std::set<std::pair<const void*, int>> done;
    const auto key = std::make_pair(reinterpret_cast<const void*>(kernel), dev);
    std::lock_guard<std::mutex> lk(m);
    if (done.count(key) != 0) return true;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    done.insert(key);
    return true;
}

// Up to 64 rows of A, on tcgen05.
template <typename T, int G, int NP, bool ZERO>
tg_status_t launch_tc(const W4Params& p, const tg::OpDevice& dev, cudaStream_t s) {
    using S = tg::TcShape<G, NP>;
    auto kernel = tg::tg_gemm_w4_tc<T, G, NP, ZERO>;
    if (!allow_smem(kernel, S::kSmem, dev.dev)) return TG_ERR_LAUNCH;
    tg::TcLaunch q;
    q.p = p;
    q.limit_ns = tg::op_wait_limit_ns();
    q.timeouts = dev.timeouts;
    q.inject = 0;
    q.k_units = static_cast<int32_t>((p.K + tg::kTcK - 1) / tg::kTcK);
    q.units = (p.N + tg::kTcRows - 1) / tg::kTcRows * q.k_units;
    const int64_t blocks = q.units < dev.num_sms ? q.units : dev.num_sms;
    if (blocks * 32 > kCounterBytes) return TG_ERR_UNSUPPORTED_DEVICE;
    const int64_t slot_bytes = 2 * blocks * NP * tg::kTcRows * 4;
    const int64_t ldo = int64_t{q.k_units} * tg::kTcK;
    void* ws = nullptr;
    tg::OpWorkspace::Hold hold;  // until the product is launched
    tg_status_t st = g_tc.get(dev.dev, s, static_cast<size_t>(kCounterBytes + slot_bytes + p.M * ldo * 2),
                              &ws, &hold);
    if (st != TG_OK) return st;
    q.counters = static_cast<uint32_t*>(ws);
    q.slots = reinterpret_cast<float*>(static_cast<char*>(ws) + kCounterBytes);
    uint16_t* order = reinterpret_cast<uint16_t*>(static_cast<char*>(ws) + kCounterBytes + slot_bytes);
    constexpr CUtensorMapDataType type =
        std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const uint64_t groups = (p.K + G - 1) / G;
    CUtensorMap codes, scales, zeros, ordered;
    if (!tg::op_map_2d(&codes, p.Bq, CU_TENSOR_MAP_DATA_TYPE_UINT8, (p.K + 1) / 2, p.N, p.ldbq,
                       tg::kTcK / 2, tg::kTcRows, CU_TENSOR_MAP_SWIZZLE_64B) ||
        !tg::op_map_2d(&scales, p.scale, type, p.N, groups, p.lds * 2, tg::kTcRows, S::kGroups,
                       CU_TENSOR_MAP_SWIZZLE_NONE) ||
        !tg::op_map_2d(&ordered, order, type, ldo, p.M, ldo * 2, 64, NP, CU_TENSOR_MAP_SWIZZLE_128B))
        return TG_ERR_LAUNCH;
    zeros = scales;
    if (ZERO && !tg::op_map_2d(&zeros, p.zero, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.N, groups, p.ldz,
                               tg::kTcRows, S::kGroups, CU_TENSOR_MAP_SWIZZLE_NONE))
        return TG_ERR_LAUNCH;
    q.inject = tg::op_take_inject();
    st = launch(tg::tg_w4_order,
                dim3(static_cast<unsigned>((ldo / 8 + 255) / 256), static_cast<unsigned>(p.M)), 256, 0, 1, s,
                static_cast<const uint16_t*>(p.A), p.lda, p.M, p.K, order, ldo);
    if (st != TG_OK) return st;
    return launch(kernel, dim3(static_cast<unsigned>(blocks)), S::kThreads, S::kSmem, 1, s, q, codes,
                  scales, zeros, ordered);
}

// Fills in the tile's width and the division of the work with the least time, and returns
// that time in us.  Measured: a unit takes 2.4 ns per token, and 0.43 us at least (what the
// codes take to come and be decoded); a tile that is shared 4 us + 18 ns per token and share
// more; A in order 4 bytes an element at 4 TB/s.  16384×8192 with 65 / 128 / 192 / 256 / 512
// rows: 34 / 35 / 38 / 47 / 87 us, on 64 of 76 pairs, with whole tiles.
double plan_wide(const W4Params& p, int64_t limit, tg::WideLaunch* q) {
    q->k_units = static_cast<int32_t>((p.K + tg::kTcK - 1) / tg::kTcK);
    constexpr int64_t rows = int64_t{tg::kTcRows} * tg::kWideCluster;
    const int64_t row_tiles = (p.N + rows - 1) / rows;
    double least = 1e300;
    for (int32_t tokens = 32; tokens <= tg::kWideTokens; tokens += 32) {
        const int64_t m_tiles = (p.M + tokens - 1) / tokens, tiles = row_tiles * m_tiles;
        const double mma = 0.0024 * tokens * (p.out_f32 ? 2 : 1);
        const double unit = mma < 0.43 ? 0.43 : mma;
        for (const int32_t grain : {q->k_units, 1}) {
            const int64_t grains = tiles * q->k_units / grain;
            const int64_t clusters = grains < limit ? grains : limit;
            const int64_t most = (grains + clusters - 1) / clusters * grain;
            double time = unit * static_cast<double>(most);
            if (grain != q->k_units && (most % q->k_units != 0 || grains % clusters != 0))
                time += 4.0 + 0.018 * tokens * (2.0 + static_cast<double>(q->k_units) / static_cast<double>(most));
            if (time < least) {
                least = time;
                q->tokens = tokens;
                q->m_tiles = static_cast<int32_t>(m_tiles);
                q->grain = grain;
                q->clusters = static_cast<int32_t>(clusters);
                q->units = tiles * q->k_units;
            }
        }
    }
    return 5.5 + least + 1e-6 * static_cast<double>(p.M) * static_cast<double>(p.K);
}

// Many rows of A, on tcgen05.
template <typename T, int G, bool ZERO, bool EXACT>
tg_status_t launch_wide(const W4Params& p, const tg::OpDevice& dev, cudaStream_t s) {
    auto kernel = tg::tg_gemm_w4_wide<T, G, ZERO, EXACT>;
    struct Limits {
        std::once_flag once;
        int clusters = 0;
    };
    static Limits limits[tg::kOpMaxDevices];
    Limits& lim = limits[dev.dev];
    std::call_once(lim.once, [&] {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, tg::kWideSmem) ==
            cudaSuccess)
            lim.clusters = max_clusters(kernel, tg::kWideCluster, tg::kWideThreads, tg::kWideSmem, dev);
        cudaGetLastError();
    });
    if (lim.clusters < 1) return TG_ERR_LAUNCH;
    tg::WideLaunch q;
    std::memset(&q, 0, sizeof(q));
    q.p = p;
    q.limit_ns = tg::op_wait_limit_ns();
    q.timeouts = dev.timeouts;
    plan_wide(p, lim.clusters, &q);
    const int64_t blocks = int64_t{q.clusters} * tg::kWideCluster;
    if (blocks * 32 > kCounterBytes) return TG_ERR_UNSUPPORTED_DEVICE;
    const int64_t slot_bytes = 2 * blocks * q.tokens * tg::kTcRows * 4;
    const int64_t ldo = int64_t{q.k_units} * tg::kTcK;
    void* ws = nullptr;
    tg::OpWorkspace::Hold hold;  // until the product is launched
    tg_status_t st = g_tc.get(dev.dev, s, static_cast<size_t>(kCounterBytes + slot_bytes + p.M * ldo * 2),
                              &ws, &hold);
    if (st != TG_OK) return st;
    q.counters = static_cast<uint32_t*>(ws);
    q.slots = reinterpret_cast<float*>(static_cast<char*>(ws) + kCounterBytes);
    uint16_t* order = reinterpret_cast<uint16_t*>(static_cast<char*>(ws) + kCounterBytes + slot_bytes);
    constexpr CUtensorMapDataType type =
        std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const uint64_t groups = (p.K + G - 1) / G;
    constexpr uint32_t unit_groups = tg::kTcK / G;
    CUtensorMap codes, scales, zeros, ordered;
    if (!tg::op_map_2d(&codes, p.Bq, CU_TENSOR_MAP_DATA_TYPE_UINT8, (p.K + 1) / 2, p.N, p.ldbq,
                       tg::kTcK / 2, tg::kTcRows, CU_TENSOR_MAP_SWIZZLE_64B) ||
        !tg::op_map_2d(&scales, p.scale, type, p.N, groups, p.lds * 2, tg::kTcRows, unit_groups,
                       CU_TENSOR_MAP_SWIZZLE_NONE) ||
        !tg::op_map_2d(&ordered, order, type, ldo, p.M, ldo * 2, 64,
                       static_cast<uint32_t>(q.tokens / tg::kWideCluster), CU_TENSOR_MAP_SWIZZLE_128B))
        return TG_ERR_LAUNCH;
    zeros = scales;
    if (ZERO && !tg::op_map_2d(&zeros, p.zero, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.N, groups, p.ldz,
                               tg::kTcRows, unit_groups, CU_TENSOR_MAP_SWIZZLE_NONE))
        return TG_ERR_LAUNCH;
    q.inject = tg::op_take_inject();
    st = launch(tg::tg_w4_order,
                dim3(static_cast<unsigned>((ldo / 8 + 255) / 256),
                     static_cast<unsigned>(p.M < 32768 ? p.M : 32768)),
                256, 0, 1, s, static_cast<const uint16_t*>(p.A), p.lda, p.M, p.K, order, ldo);
    if (st != TG_OK) return st;
    return launch(kernel, dim3(static_cast<unsigned>(blocks)), tg::kWideThreads, tg::kWideSmem,
                  tg::kWideCluster, s, q, codes, scales, zeros, ordered);
}

// Whether the tcgen05 kernel is the faster one.  With B MB of codes it took about 7 us +
// 0.3·B (up to 32 rows; 0.5·B up to 64), the other 3 us + 0.53·B for every 16 rows
// (16384×8192, B = 67, 16 / 32 / 64 rows: 29 / 33 / 42 us against 35 / 67 / 123).
bool prefer_tc(const W4Params& p) {
    if (p.M <= 8) return false;
    const double mb = static_cast<double>(p.N) * static_cast<double>(p.K) / 2e6;
    return 7.0 + (p.M <= 32 ? 0.3 : 0.5) * mb < 3.0 + 0.53 * static_cast<double>((p.M + 15) / 16) * mb;
}

// Up to 64 rows no weight is rounded, and the kernels are those that need not.  (64 is not where
// the times cross: the pair kernel without rounding takes 65 rows of 16384×8192 in 41 us with
// G = 128 and 45 with G = 32, tg_gemm_w4_tc 64 rows in 41 and 52.)
template <typename T, int G, bool ZERO>
tg_status_t launch_group(const W4Params& p, const tg::OpDevice& dev, cudaStream_t s) {
    if (p.M > 64)
        return p.out_f32 ? launch_wide<T, G, ZERO, true>(p, dev, s)
                         : launch_wide<T, G, ZERO, false>(p, dev, s);
    if (prefer_tc(p)) {
        if (p.M <= 16) return launch_tc<T, G, 16, ZERO>(p, dev, s);
        if (p.M <= 32) return launch_tc<T, G, 32, ZERO>(p, dev, s);
        return launch_tc<T, G, 64, ZERO>(p, dev, s);
    }
    if (p.M <= 8) return launch_tiles<T, G, 1, ZERO>(p, dev, s);
    return launch_tiles<T, G, 2, ZERO>(p, dev, s);
}

template <typename T, int G>
tg_status_t launch_zero(const W4Params& p, const tg::OpDevice& dev, cudaStream_t s) {
    return p.zero != nullptr ? launch_group<T, G, true>(p, dev, s)
                             : launch_group<T, G, false>(p, dev, s);
}

// Very many rows, a 16-bit result: whether the weights are decoded to T in memory and the
// dense GEMM runs on them.  With B MB of codes that takes about 10 us + 1.5·B and the GEMM at
// 1800 TFLOP/s; tg_gemm_w4_wide decodes every weight once for 256 rows, which costs it a tenth
// of that rate.  Measured, dense / wide: 16384×8192 with 2048 / 4096 / 6000 / 8192 rows
// 437 / 791 / 1156 / 1508 us against 386 / 801 / 1208 / 1653, 512×4096 with 3000 22.5 us against
// 25.2, 1024×1024 with 6000 17.0 against 21.3.  Below 2048 rows the model does not hold for the
// dense GEMM of small weights (512×2048 with 100 rows 30 us against 11).
bool prefer_dense(const W4Params& p, const tg::OpDevice& dev) {
    if (p.M < 2048) return false;
    tg::WideLaunch q;
    const double nk = static_cast<double>(p.N) * static_cast<double>(p.K);
    const double flops = 2.0 * nk * static_cast<double>(p.M);
    const double wide = plan_wide(p, dev.num_sms / tg::kWideCluster, &q);
    return 10.0 + 1.5 * nk / 2e6 + flops / 1800e6 < (wide > flops / 1600e6 ? wide : flops / 1600e6);
}

template <typename T>
tg_status_t launch_rows(int32_t in_dtype, const W4Params& p, const tg_epilogue_ex_t& x,
                        const tg::OpDevice& dev, cudaStream_t s) {
    if (!p.out_f32 && prefer_dense(p, dev)) return launch_dense<T>(in_dtype, p, x, dev, s);
    if (p.group == 32) return launch_zero<T, 32>(p, dev, s);
    if (p.group == 64) return launch_zero<T, 64>(p, dev, s);
    return launch_zero<T, 128>(p, dev, s);
}

}  // namespace

void tg::w4_clear_counters(int dev) { g_tc.clear(dev); }

static tg_status_t gemm_w4(int32_t in_dtype, const void* A, const void* Bq, const void* Bscale,
                           const void* Bzero, void* C, int64_t M, int64_t N, int64_t K,
                           int32_t group, int64_t lda, int64_t ldbq, int64_t ldbs, int64_t ldbz,
                           int64_t ldc, const tg_epilogue_ex_t* epi, void* stream) {
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
    return in_dtype == TG_DTYPE_BF16 ? launch_rows<__nv_bfloat16>(in_dtype, p, x, dev, s)
                                     : launch_rows<__half>(in_dtype, p, x, dev, s);
}

extern "C" tg_status_t tg_gemm_w4(int32_t in_dtype, const void* A, const void* Bq,
                                  const void* Bscale, const void* Bzero, void* C, int64_t M,
                                  int64_t N, int64_t K, int32_t group, int64_t lda, int64_t ldbq,
                                  int64_t ldbs, int64_t ldbz, int64_t ldc,
                                  const tg_epilogue_ex_t* epi, void* stream) {
    return tg::op_entry([&] {
        return gemm_w4(in_dtype, A, Bq, Bscale, Bzero, C, M, N, K, group, lda, ldbq, ldbs, ldbz, ldc, epi,
                       stream);
    });
}
