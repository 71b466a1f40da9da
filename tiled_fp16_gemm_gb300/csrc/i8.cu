// tg_gemm_i8 (include/tgemm.h): argument checks and launches.  The kernels and the
// formulas: gemm_i8.cuh and gemm_i8_wide.cuh.
#include <cstring>

#include "gemm_i8.cuh"
#include "gemm_i8_wide.cuh"
#include "launch_host.h"

namespace {

using tg::I8Params;
using tg::launch;
using tg::max_clusters;
using tg::misaligned;

constexpr int64_t kMaxK = 131071;  // 2^17 - 1: a sum of K products of -128 · -128 fits 32 bits

constexpr int kSmem = 226 * 1024;

// What a device holds of a kernel that uses clusters, asked once.
struct Limits {
    std::once_flag once;
    int clusters[4] = {};  // of 1, 2, 4, 8 blocks; 0: the kernel cannot run
};
template <typename Kernel>
const Limits& limits_of(Kernel kernel, int threads, int smem, const tg::OpDevice& dev, Limits* all) {
    Limits& lim = all[dev.dev];
    std::call_once(lim.once, [&] {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) == cudaSuccess)
            for (int i = 0; i < 4; ++i) lim.clusters[i] = max_clusters(kernel, 1 << i, threads, smem, dev);
        cudaGetLastError();
    });
    return lim;
}

int64_t chunks_of(int64_t K) { return (K + tg::kI8FewK - 1) / tg::kI8FewK; }

// What a block of the kernel for few rows has in shared memory.
struct FewRoom {
    int64_t x_pitch;  // bytes of a token
    int64_t fixed;    // bytes besides the sums
    int64_t tiles;    // whose sums fit besides
};
FewRoom few_room(int64_t M, int64_t K, int cluster, int stages) {
    FewRoom r;
    const int64_t slice = (chunks_of(K) + cluster - 1) / cluster;
    r.x_pitch = slice * tg::kI8FewK * (M > 8 ? 2 : 1) + 64;
    r.fixed = 1024 + int64_t{tg::kI8FewWarps} * stages * tg::kI8FewStep + tg::kI8FewBars + M * r.x_pitch;
    const int64_t room = kSmem - r.fixed - M * 16;
    r.tiles = room < 0 ? 0 : room / (M * tg::kI8FewRows * 4);
    return r;
}
// Whether a block, of a cluster of eight at most, has room for them.
bool few_fits(int64_t M, int64_t K) {
    for (int cluster = 1; cluster <= 8 && cluster <= chunks_of(K); cluster *= 2)
        if (few_room(M, K, cluster, 2).tiles >= 1) return true;
    return false;
}

// Few rows of A (NT: tokens / 8).
struct FewPlan {
    tg::I8Few q;
    size_t smem;
    int64_t grid;
    double time;  // us; 1e300: no shape fits
};

// The shape with the least time.  A round of a block's warps is 16 steps, 32 KB of B: 0.73 us of
// memory, or what the tensor pipe or shared memory takes (measured, 16384×8192: see below); then
// the fetch of the block's part of A, the joins of a cluster, a shallow ring.
template <typename TC, int NT>
FewPlan plan_few(const I8Params& p, const tg::OpDevice& dev) {
    auto kernel = tg::tg_gemm_i8_few<TC, NT>;
    static Limits limits[tg::kOpMaxDevices];
    const Limits& lim = limits_of(kernel, tg::kI8FewThreads, kSmem, dev, limits);
    FewPlan best;
    best.time = 1e300;
    tg::I8Few q;
    std::memset(&q, 0, sizeof(q));
    q.p = p;
    const int64_t tiles = (p.N + tg::kI8FewRows - 1) / tg::kI8FewRows;
    q.tiles = static_cast<int32_t>(tiles);
    q.chunks = static_cast<int32_t>(chunks_of(p.K));
    constexpr double round = NT <= 2 ? 0.73 : NT == 4 ? 0.8 : 1.4;
    for (int i = 0; i < 4; ++i) {
        q.cluster = 1 << i;
        if (q.cluster > q.chunks || lim.clusters[i] < 1) break;
        const int64_t slice = (q.chunks + q.cluster - 1) / q.cluster;
        int64_t clusters = tiles < lim.clusters[i] ? tiles : lim.clusters[i];
        // (with few steps a shallow ring: then the next call's blocks find room beside this one's, and
        // B comes to L2 meanwhile; one row of 4096×4096 5.4 us, with three stages 6.0)
        const int64_t each = ((tiles + clusters - 1) / clusters * slice + tg::kI8FewWarps - 1) / tg::kI8FewWarps;
        for (q.stages = each <= 6 ? 2 : tg::kI8FewStages; q.stages >= 2; --q.stages) {
            const FewRoom of_block = few_room(p.M, p.K, q.cluster, q.stages);
            q.x_pitch = static_cast<int32_t>(of_block.x_pitch);
            // (a block keeps the sums of its tiles: very many rows of B take several waves)
            const int64_t room = of_block.tiles;
            int64_t rounds = (tiles + clusters - 1) / clusters;
            if (room < 1 || (room < rounds && q.stages > 2)) continue;
            if (rounds > room) {
                rounds = room;
                clusters = (tiles + rounds - 1) / rounds;
            }
            q.sums_pitch = static_cast<int32_t>(rounds * tg::kI8FewRows + 4);
            const int64_t waves = (clusters + lim.clusters[i] - 1) / lim.clusters[i];
            const double steps = static_cast<double>((rounds * slice + tg::kI8FewWarps - 1) / tg::kI8FewWarps);
            const double time =
                2.0 + static_cast<double>(waves) * (round * steps + 8e-6 * static_cast<double>(slice * tg::kI8FewK * p.M) +
                                                    (q.cluster > 1 ? 1.1 : 0.0) + (q.stages < 3 && each > 6 ? 1.5 : 0.0));
            if (time < best.time && clusters * q.cluster <= tg::kOpMaxDim) {
                best.time = time;
                best.q = q;
                best.smem = static_cast<size_t>(of_block.fixed + 4 * p.M * q.sums_pitch);
                best.grid = clusters * q.cluster;
            }
            break;
        }
    }
    return best;
}

template <typename TC, int NT>
tg_status_t launch_few(FewPlan& plan, const tg::OpDevice& dev, cudaStream_t s) {
    const I8Params& p = plan.q.p;
    CUtensorMap codes;
    if (!tg::op_map_2d(&codes, p.B, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.K, p.N, p.ldb, tg::kI8FewK, tg::kI8FewRows,
                       CU_TENSOR_MAP_SWIZZLE_128B))
        return TG_ERR_LAUNCH;
    plan.q.limit_ns = tg::op_wait_limit_ns();
    plan.q.timeouts = dev.timeouts;
    plan.q.inject = tg::op_take_inject();
    return launch(tg::tg_gemm_i8_few<TC, NT>, dim3(static_cast<unsigned>(plan.grid)), tg::kI8FewThreads, plan.smem,
                  plan.q.cluster, s, plan.q, codes);
}

// ------------------------------------------------------------------ many rows

tg::OpWorkspace g_workspace;  // where the caller has none

// Rows of A at a time: fp16 rows of A take 1 GB at most.
int64_t slab_rows(int64_t M, int64_t K) {
    const int64_t ldo = (K + tg::kTcK - 1) / tg::kTcK * tg::kTcK;
    const int64_t rows = (int64_t{1} << 29) / ldo / tg::kI8Tokens * tg::kI8Tokens;
    return M < rows ? M : rows;
}
int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }
// Of a tile, at most: what the shares' places are made for.
int64_t tile_tokens(int64_t M) { return M < tg::kI8Tokens ? up(M, 32) : tg::kI8Tokens; }

// Fills in the tile's width and the division of the work with the least time.  Measured, on random
// codes: a unit takes 2.4 ns per token, and 0.4 us at least (what B takes to be decoded; to come, 6 ns
// per cluster); the end of a tile 8 ns per token; the sums of a shared tile 2.5 us + 25 ns per token,
// twice as much per token where a cluster has two of them.  Whole tiles / even runs / equal parts,
// us: 2048×8192 with 64 rows 28.6 / 14.9 / 13.8, 4096×8192 with 128 30.3 / 21.4 / 20.3, 4096×28672
// with 128 86 / 36.0 / 37.0, 5120×2048 with 64 12.3 / 13.8 / -, 16384×8192 with 64 32.0 / 36.0 / -.
void plan_wide(const I8Params& p, int64_t limit, tg::I8Wide* q) {
    const int32_t k_units = static_cast<int32_t>((p.K + tg::kTcK - 1) / tg::kTcK);
    constexpr int64_t rows = int64_t{tg::kTcRows} * tg::kWideCluster;
    const int64_t row_tiles = (p.N + rows - 1) / rows;
    q->k_units = k_units;
    double least = 1e300;
    const int32_t widest = static_cast<int32_t>(tile_tokens(p.M));
    for (int32_t tokens = 32; tokens <= widest; tokens += 32) {
        const int64_t m_tiles = (p.M + tokens - 1) / tokens, tiles = row_tiles * m_tiles;
        const double mma = 0.0024 * tokens, decoded = mma < 0.4 ? 0.4 : mma;
        auto offer = [&](int32_t parts, int32_t grain, int64_t clusters, int64_t most, double sums) {
            const double memory = 0.006 * static_cast<double>(clusters);
            const double time = (memory < decoded ? decoded : memory) * static_cast<double>(most) +
                                0.008 * tokens * static_cast<double>((most + k_units - 1) / k_units) + sums;
            if (time >= least) return;
            least = time;
            q->tokens = tokens;
            q->m_tiles = static_cast<int32_t>(m_tiles);
            q->parts = parts;
            q->grain = grain;
            q->clusters = static_cast<int32_t>(clusters);
            q->units = tiles * k_units;
        };
        const int64_t whole = tiles < limit ? tiles : limit;
        offer(0, k_units, whole, (tiles + whole - 1) / whole * k_units, 0.0);
        const int64_t units = tiles * k_units, even = units < limit ? units : limit;
        offer(0, 1, even, (units + even - 1) / even, 2.5 + 0.05 * tokens);
        const int64_t each = limit / tiles, parts = each < k_units ? each : k_units;
        if (parts > 1)
            offer(static_cast<int32_t>(parts), 1, tiles * parts, (k_units + parts - 1) / parts, 2.5 + 0.025 * tokens);
    }
}

// Counters and peaks, the tiles' sums (those of shared ones, and where the accumulator may not take all of K
// also of each cluster's own), A as fp16: for any plan of these sizes.
bool more_runs(int64_t K) { return K > int64_t{tg::kI8WideRun} * tg::kTcK; }
int64_t slot_bytes(int64_t M, int64_t K) {
    return int64_t{tg::kI8MaxClusters} * tg::kWideCluster * tile_tokens(M) * tg::kTcRows * 4 * (more_runs(K) ? 2 : 1);
}
constexpr int64_t kHeadBytes = tg::kI8CounterBytes + tg::kI8PeakBytes;
int64_t wide_bytes(int64_t M, int64_t K) {
    return kHeadBytes + slot_bytes(M, K) + slab_rows(M, K) * up(K, tg::kTcK) * 2;
}

// Whether the kernel for few rows is the faster one: up to 16 rows always, more of them with small
// weights.  Measured, us, few / wide: 16384×8192 with 16 rows 28.7 / 30.9, 32 rows 48 / 31;
// 4096×28672 with 16 rows 29.8 / 31.2; 9728×2560 with 32 rows 13.6 / 13.8, 9728×4096 18.0 / 17.4;
// 4096×1024 with 48 rows 8.6 / 9.1, 64 rows 11.6 / 9.2; 2560×2560 with 48 rows 10.8 / 10.8;
// 1024×1024 with 64 rows 9.0 / 9.0.
bool prefer_few(int64_t M, int64_t N, int64_t K) {
    const int64_t codes = N * K;
    return M <= 16 || (M <= 32 && codes <= 30000000) || (M <= 48 && codes <= 5000000) ||
           (M <= 64 && codes <= 1000000);
}
// None for the kernel for few rows.  (On a device that holds none of its clusters the other takes the
// library's buffer.)
int64_t workspace_bytes(int64_t M, int64_t N, int64_t K) {
    return M <= 8 || K == 0 || (prefer_few(M, N, K) && few_fits(M, K)) ? 0 : wide_bytes(M, K);
}

template <typename TC>
tg_status_t launch_wide(const I8Params& whole, const tg::OpDevice& dev, void* ws, cudaStream_t s) {
    auto kernel = tg::tg_gemm_i8_wide<TC>;
    static Limits limits[tg::kOpMaxDevices];
    const Limits& lim = limits_of(kernel, tg::kWideThreads, tg::kI8WideSmem, dev, limits);
    if (lim.clusters[1] < 1) return TG_ERR_LAUNCH;
    tg::OpWorkspace::Hold hold;  // until the last product is launched
    if (ws == nullptr) {
        const tg_status_t st = g_workspace.get(
            dev.dev, s, static_cast<size_t>(wide_bytes(whole.M, whole.K)), &ws, &hold);
        if (st != TG_OK) return st;
    }
    tg::I8Wide q;
    std::memset(&q, 0, sizeof(q));
    q.limit_ns = tg::op_wait_limit_ns();
    q.timeouts = dev.timeouts;
    q.counters = static_cast<uint32_t*>(ws);
    tg::I8Peak* peaks = nullptr;
    if (more_runs(whole.K)) peaks = reinterpret_cast<tg::I8Peak*>(static_cast<char*>(ws) + tg::kI8CounterBytes);
    q.peaks = peaks;
    q.sums = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + kHeadBytes);
    uint16_t* order = reinterpret_cast<uint16_t*>(static_cast<char*>(ws) + kHeadBytes + slot_bytes(whole.M, whole.K));
    const int64_t ldo = up(whole.K, tg::kTcK), slab = slab_rows(whole.M, whole.K);
    CUtensorMap codes, ordered;
    if (!tg::op_map_2d(&codes, whole.B, CU_TENSOR_MAP_DATA_TYPE_UINT8, whole.K, whole.N, whole.ldb, tg::kTcK,
                       tg::kTcRows, CU_TENSOR_MAP_SWIZZLE_128B))
        return TG_ERR_LAUNCH;
    const int elem = sizeof(TC);
    for (int64_t m = 0; m < whole.M; m += slab) {
        I8Params& p = q.p;
        p = whole;
        p.M = whole.M - m < slab ? whole.M - m : slab;
        p.A += m * p.lda;
        p.sa += m;
        p.C = static_cast<char*>(p.C) + m * p.ldc * elem;
        if (p.resid != nullptr) p.resid = static_cast<const char*>(p.resid) + m * p.ldr * elem;
        const int64_t limit = lim.clusters[1] < tg::kI8MaxClusters ? lim.clusters[1] : tg::kI8MaxClusters;
        plan_wide(p, limit, &q);
        if (!tg::op_map_2d(&ordered, order, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, ldo, p.M, ldo * 2, 64,
                           static_cast<uint32_t>(q.tokens / tg::kWideCluster), CU_TENSOR_MAP_SWIZZLE_128B))
            return TG_ERR_LAUNCH;
        q.inject = tg::op_take_inject();
        // a cluster is the first of one shared tile at most
        const int64_t tiles = q.units / q.k_units, places = tiles < q.clusters ? tiles : q.clusters;
        const bool shares = q.grain != q.k_units;
        q.by_tile = tiles < q.clusters ? 1 : 0;
        q.places = shares ? static_cast<int32_t>(places) : 0;
        // (what the SMs hold at once, so that the peaks are few; with sums to zero, blocks on all SMs)
        const int64_t across = (ldo + tg::kI8PeakColumns - 1) / tg::kI8PeakColumns;
        const int64_t held = 8 * int64_t{dev.num_sms} < tg::kI8Peaks ? 8 * int64_t{dev.num_sms} : tg::kI8Peaks;
        const int64_t least = shares ? (dev.num_sms + across - 1) / across : 1, most = held / across;
        const int64_t down = p.M < least ? least : p.M < most ? p.M : most;
        q.across = static_cast<int32_t>(across);
        q.down = static_cast<int32_t>(down);
        tg_status_t st = launch(tg::tg_i8_expand, dim3(static_cast<unsigned>(across), static_cast<unsigned>(down)), 256,
                                0, 1, s, p.A, p.lda, p.M, p.K, order, ldo, q.counters,
                                reinterpret_cast<uint4*>(q.sums),
                                shares ? places * tg::kWideCluster * q.tokens * tg::kTcRows / 4 : int64_t{0}, peaks);
        if (st != TG_OK) return st;
        st = launch(kernel, dim3(static_cast<unsigned>(q.clusters * tg::kWideCluster)), tg::kWideThreads,
                    tg::kI8WideSmem, tg::kWideCluster, s, q, codes, ordered);
        if (st != TG_OK) return st;
    }
    return TG_OK;
}

// Launches the kernel for few rows; false where no shape fits.
template <typename TC, int NT>
bool take_few(const I8Params& p, const tg::OpDevice& dev, cudaStream_t s, tg_status_t* st) {
    FewPlan plan = plan_few<TC, NT>(p, dev);
    if (plan.time > 1e299) return false;
    *st = launch_few<TC, NT>(plan, dev, s);
    return true;
}

template <typename TC>
tg_status_t launch_type(const I8Params& p, const tg::OpDevice& dev, void* ws, cudaStream_t s) {
    tg_status_t st = TG_OK;
    if (p.K > 0 && prefer_few(p.M, p.N, p.K)) {
        if (p.M <= 8 ? take_few<TC, 1>(p, dev, s, &st)
            : p.M <= 16 ? take_few<TC, 2>(p, dev, s, &st)
            : p.M <= 32 ? take_few<TC, 4>(p, dev, s, &st)
                        : take_few<TC, 8>(p, dev, s, &st))
            return st;
    }
    if (p.K > 0 && p.M > 8) return launch_wide<TC>(p, dev, ws, s);
    const int64_t blocks = (p.M * p.N + 7) / 8, most = 8 * int64_t{dev.num_sms};
    return launch(tg::tg_gemm_i8_simple<TC>, dim3(static_cast<unsigned>(blocks < most ? blocks : most)), 256, 0, 1, s,
                  p);
}

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
    if (K > 0 && bytes < wide_bytes(M, K)) workspace = nullptr;  // (none is needed)
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
    if (x.out_dtype == TG_DTYPE_F32) return launch_type<float>(p, dev, workspace, s);
    return x.out_dtype == TG_DTYPE_F16 ? launch_type<__half>(p, dev, workspace, s) : launch_type<__nv_bfloat16>(p, dev, workspace, s);
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
