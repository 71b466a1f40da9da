// Host helpers of the norms (norm.cu, layer_norm.cu): checks of their matrices, the plan of the
// kernels that take rows through rings, and launches.
#pragma once

#include <cstring>
#include <set>
#include <utility>

#include "norm.cuh"
#include "op_host.h"

namespace tg {

inline int elem_bytes(int32_t dtype) { return dtype == TG_DTYPE_F32 ? 4 : 2; }

inline bool misaligned(const void* p, int bytes) {
    return (reinterpret_cast<uintptr_t>(p) & static_cast<uintptr_t>(bytes - 1)) != 0;
}

// One matrix argument: present or not, its stride, its alignment.
inline tg_status_t check_matrix(const void* p, int64_t ld, int64_t cols, int bytes) {
    if (p == nullptr) return TG_OK;
    if (ld < cols) return TG_ERR_INVALID_VALUE;
    return misaligned(p, bytes) ? TG_ERR_MISALIGNED : TG_OK;
}

// The row kernels count strides in 32 bits.
inline bool narrow(int64_t a, int64_t b, int64_t c, int64_t d, int64_t e) {
    return (a | b | c | d | e) < (int64_t{1} << 32);
}

// Whether every row of a matrix (or of none) lies on 8 elements: 16 or 32 bytes.
inline bool wide(const void* p, int64_t ld, int bytes) {
    return p == nullptr || (!misaligned(p, 8 * bytes) && ld % 8 == 0);
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

// Of an SM's 228 KB of shared memory, for rings (a block has 5 KB and a reserved one besides).
constexpr int kRingBytes = 214 * 1024;

// How a kernel takes rows through rings.
struct RowPlan {
    int threads;  // of a group
    int groups;   // of a block
    int stages, stage_bytes;
    int per_sm;   // blocks
    size_t smem;
};

// `stage`: bytes of a group's stage; `more`: of a group besides its ring; `per_sm`: the blocks that registers allow on an SM.  False if no ring fits.
inline bool plan_rows(int64_t rows, int threads, int stage, int more, int per_sm, int num_sms, RowPlan* r) {
    if (rows > kOpMaxDim - 65536) return false;  // they count rows ahead in 31 bits
    r->threads = threads;
    r->groups = kNormThreads / threads;
    // few rows: blocks on every SM before groups in a block
    const int64_t each = (rows + num_sms - 1) / num_sms;
    if (r->groups > each) r->groups = static_cast<int>(each);
    r->stage_bytes = stage;
    for (r->per_sm = per_sm; r->per_sm >= 1; --r->per_sm)
        for (r->stages = 4; r->stages >= (r->per_sm > 1 ? 3 : 2); --r->stages) {
            r->smem = static_cast<size_t>(r->groups) * (r->stages * stage + more);
            if (r->per_sm * (r->smem + 6 * 1024) <= kRingBytes + 6 * 1024) return true;
        }
    return false;
}

// Lets a kernel use the shared memory that a block may have, once per device.
template <typename Kernel>
bool allow_smem(Kernel k, int dev) {
    static std::mutex m;
    static std::set<std::pair<const void*, int>> done;
    const auto key = std::make_pair(reinterpret_cast<const void*>(k), dev);
    std::lock_guard<std::mutex> lk(m);
    if (done.count(key) != 0) return true;
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, 220 * 1024) !=
        cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    done.insert(key);
    return true;
}

// Clusters of `size` blocks that the device holds at once (asked once for each shape).
template <typename Kernel>
int64_t max_clusters(Kernel kernel, int size, int threads, size_t smem, const OpDevice& dev) {
    static std::mutex m;
    static std::map<std::tuple<const void*, int, int, size_t, int>, int> known;
    const auto key = std::make_tuple(reinterpret_cast<const void*>(kernel), size, threads, smem, dev.dev);
    std::lock_guard<std::mutex> lk(m);
    const auto it = known.find(key);
    if (it != known.end()) return it->second;
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
        n = 0;
    }
    known[key] = n;
    return n;
}

}  // namespace tg
