// Host helpers of the norms (norm.cu, layer_norm.cu): checks of their matrices, and the plan of the
// kernels that take rows through rings.
#pragma once

#include <set>
#include <utility>

#include "launch_host.h"
#include "norm.cuh"

namespace tg {

inline int elem_bytes(int32_t dtype) { return dtype == TG_DTYPE_F32 ? 4 : 2; }

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

// max_clusters, asked once for each shape.
template <typename Kernel>
int64_t known_clusters(Kernel kernel, int size, int threads, size_t smem, const OpDevice& dev) {
    static std::mutex m;
    static std::map<std::tuple<const void*, int, int, size_t, int>, int> known;
    const auto key = std::make_tuple(reinterpret_cast<const void*>(kernel), size, threads, smem, dev.dev);
    std::lock_guard<std::mutex> lk(m);
    const auto it = known.find(key);
    if (it != known.end()) return it->second;
    const int n = max_clusters(kernel, size, threads, smem, dev);
    known[key] = n;
    return n;
}

}  // namespace tg
