// Host helpers of the operators beside the GEMM (w4.cu, norm.cu): the device
// they run on, and workspaces that belong to a stream.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <map>
#include <mutex>
#include <new>
#include <tuple>
#include <vector>

#include "stream_key.h"
#include "tgemm.h"

namespace tg {

// The body of a C entry point: no exception leaves it (a host allocation that fails, in a
// workspace's bookkeeping, is one).
template <typename F>
tg_status_t op_entry(F body) noexcept {
    try {
        return body();
    } catch (const std::bad_alloc&) {
        return TG_ERR_NO_MEMORY;
    } catch (...) {
        return TG_ERR_LAUNCH;
    }
}

constexpr int kOpMaxDevices = 64;
constexpr int64_t kOpMaxDim = 2147483647LL;

struct OpDevice {
    int dev = 0;
    int num_sms = 0;
    unsigned int* timeouts = nullptr;  // the device's word for waits that ran out
};

// That word of the current device, which tg_sync_status reads; null on an error.  In tgemm.cu.
unsigned int* op_timeout_word();

// The current device, if it is an sm_103 one (probed once per device).
inline tg_status_t op_device(OpDevice* out) {
    static std::mutex m;
    static int sms[kOpMaxDevices] = {};  // 0: not probed, -1: another architecture
    static unsigned int* words[kOpMaxDevices] = {};
    int d = -1;
    if (cudaGetDevice(&d) != cudaSuccess || d < 0 || d >= kOpMaxDevices) {
        cudaGetLastError();
        return TG_ERR_UNSUPPORTED_DEVICE;
    }
    std::lock_guard<std::mutex> lk(m);
    if (sms[d] == 0) {
        int major = 0, minor = 0, n = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, d) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, d) != cudaSuccess ||
            cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, d) != cudaSuccess) {
            cudaGetLastError();
            return TG_ERR_UNSUPPORTED_DEVICE;
        }
        sms[d] = major == 10 && minor == 3 ? n : -1;
    }
    if (sms[d] < 0) return TG_ERR_UNSUPPORTED_DEVICE;
    if (words[d] == nullptr && (words[d] = op_timeout_word()) == nullptr) return TG_ERR_LAUNCH;
    out->dev = d;
    out->num_sms = sms[d];
    out->timeouts = words[d];
    return TG_OK;
}

// Limit of every wait in a kernel (tg_debug_set_wait_timeout_ns), in tgemm.cu.
uint64_t op_wait_limit_ns();

// The mode that tg_debug_inject set for the next launch, which is then 0 again.
int32_t op_take_inject();

// After a wait ran out on `dev`, the current device: clears counters that a kernel of w4.cu
// may have left, once everything queued there has ended.
void w4_clear_counters(int dev);

// Whether `encode`, a call of cuTensorMapEncodeTiled, succeeds.  That needs a current context,
// which a host thread does not have before its first call that binds one: then it is bound here.
template <typename F>
bool op_encode(F encode) {
    CUresult r = encode();
    int d = 0;
    if (r == CUDA_ERROR_INVALID_CONTEXT && cudaGetDevice(&d) == cudaSuccess && cudaSetDevice(d) == cudaSuccess)
        r = encode();
    return r == CUDA_SUCCESS;
}

// The 2-D tensor map of rows of `inner` elements, `row_bytes` apart, read in boxes of
// box_inner × box_outer; zero outside.
inline bool op_map_2d(CUtensorMap* map, const void* ptr, CUtensorMapDataType type, uint64_t inner,
                      uint64_t outer, uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer,
                      CUtensorMapSwizzle swizzle) {
    static PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                             &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            fn = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    }();
    if (encode == nullptr) return false;
    cuuint64_t dims[2] = {inner, outer};
    cuuint64_t strides[1] = {row_bytes};
    cuuint32_t box[2] = {box_inner, box_outer};
    cuuint32_t steps[2] = {1, 1};
    return op_encode([&] {
        return encode(map, type, 2, const_cast<void*>(ptr), dims, strides, box, steps,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    });
}

// Device memory per (device, stream), grown on demand.  A buffer that became
// too small is kept, not freed: work in flight and captured graphs may still
// use it.  It grows to at least twice its size, so all buffers of a stream
// together hold less than twice the largest.  Growth allocates, which a
// stream capture forbids: there it fails with TG_ERR_NO_MEMORY before
// anything is enqueued, and the capture stays valid.
//
// A call's launches hand each other what lies there, so no launch of another host
// thread's call on the stream may come between them: the caller keeps `hold` until
// its last one.  Other streams do not wait.
//
// The first `counters` bytes of a buffer are zero when it is made, and every launch
// leaves them at zero, but for one that gives up on a wait: then clear() is needed.
class OpWorkspace {
  public:
    using Hold = std::unique_lock<std::mutex>;
    explicit OpWorkspace(size_t counters = 0) : counters_(counters) {}

    tg_status_t get(int dev, cudaStream_t s, size_t bytes, void** out, Hold* hold) {
        Buffer* found;
        {
            std::lock_guard<std::mutex> lk(m_);
            found = &of_[stream_key(dev, s)];  // (entries stay where they are)
        }
        Buffer& b = *found;
        *hold = Hold(b.m);
        if (b.bytes < bytes) {
            cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
            if (cudaStreamIsCapturing(s, &capture) != cudaSuccess ||
                capture != cudaStreamCaptureStatusNone) {
                cudaGetLastError();
                return TG_ERR_NO_MEMORY;
            }
            b.all.reserve(b.all.size() + 1);  // (what may throw, before there is memory to lose)
            size_t want = bytes > 2 * b.bytes ? bytes : 2 * b.bytes;
            void* p = nullptr;
            if (cudaMalloc(&p, want) != cudaSuccess) {
                cudaGetLastError();
                want = bytes;
                if (cudaMalloc(&p, want) != cudaSuccess) {
                    cudaGetLastError();
                    return TG_ERR_NO_MEMORY;
                }
            }
            if (counters_ > 0 && cudaMemsetAsync(p, 0, counters_, s) != cudaSuccess) {
                cudaGetLastError();
                cudaFree(p);
                return TG_ERR_LAUNCH;
            }
            b.all.push_back(p);
            b.bytes = want;
        }
        *out = b.all.back();
        return TG_OK;
    }

    // Zeroes the counters of all buffers of `dev`, the current device, those that became
    // too small too (captured graphs may use them), once everything queued there has
    // ended.  No call is between get() and its last launch meanwhile.
    void clear(int dev) {
        std::lock_guard<std::mutex> lk(m_);
        std::vector<Hold> holds;
        for (auto& of : of_)
            if (std::get<0>(of.first) == dev) holds.emplace_back(of.second.m);
        cudaDeviceSynchronize();
        for (auto& of : of_)
            if (std::get<0>(of.first) == dev)
                for (void* p : of.second.all) cudaMemset(p, 0, counters_);
        cudaDeviceSynchronize();
        cudaGetLastError();
    }

  private:
    struct Buffer {
        std::mutex m;
        std::vector<void*> all;  // the last one is in use
        size_t bytes = 0;        // of that one
    };
    const size_t counters_;
    std::mutex m_;
    std::map<StreamKey, Buffer> of_;
};

}  // namespace tg
