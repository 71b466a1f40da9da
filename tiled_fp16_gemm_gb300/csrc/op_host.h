// Host helpers of the operators beside the GEMM (w4.cu, norm.cu): the device
// they run on, and workspaces that belong to a stream.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>
#include <functional>
#include <map>
#include <mutex>
#include <thread>
#include <tuple>

#include "tgemm.h"

namespace tg {

constexpr int kOpMaxDevices = 64;
constexpr int64_t kOpMaxDim = 2147483647LL;

struct OpDevice {
    int dev = 0;
    int num_sms = 0;
};

// The current device, if it is an sm_103 one (probed once per device).
inline tg_status_t op_device(OpDevice* out) {
    static std::mutex m;
    static int sms[kOpMaxDevices] = {};  // 0: not probed, -1: another architecture
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
    out->dev = d;
    out->num_sms = sms[d];
    return TG_OK;
}

// Device memory per (device, stream), grown on demand.  A buffer that became
// too small is kept, not freed: work in flight and captured graphs may still
// use it.  It grows to at least twice its size, so all buffers of a stream
// together hold less than twice the largest.  Growth allocates, which a
// stream capture forbids: there it fails with TG_ERR_NO_MEMORY before
// anything is enqueued, and the capture stays valid.
class OpWorkspace {
  public:
    tg_status_t get(int dev, cudaStream_t s, size_t bytes, void** out) {
        // the per-thread default stream is one handle for a stream per thread
        const size_t thread =
            s == cudaStreamPerThread ? std::hash<std::thread::id>{}(std::this_thread::get_id()) : 0;
        std::lock_guard<std::mutex> lk(m_);
        Buffer& b = of_[std::make_tuple(dev, s, thread)];
        if (b.bytes < bytes) {
            cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
            if (cudaStreamIsCapturing(s, &capture) != cudaSuccess ||
                capture != cudaStreamCaptureStatusNone) {
                cudaGetLastError();
                return TG_ERR_NO_MEMORY;
            }
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
            b.p = p;
            b.bytes = want;
        }
        *out = b.p;
        return TG_OK;
    }

  private:
    struct Buffer {
        void* p = nullptr;
        size_t bytes = 0;
    };
    std::mutex m_;
    std::map<std::tuple<int, cudaStream_t, size_t>, Buffer> of_;
};

}  // namespace tg
