// What a stream's buffers are found by.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <functional>
#include <thread>
#include <tuple>

namespace tg {

// Device, stream, and the calling thread where the handle alone does not name a stream:
// the per-thread default stream is one handle for a stream of every thread.
using StreamKey = std::tuple<int, cudaStream_t, size_t>;

inline StreamKey stream_key(int dev, cudaStream_t s) {
    const size_t thread =
        s == cudaStreamPerThread ? std::hash<std::thread::id>{}(std::this_thread::get_id()) : 0;
    return StreamKey(dev, s, thread);
}

}  // namespace tg
