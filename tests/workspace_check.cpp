// Host-side check of the workspaces in op_host.h, on stand-ins for the CUDA calls that they
// make (compiled and run by test_threads.py with the system C++ compiler).  "Launches" are
// entries of a log.
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <thread>
#include <vector>

#include "op_host.h"

static thread_local bool g_fail_new = false;
void* operator new(size_t n) {
    void* p = g_fail_new ? nullptr : std::malloc(n);
    if (p == nullptr) throw std::bad_alloc();
    return p;
}
void operator delete(void* p) noexcept { std::free(p); }
void operator delete(void* p, size_t) noexcept { std::free(p); }

extern "C" {
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaMalloc(void** p, size_t bytes) {
    *p = std::malloc(bytes);
    return cudaSuccess;
}
cudaError_t cudaFree(void* p) {
    std::free(p);
    return cudaSuccess;
}
cudaError_t cudaMemset(void* p, int v, size_t bytes) {
    std::memset(p, v, bytes);
    return cudaSuccess;
}
cudaError_t cudaMemsetAsync(void* p, int v, size_t bytes, cudaStream_t) { return cudaMemset(p, v, bytes); }
cudaError_t cudaDeviceSynchronize() { return cudaSuccess; }
cudaError_t cudaStreamIsCapturing(cudaStream_t, cudaStreamCaptureStatus* s) {
    *s = cudaStreamCaptureStatusNone;
    return cudaSuccess;
}
}

namespace {

cudaStream_t stream(int i) { return reinterpret_cast<cudaStream_t>(static_cast<uintptr_t>(64 * i)); }

struct Launch {
    int stream, thread;
};
std::mutex g_log_mutex;
std::vector<Launch> g_log;

void launch(int stream, int thread) {
    {
        std::lock_guard<std::mutex> lk(g_log_mutex);
        g_log.push_back({stream, thread});
    }
    std::this_thread::yield();
}

}  // namespace

int main() {
    tg::OpWorkspace ws;
    // Two threads on each of two streams, two launches a call, sizes that grow: on a stream
    // the launches of a call follow one another.
    std::vector<std::thread> threads;
    for (int t = 0; t < 4; ++t)
        threads.emplace_back([&, t] {
            const int s = 1 + t % 2;
            for (int i = 0; i < 5000; ++i) {
                tg::OpWorkspace::Hold hold;
                void* p = nullptr;
                if (ws.get(0, stream(s), static_cast<size_t>(1 + i / 1000) << 10, &p, &hold) != TG_OK || p == nullptr)
                    std::abort();
                launch(s, t);
                launch(s, t);
            }
        });
    for (auto& t : threads) t.join();
    for (int s = 1; s <= 2; ++s) {
        std::vector<int> of;
        for (const Launch& l : g_log)
            if (l.stream == s) of.push_back(l.thread);
        for (size_t i = 0; i + 1 < of.size(); i += 2)
            if (of[i] != of[i + 1]) {
                std::printf("FAIL stream %d: launch %zu is thread %d's, the next one thread %d's\n", s, i, of[i], of[i + 1]);
                return 1;
            }
    }
    // A call under way on one stream keeps no other stream waiting.
    tg::OpWorkspace::Hold one, two;
    void *p = nullptr, *q = nullptr;
    if (ws.get(0, stream(1), 64, &p, &one) != TG_OK || ws.get(0, stream(2), 64, &q, &two) != TG_OK || p == q) {
        std::printf("FAIL two streams\n");
        return 1;
    }
    // Counters: zero at first, cleared in every buffer of the device, one that became too
    // small among them, and on no other device.
    tg::OpWorkspace counted(256);
    unsigned char* at[4];
    for (int i = 0; i < 4; ++i) {
        tg::OpWorkspace::Hold hold;
        void* r = nullptr;
        if (counted.get(i == 3, stream(i == 2 ? 2 : 1), i == 1 ? 4096 : 512, &r, &hold) != TG_OK) std::abort();
        at[i] = static_cast<unsigned char*>(r);
        for (int j = 0; j < 256; ++j)
            if (at[i][j] != 0) {
                std::printf("FAIL buffer %d is not zero at first\n", i);
                return 1;
            }
        std::memset(at[i], i + 1, 512);
    }
    counted.clear(0);
    for (int i = 0; i < 4; ++i)
        if (at[i][0] != (i == 3 ? 4 : 0) || at[i][255] != at[i][0] || at[i][256] != i + 1) {
            std::printf("FAIL buffer %d after the clearing: %d %d\n", i, at[i][0], at[i][256]);
            return 1;
        }
    // No exception leaves an entry point.
    if (tg::op_entry([]() -> tg_status_t { throw std::bad_alloc(); }) != TG_ERR_NO_MEMORY ||
        tg::op_entry([]() -> tg_status_t { throw 1; }) != TG_ERR_LAUNCH ||
        tg::op_entry([] { return TG_ERR_MISALIGNED; }) != TG_ERR_MISALIGNED) {
        std::printf("FAIL exceptions\n");
        return 1;
    }
    // Nor that of a workspace whose bookkeeping finds no host memory: later calls go on.
    tg::OpWorkspace poor;
    void* r = nullptr;
    g_fail_new = true;
    const tg_status_t none = tg::op_entry([&] {
        tg::OpWorkspace::Hold hold;
        return poor.get(0, stream(1), 64, &r, &hold);
    });
    g_fail_new = false;
    const tg_status_t then = tg::op_entry([&] {
        tg::OpWorkspace::Hold hold;
        return poor.get(0, stream(1), 64, &r, &hold);
    });
    if (none != TG_ERR_NO_MEMORY || then != TG_OK || r == nullptr) {
        std::printf("FAIL without host memory: %d, then %d\n", none, then);
        return 1;
    }
    std::printf("OK\n");
    return 0;
}
