// workspace.cuh -- what streams' device buffers are kept under, and the lease of a
// stream's workspace to one call (host code; apart from common.cuh, which every
// kernel is compiled from).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <mutex>

namespace sgemm_gb300 {

// What the buffers of a stream are kept under: device, handle and, for
// cudaStreamPerThread, which names another stream in each host thread, the
// thread (0 otherwise; a thread's number is never given again).
struct StreamKey {
    int dev;
    uintptr_t stream;
    uint64_t thread;
    StreamKey(int d, cudaStream_t s) : dev(d), stream(reinterpret_cast<uintptr_t>(s)), thread(thread_of(s)) {}
    bool operator<(const StreamKey &o) const {
        return dev != o.dev ? dev < o.dev : stream != o.stream ? stream < o.stream : thread < o.thread;
    }
    // Waits for the stream's work, from any thread (the device current).
    cudaError_t synchronize() const {
        return thread != 0 ? cudaDeviceSynchronize() : cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream));
    }

private:
    static uint64_t thread_of(cudaStream_t s) {
        if (s != cudaStreamPerThread) return 0;
        static std::atomic<uint64_t> threads{0};
        thread_local const uint64_t mine = ++threads;
        return mine;
    }
};

// The workspace of (current device, s), at least `bytes` large and 256-byte
// aligned, for one call: it stays that call's until the lease goes, which has to be
// after the last launch that uses it.  Launches of another host thread's call on
// the stream would otherwise come between this call's.
struct WorkspaceLease {
    std::unique_lock<std::mutex> lock;
    void *p = nullptr;
};
// Returns an SGEMM_* status.
int stream_workspace(size_t bytes, cudaStream_t s, WorkspaceLease &out);

// Names a function that sgemm_release_workspaces calls: frees what its file keeps
// per stream, false if a CUDA call failed.
void on_release(bool (*f)());

}  // namespace sgemm_gb300
