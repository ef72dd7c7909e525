// fake_device.cpp -- the entry points of api.cu, noalloc.cu and q8_api.cu on a stand-in for
// the CUDA runtime and the kernel launchers, so that what the host does with its
// workspaces can be followed without a GPU.
//
// Device memory is a list of live buffers, never touched; a launcher stands for the
// kernels that it would enqueue: it takes a while, and checks that its
// workspace is live and that no other launcher works with it meanwhile.  The
// program runs the scenario named on its command line and exits with the number
// of faults found, each with a line on stderr.
#include <cuda_runtime_api.h>

#include <atomic>
#include <chrono>
#include <cstdio>
#include <cstring>
#include <map>
#include <mutex>
#include <set>
#include <thread>
#include <vector>

#include "common.cuh"
#include "q8.cuh"
#include "sgemm_gb300.h"

namespace {

std::mutex mu;
std::set<void *> live;                      // buffers
std::map<void *, std::thread::id> users;    // buffers a launcher works with
std::set<cudaStream_t> captured;            // streams under capture
alignas(256) unsigned symbol[64];   // the address of every __device__ variable
std::atomic<int> faults{0}, launches{0};
thread_local void *last = nullptr;          // workspace of this thread's last launch
size_t most_users = 0;                      // launchers at work at one time, at most

void fault(const char *what) {
    ++faults;
    std::fprintf(stderr, "fault: %s\n", what);
}

bool usable(void *p) { return p == symbol || live.count(p) != 0; }

// What a launcher does with its workspace.
cudaError_t launched(void *ws) {
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!usable(ws)) fault("a launch got a workspace that is not allocated");
        if (!users.emplace(ws, std::this_thread::get_id()).second)
            fault("two calls' launches into one workspace are mixed");
        if (users.size() > most_users) most_users = users.size();
    }
    std::this_thread::sleep_for(std::chrono::microseconds(300));
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!usable(ws)) fault("a workspace was freed between a call's launches");
        auto it = users.find(ws);
        if (it != users.end() && it->second == std::this_thread::get_id()) users.erase(it);
    }
    last = ws;
    ++launches;
    return cudaSuccess;
}

cudaError_t release(void *p) {
    std::lock_guard<std::mutex> lock(mu);
    if (live.erase(p) != 0) return cudaSuccess;
    fault("a buffer was freed that is not allocated");
    return cudaErrorInvalidValue;
}

}  // namespace

// ---- the runtime -------------------------------------------------------------------

extern "C" {
cudaError_t cudaGetDevice(int *d) { *d = 0; return cudaSuccess; }
cudaError_t cudaSetDevice(int) { return cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaDeviceSynchronize() { return cudaSuccess; }
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int *v, cudaDeviceAttr a, int) {
    *v = a == cudaDevAttrComputeCapabilityMajor ? 10 : a == cudaDevAttrComputeCapabilityMinor ? 3 : 152;
    return cudaSuccess;
}
cudaError_t cudaGetSymbolAddress(void **p, const void *) { *p = symbol; return cudaSuccess; }
cudaError_t cudaMemset(void *p, int v, size_t n) { std::memset(p, v, n); return cudaSuccess; }
cudaError_t cudaMemcpy(void *d, const void *s, size_t n, cudaMemcpyKind) { std::memcpy(d, s, n); return cudaSuccess; }
cudaError_t cudaGetDriverEntryPointByVersion(const char *, void **f, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult *q) {
    *f = reinterpret_cast<void *>(&cudaGetDevice);      // never called here
    *q = cudaDriverEntryPointSuccess;
    return cudaSuccess;
}
cudaError_t cudaStreamIsCapturing(cudaStream_t s, cudaStreamCaptureStatus *st) {
    std::lock_guard<std::mutex> lock(mu);
    *st = captured.count(s) ? cudaStreamCaptureStatusActive : cudaStreamCaptureStatusNone;
    return cudaSuccess;
}
cudaError_t cudaMallocAsync(void **p, size_t, cudaStream_t s) {
    std::lock_guard<std::mutex> lock(mu);
    if (captured.count(s)) fault("an allocation on a stream under capture");
    static uintptr_t next = (uintptr_t)1 << 50;     // an address is given once
    *p = reinterpret_cast<void *>(next += 256);
    live.insert(*p);
    return cudaSuccess;
}
cudaError_t cudaFreeAsync(void *p, cudaStream_t) { return release(p); }
cudaError_t cudaFree(void *p) { return p ? release(p) : cudaSuccess; }

// what nvcc's registration of the two files' own kernels calls
void **__cudaRegisterFatBinary(void *) { static void *h; return &h; }
void __cudaRegisterFatBinaryEnd(void **) {}
void __cudaUnregisterFatBinary(void **) {}
void __cudaRegisterFunction(void **, const char *, char *, const char *, int, uint3 *, uint3 *, dim3 *, dim3 *, int *) {}
void __cudaRegisterVar(void **, char *, char *, const char *, int, size_t, int, int) {}
unsigned __cudaPushCallConfiguration(dim3, dim3, size_t, struct CUstream_st *) { return 0; }
cudaError_t __cudaPopCallConfiguration(dim3 *, dim3 *, size_t *, void *) { return cudaSuccess; }
cudaError_t __cudaGetKernel(cudaKernel_t *, const void *) { return cudaSuccess; }
cudaError_t __cudaLaunchKernel(cudaKernel_t, dim3, dim3, void **, size_t, cudaStream_t) { return cudaSuccess; }
}

// ---- the launchers -----------------------------------------------------------------

namespace sgemm_gb300 {
int ffma_config_count() { return 1; }
int ffma_config_for(int64_t, int64_t, int64_t) { return 0; }
bool ffma_config_info(int, int *, int *, int *, int *, int *, int *) { return false; }
int ffma_force_config(int) { return -1; }
int ffma_force_tail_sum(int) { return -1; }
int64_t ffma_tma_at_ld(int64_t M) { return (M + 3) / 4 * 4; }
int64_t ffma_tma_max_m() { return 1 << 20; }
void ffma_tma_plan_info(const GemmArgs &, int64_t *, int *, int *) {}
int64_t ffma_tma_workspace_floats(const GemmArgs &g, int64_t) { return g.K * ffma_tma_at_ld(g.M); }
int kernel_timing(int) { return 0; }
bool kernel_timing_result(double *, int64_t *) { return true; }
bool release_host_paths() { return true; }
bool tf32x3_can_run(int64_t, int64_t, int64_t) { return true; }
size_t tf32_workspace_floats(int64_t M, int64_t N, int64_t K, int) { return (size_t)((M + N) * K); }
cudaError_t launch_decode(const GemmArgs &) { return cudaSuccess; }
cudaError_t launch_ffma_generic(const GemmArgs &) { return cudaSuccess; }
cudaError_t launch_scale_c(const GemmArgs &) { return cudaSuccess; }
cudaError_t launch_ffma_tma(const GemmArgs &, float *ws, int64_t) { return launched(ws); }
cudaError_t launch_tf32(const GemmArgs &, float *ws, int) { return launched(ws); }
cudaError_t launch_q8_rows(const Q8RowsArgs &) { return cudaSuccess; }
cudaError_t launch_q8_stream(const Q8LinearArgs &) { return cudaSuccess; }
bool q8_mma_can_run(const Q8LinearArgs &) { return true; }
size_t q8_mma_workspace_bytes(const Q8LinearArgs &a) { return (size_t)(a.M * a.K * 2); }
cudaError_t launch_q8_mma(const Q8LinearArgs &, void *ws) { return launched(ws); }
size_t q8_moe_workspace_bytes(int T, int, int top_k, int H, int I) { return (size_t)T * top_k * (H + I) * 9; }
cudaError_t launch_q8_moe(const Q8MoeArgs &, void *ws) { return launched(ws); }
}  // namespace sgemm_gb300

// ---- calls ---------------------------------------------------------------------------

namespace {

template <typename T>
T *at(int i) { return reinterpret_cast<T *>((uintptr_t)(i + 1) << 40); }     // never read

cudaStream_t stream(int i) { return reinterpret_cast<cudaStream_t>((uintptr_t)0x10000 * (i + 1)); }

int linear(int64_t M, cudaStream_t s) {
    return sgemm_q8_linear(M, 20000, 256, at<int8_t>(0), 256, at<float>(1), at<int8_t>(2), 256, at<float>(3), nullptr, 0,
                           at<void>(4), 20000, SGEMM_TYPE_BF16, s);
}
int moe(int64_t T, cudaStream_t s) {
    return sgemm_q8_moe(T, 8, 2, 512, 256, at<void>(0), 512, SGEMM_TYPE_BF16, at<float>(1), 512, at<int8_t>(2), 512,
                        at<float>(3), at<int8_t>(4), 256, at<float>(5), 1, at<void>(6), 512, nullptr, nullptr, s);
}
int product(int64_t M, cudaStream_t s) {
    return sgemm(M, 512, 512, 1.0f, at<float>(0), 512, at<float>(1), 512, 0.0f, at<float>(2), 512, s);
}
int fixed_product(int64_t M, cudaStream_t s) {
    return sgemm_noalloc(M, 512, 512, 1.0f, at<float>(0), 512, at<float>(1), 512, 0.0f, at<float>(2), 512, s);
}
void expect(int rc, int want, const char *what) {
    if (rc != want) {
        fault(what);
        std::fprintf(stderr, "  status %d, not %d\n", rc, want);
    }
}

// Calls of every kind and of growing size from several host threads on one stream.
void threads_share_a_stream() {
    std::vector<std::thread> all;
    for (int t = 0; t < 4; ++t)
        all.emplace_back([t] {
            for (int i = 0; i < 25; ++i) {
                expect(linear(200 + 100 * i, stream(0)), SGEMM_OK, "linear");
                expect(moe(1 + (i + t) % 64, stream(0)), SGEMM_OK, "moe");
                expect(product(300 + 50 * i, stream(0)), SGEMM_OK, "sgemm");
                expect(fixed_product(300, stream(0)), SGEMM_OK, "sgemm_noalloc");
            }
        });
    for (auto &t : all) t.join();
    if (launches != 4 * 25 * 4) fault("calls are missing");
}

// Threads on streams of their own do not wait for one another.
void threads_on_their_own_streams() {
    std::vector<std::thread> all;
    for (int t = 0; t < 4; ++t)
        all.emplace_back([t] {
            for (int i = 0; i < 100; ++i) expect(moe(8, stream(t)), SGEMM_OK, "moe");
        });
    for (auto &t : all) t.join();
    if (most_users < 2) fault("calls on different streams ran one after another");
}

// cudaStreamPerThread names another stream in each thread: no buffer is shared.
void per_thread_streams_share_nothing() {
    void *seen[3] = {};
    std::vector<std::thread> all;
    for (int t = 0; t < 3; ++t)
        all.emplace_back([t, &seen] {
            for (int i = 0; i < 20; ++i) expect(moe(8 + i, cudaStreamPerThread), SGEMM_OK, "moe");
            seen[t] = last;
        });
    for (auto &t : all) t.join();
    if (seen[0] == seen[1] || seen[1] == seen[2] || seen[0] == seen[2])
        fault("streams of different threads got one workspace");
}

void capture(cudaStream_t s, bool on) {
    std::lock_guard<std::mutex> lock(mu);
    if (on) captured.insert(s);
    else captured.erase(s);
}

// A workspace that a captured call used is there for the graph's replays, whatever
// is called on the stream afterwards.
void graph_keeps_its_workspace() {
    const cudaStream_t s = stream(0);
    std::vector<void *> in_graph;
    for (int64_t size : {100, 1000, 30000}) {       // a graph on each of three growing workspaces
        expect(linear(size, s), SGEMM_OK, "eager");
        expect(moe(8, s), SGEMM_OK, "eager");
        capture(s, true);
        expect(moe(8, s), SGEMM_OK, "captured");
        in_graph.push_back(last);
        expect(linear(size, s), SGEMM_OK, "captured again");
        if (last != in_graph.back()) fault("two captured calls got different workspaces");
        const int before = launches;
        expect(linear(100 * size, s), SGEMM_ERR_CAPTURE, "a captured call that needs a larger workspace");
        if (launches != before) fault("a refused call launched something");
        capture(s, false);
        expect(moe(8, s), SGEMM_OK, "eager again");
    }
    expect(product(20000, s), SGEMM_OK, "a last growth");
    expect(linear(300000, s), SGEMM_OK, "a last growth");
    std::lock_guard<std::mutex> lock(mu);
    for (void *p : in_graph)
        if (live.count(p) == 0) fault("a graph's workspace was freed");
}

// Without a capture, growth frees what it replaces.
void growth_frees_the_old_workspace() {
    for (int64_t size : {100, 1000, 30000, 200000}) {
        expect(linear(size, stream(0)), SGEMM_OK, "linear");
        if (live.size() != 1) fault("a replaced workspace was kept");
    }
}

}  // namespace

int main(int argc, char **argv) {
    const struct { const char *name; void (*run)(); } scenarios[] = {
        {"threads_share_a_stream", threads_share_a_stream},
        {"threads_on_their_own_streams", threads_on_their_own_streams},
        {"per_thread_streams_share_nothing", per_thread_streams_share_nothing},
        {"graph_keeps_its_workspace", graph_keeps_its_workspace},
        {"growth_frees_the_old_workspace", growth_frees_the_old_workspace},
    };
    for (const auto &s : scenarios)
        if (argc == 2 && std::strcmp(argv[1], s.name) == 0) {
            s.run();
            expect(sgemm_release_workspaces(), SGEMM_OK, "release");
            if (!live.empty()) fault("buffers are left after the release");
            return faults > 250 ? 250 : (int)faults;
        }
    std::fprintf(stderr, "unknown scenario\n");
    return 255;
}
