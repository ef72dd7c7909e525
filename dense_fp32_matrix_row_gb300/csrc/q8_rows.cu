// q8_rows.cu -- rows to 8-bit whole numbers with one scale each, alone or
// behind a residual addition and an RMS norm.
//
//     h = x + residual        p = h * weight        m = max_k |p_k|
//     r = 1 / sqrt(mean_k h_k^2 + eps)
//     y = p * r               q = rint(p * (127 / m))      scale = (m / 127) * r
//
// (weight absent: p = x, r = 1.)  q * scale stands for y.  The norm's factor r
// is the same for the whole row, so it cancels out of q: the 8-bit values
// need the row's maximum only, which no summation order can change, and the
// sum of squares reaches the scale alone.  h is the FP32 sum; it is rounded
// once, to the stored h.
//
// Bound by memory: each of x, residual, h, y is touched once and q written
// once.  One block takes one row and keeps it in registers between the
// reduction and the store (rows up to 16384 elements); longer rows are read
// twice.
#include "q8.cuh"

namespace sgemm_gb300 {
namespace {

// The norm's factor is r * lift.  lift is 1 unless the sum of squares left
// FP32's range: squares that overflow (elements above about 1e18) are summed
// again of h * 2^-100, and a mean (with eps) below 2^-100, whose squares may
// have underflowed, of h * 2^100.
constexpr float kLargest = 3.402823466e38f;
constexpr float kTwo100 = 1.2676506002282294e30f, kTwoM100 = 7.8886090522101181e-31f;

__device__ __forceinline__ float inv_rms(float ss, int64_t K, float eps) {
    return __fdiv_rn(1.0f, __fsqrt_rn(__fdiv_rn(ss, (float)(K > 0 ? K : 1)) + eps));
}

// lift for a row with this sum of squares and largest |p| (see above).
__device__ __forceinline__ float norm_lift(float ss, int64_t K, float eps, uint32_t max_bits) {
    if (ss > kLargest && max_bits < 0x7f800000u) return kTwoM100;
    if (ss < kTwoM100 * (float)K && eps < kTwoM100) return kTwo100;
    return 1.0f;
}

// scale of a row: step times the norm's factor.
__device__ __forceinline__ float row_scale(const RowQuant &rq, float lift, float r) {
    return rq.step == 0.0f ? 0.0f : rq.step * (rq.unpre * lift) * r;
}

// One row per block, NV vectors of V elements per thread held in registers.
template <typename T, int V, int NV>
__global__ void __launch_bounds__(512)
q8_rows_kernel(int64_t K, const T *x, int64_t ldx, const T *residual,
               int64_t ldr, const float *__restrict__ weight, float eps, T *h, int64_t ldh, T *y,
               int64_t ldy, int8_t *__restrict__ q, int64_t ldq, float *__restrict__ scale) {
    __shared__ uint32_t red[64];
    const int64_t row = blockIdx.x;
    pdl_wait();
    const T *xr = x + row * ldx;
    const T *rr = residual ? residual + row * ldr : nullptr;
    const int nvec = (int)(K / V);
    float v[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = threadIdx.x + i * (int)blockDim.x;
        if (c < nvec) {
            load_vec<T, V>(xr + (int64_t)c * V, v[i]);
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) v[i][e] = 0.0f;
        }
    }
    if (rr) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = threadIdx.x + i * (int)blockDim.x;
            if (c < nvec) {
                float t[V];
                load_vec<T, V>(rr + (int64_t)c * V, t);
#pragma unroll
                for (int e = 0; e < V; ++e) v[i][e] += t[e];
            }
        }
    }
    uint32_t mx = 0;
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = threadIdx.x + i * (int)blockDim.x;
        if (c < nvec) {
            if (h) store_vec<T, V>(h + row * ldh + (int64_t)c * V, v[i]);
            float w[V];
            if (weight) load_vec<float, V>(weight + (int64_t)c * V, w);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                ss = fmaf(v[i][e], v[i][e], ss);
                mx = max(mx, abs_bits(weight ? v[i][e] * w[e] : v[i][e]));
            }
        }
    }
    block_max_sum(mx, ss, red);
    const RowQuant rq(mx);
    float r = 1.0f, lift = 1.0f;
    if (weight) {
        r = inv_rms(ss, K, eps);   // 0 for an infinite row, NaN for one with a NaN
        lift = norm_lift(ss, K, eps, mx);
        if (lift != 1.0f) {
            float s2 = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float t = v[i][e] * lift;
                    s2 = fmaf(t, t, s2);
                }
            uint32_t none = 0;
            block_max_sum(none, s2, red);
            r = inv_rms(s2, K, lift > 1.0f ? eps * lift * lift : 0.0f);
        }
    }
    if (threadIdx.x == 0) scale[row] = row_scale(rq, lift, r);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = threadIdx.x + i * (int)blockDim.x;
        if (c < nvec) {
            if (weight) {
                float w[V];
                load_vec<float, V>(weight + (int64_t)c * V, w);
#pragma unroll
                for (int e = 0; e < V; ++e) v[i][e] *= w[e];
                if (y) {
                    float t[V];
#pragma unroll
                    for (int e = 0; e < V; ++e) t[e] = v[i][e] * lift * r;
                    store_vec<T, V>(y + row * ldy + (int64_t)c * V, t);
                }
            }
            store_q<V>(q + row * ldq + (int64_t)c * V, rq, v[i]);
        }
    }
}

// Rows too long for registers: one pass for the maximum and the sum, a second
// that reads x and residual again (mostly from L2) and writes.  Nothing is
// written before the second pass, so h may be x or residual itself.
template <typename T>
__global__ void __launch_bounds__(1024)
q8_rows_long_kernel(int64_t K, const T *x, int64_t ldx, const T *residual, int64_t ldr,
                    const float *__restrict__ weight, float eps, T *h, int64_t ldh, T *y,
                    int64_t ldy, int8_t *__restrict__ q, int64_t ldq, float *__restrict__ scale) {
    __shared__ uint32_t red[64];
    const int64_t row = blockIdx.x;
    pdl_wait();
    const T *xr = x + row * ldx;
    const T *rr = residual ? residual + row * ldr : nullptr;
    auto sum_at = [&](int64_t k) { return to_f32<T>(xr[k]) + (rr ? to_f32<T>(rr[k]) : 0.0f); };
    uint32_t mx = 0;
    float ss = 0.0f;
    for (int64_t k = threadIdx.x; k < K; k += blockDim.x) {
        const float t = sum_at(k);
        ss = fmaf(t, t, ss);
        mx = max(mx, abs_bits(weight ? t * weight[k] : t));
    }
    block_max_sum(mx, ss, red);
    const RowQuant rq(mx);
    float r = 1.0f, lift = 1.0f;
    if (weight) {
        r = inv_rms(ss, K, eps);
        lift = norm_lift(ss, K, eps, mx);
        if (lift != 1.0f) {
            float s2 = 0.0f;
            for (int64_t k = threadIdx.x; k < K; k += blockDim.x) {
                const float t = sum_at(k) * lift;
                s2 = fmaf(t, t, s2);
            }
            uint32_t none = 0;
            block_max_sum(none, s2, red);
            r = inv_rms(s2, K, lift > 1.0f ? eps * lift * lift : 0.0f);
        }
    }
    if (threadIdx.x == 0) scale[row] = row_scale(rq, lift, r);
    for (int64_t k = threadIdx.x; k < K; k += blockDim.x) {
        const float t = sum_at(k);
        const float p = weight ? t * weight[k] : t;
        if (h) h[row * ldh + k] = from_f32<T>(t);
        if (y) y[row * ldy + k] = from_f32<T>(p * lift * r);
        q[row * ldq + k] = (int8_t)rq(p);
    }
}

template <typename K, typename... A>
cudaError_t launch_rows_pdl(K kern, dim3 grid, int threads, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <typename T, int V, int NV>
cudaError_t launch_reg(const Q8RowsArgs &a, int threads) {
    return launch_rows_pdl(q8_rows_kernel<T, V, NV>, dim3((unsigned)a.M), threads, a.stream, a.K,
                           (const T *)a.x, a.ldx, (const T *)a.residual, a.ldr, a.weight, a.eps,
                           (T *)a.h, a.ldh, (T *)a.y, a.ldy, a.q, a.ldq, a.scale);
}

// Vectors per thread: as few as 512 threads a row allow.
template <typename T, int V>
cudaError_t launch_v(const Q8RowsArgs &a) {
    const int64_t nvec = a.K / V;
    const int nv = nvec <= 512 ? 1 : nvec <= 1024 ? 2 : nvec <= 2048 ? 4 : nvec <= 4096 ? 8 : 16;
    int threads = (int)((((nvec + nv - 1) / nv) + 31) / 32 * 32);
    if (threads < 32) threads = 32;
    switch (nv) {
        case 1: return launch_reg<T, V, 1>(a, threads);
        case 2: return launch_reg<T, V, 2>(a, threads);
        case 4: return launch_reg<T, V, 4>(a, threads);
        default: break;
    }
    if constexpr (V <= 4) {
        if (nv == 8) return launch_reg<T, V, 8>(a, threads);
    }
    if constexpr (V == 1) {
        if (nv == 16) return launch_reg<T, V, 16>(a, threads);
    }
    return cudaErrorInvalidValue;
}

template <typename T>
cudaError_t launch_t(const Q8RowsArgs &a) {
    // A vector of V elements is one aligned access of every array (16 bytes
    // at V = 8 in bf16, at V = 4 in FP32): base and row stride have to allow it.
    auto ok = [](const void *p, int64_t ld, size_t elem, int v) {
        const size_t bytes = elem * (size_t)v > 16 ? 16 : elem * (size_t)v;
        return p == nullptr || (reinterpret_cast<uintptr_t>(p) % bytes == 0 && ((size_t)ld * elem) % bytes == 0);
    };
    auto fits = [&](int v) {
        return a.K % v == 0 && ok(a.x, a.ldx, sizeof(T), v) && ok(a.residual, a.ldr, sizeof(T), v) &&
               ok(a.h, a.ldh, sizeof(T), v) && ok(a.y, a.ldy, sizeof(T), v) && ok(a.q, a.ldq, 1, v) &&
               ok(a.weight, 0, 4, v);
    };
    if (a.K <= 16384 && fits(8)) return launch_v<T, 8>(a);
    if (a.K <= 16384 && fits(4)) return launch_v<T, 4>(a);
    if (a.K <= 8192) return launch_v<T, 1>(a);
    return launch_rows_pdl(q8_rows_long_kernel<T>, dim3((unsigned)a.M), 1024, a.stream, a.K,
                           (const T *)a.x, a.ldx, (const T *)a.residual, a.ldr, a.weight, a.eps,
                           (T *)a.h, a.ldh, (T *)a.y, a.ldy, a.q, a.ldq, a.scale);
}

}  // namespace

cudaError_t launch_q8_rows(const Q8RowsArgs &a) {
    return a.type == kTypeBf16 ? launch_t<__nv_bfloat16>(a) : launch_t<float>(a);
}

}  // namespace sgemm_gb300
