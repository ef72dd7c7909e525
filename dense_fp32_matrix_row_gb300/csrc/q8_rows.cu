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
// once.  A row stays in registers between its reduction and its stores.  Which
// kernel a call runs:
//   q8_rows_warp   rows of at most 64 vectors, many of them: a warp a row, no
//                  block barriers (at 128 vectors both take 20 us for 16384 rows);
//   q8_rows, q8_plain  longer rows, few rows, any alignment: a block a row, all its
//                  loads issued at once (q8_plain without norm and residual);
//   q8_rows_long   rows beyond registers (16384, or 8192 without vector access): read
//                  twice, an element at a time.
// Measured (bf16): 8192 x 4096 with residual, h and y, 302 MB, 46.9 us, 6.4 TB/s,
// memory; 2048 x 14336 alone, 88 MB, 15.0 us, 5.9 TB/s, the same; one row of 4096
// 2.3 us, the launch.  Not taken further: 2048 x 28672, 176 MB, 118 us alone and 126 with
// a norm (1.4 TB/s, q8_rows_long); 2048 x 8191 22 and 61 us (an element an access).
// Measured and not kept for long rows (8192 x 4096, 4096 x 8192 in FP32, 2048 x
// 16384, with residual: 39, 70 and 45 us with a block a row): persistent blocks
// that prefetch the next row into registers 46, 89 and 44 us, into shared memory
// with bulk copies 49, 122 and 64 us.
#include "q8.cuh"

namespace sgemm_gb300 {
namespace {

// V elements as they come from memory, in one aligned access (two for 32 bytes).
template <typename T, int V>
struct Raw {
    static constexpr int WORDS = V * (int)sizeof(T) / 4;
    uint32_t w[WORDS];
    __device__ __forceinline__ void load(const T *p) {
        if constexpr (WORDS >= 4) {
#pragma unroll
            for (int i = 0; i < WORDS / 4; ++i) {
                const uint4 u = reinterpret_cast<const uint4 *>(p)[i];
                w[4 * i] = u.x; w[4 * i + 1] = u.y; w[4 * i + 2] = u.z; w[4 * i + 3] = u.w;
            }
        } else {
            const uint2 u = *reinterpret_cast<const uint2 *>(p);
            w[0] = u.x; w[1] = u.y;
        }
    }
    __device__ __forceinline__ float operator[](int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else return __uint_as_float((i & 1) ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
    }
};
template <typename T>
struct Raw<T, 1> {
    T v;
    __device__ __forceinline__ void load(const T *p) { v = *p; }
    __device__ __forceinline__ float operator[](int) const { return to_f32<T>(v); }
};

// The largest |value| of some vectors, as FP32 bits.  BF16 values are the upper
// halves of FP32 ones and are compared two at a time.
template <typename T, int V, int NV>
__device__ __forceinline__ uint32_t raw_max(const Raw<T, V> (&r)[NV]) {
    uint32_t mx = 0;
    if constexpr (sizeof(T) == 2 && V > 1) {
        uint32_t m2 = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int k = 0; k < V / 2; ++k) m2 = __vmaxu2(m2, r[i].w[k] & 0x7fff7fffu);
        mx = max(m2 << 16, m2 & 0xffff0000u);
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < V; ++e) mx = max(mx, abs_bits(r[i][e]));
    }
    return mx;
}

// The arrays of a call, and what happens to one row once its sums are known.
template <typename T>
struct Rows {
    int64_t M, K;
    const T *x;
    int64_t ldx;
    const T *residual;
    int64_t ldr;
    const float *weight;
    float eps;
    T *h;
    int64_t ldh;
    T *y;
    int64_t ldy;
    int8_t *q;
    int64_t ldq;
    float *scale;
};

// One vector's part in the row's sums: v = x (+ residual), h stored, the largest
// |p| and the sum of squares extended.
template <typename T, int V>
__device__ __forceinline__ void take_vector(const Rows<T> &a, int64_t row, int c, float (&v)[V], uint32_t &mx,
                                            float &ss) {
    if (a.h) store_vec<T, V>(a.h + row * a.ldh + (int64_t)c * V, v);
    if (a.weight) {
        float w[V];
        load_vec<float, V>(a.weight + (int64_t)c * V, w);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            ss = fmaf(v[e], v[e], ss);
            mx = max(mx, abs_bits(v[e] * w[e]));
        }
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e) mx = max(mx, abs_bits(v[e]));
    }
}

// The row's results from its vectors c = first, first + step, ... in registers;
// `reduce` sums over the threads that share the row.
template <typename T, int V, int NV, typename Reduce>
__device__ __forceinline__ void finish_row(const Rows<T> &a, int64_t row, int first, int step, float (&v)[NV][V],
                                           uint32_t mx, float ss, Reduce reduce) {
    const int nvec = (int)(a.K / V);
    const RowQuant rq(mx);
    float r = 1.0f, lift = 1.0f;
    if (a.weight) {
        r = inv_rms(ss, a.K, a.eps);   // 0 for an infinite row, NaN for one with a NaN
        lift = norm_lift(ss, a.K, a.eps, mx);
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
            reduce(none, s2);
            r = inv_rms(s2, a.K, a.eps * lift * lift);
        }
    }
    if (first == 0) a.scale[row] = row_scale(rq, lift, r);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = first + i * step;
        if (c < nvec) {
            if (a.weight) {
                float w[V];
                load_vec<float, V>(a.weight + (int64_t)c * V, w);
#pragma unroll
                for (int e = 0; e < V; ++e) v[i][e] *= w[e];
                if (a.y) {
                    float t[V];
#pragma unroll
                    for (int e = 0; e < V; ++e) t[e] = lift == 1.0f ? v[i][e] * r : v[i][e] * lift * r;
                    store_vec<T, V>(a.y + row * a.ldy + (int64_t)c * V, t);
                }
            }
            store_q<V>(a.q + row * a.ldq + (int64_t)c * V, rq, v[i]);
        }
    }
}

// A row's vectors straight from memory, all loads issued before the first use.
template <typename T, int V, int NV>
__device__ __forceinline__ void load_row(const Rows<T> &a, int64_t row, int first, int step, float (&v)[NV][V],
                                         uint32_t &mx, float &ss) {
    const int nvec = (int)(a.K / V);
    Raw<T, V> rx[NV], rr[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = first + i * step;
        if (c < nvec) {
            rx[i].load(a.x + row * a.ldx + (int64_t)c * V);
            if (a.residual) rr[i].load(a.residual + row * a.ldr + (int64_t)c * V);
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = first + i * step;
#pragma unroll
        for (int e = 0; e < V; ++e) v[i][e] = 0.0f;
        if (c < nvec) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                v[i][e] = rx[i][e];
                if (a.residual) v[i][e] += rr[i][e];
            }
            take_vector<T, V>(a, row, c, v[i], mx, ss);
        }
    }
}

// A block per row.
template <typename T, int V, int NV>
__global__ void __launch_bounds__(512) q8_rows_kernel(const Rows<T> a) {
    __shared__ uint32_t red[64];
    pdl_wait();
    float v[NV][V];
    uint32_t mx = 0;
    float ss = 0.0f;
    load_row<T, V, NV>(a, blockIdx.x, threadIdx.x, blockDim.x, v, mx, ss);
    block_max_sum(mx, ss, red);
    finish_row<T, V, NV>(a, blockIdx.x, threadIdx.x, blockDim.x, v, mx, ss,
                         [&](uint32_t &m, float &s) { block_max_sum(m, s, red); });
}

// A warp per row.
constexpr int WARP_ROWS = 8;    // warps of a block
template <typename T, int V, int NV>
__global__ void __launch_bounds__(WARP_ROWS * 32, 4) q8_rows_warp_kernel(const Rows<T> a) {
    pdl_wait();
    const int lane = threadIdx.x & 31;
    auto reduce = [](uint32_t &m, float &s) {
        m = __reduce_max_sync(0xffffffffu, m);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    };
    for (int64_t row = (int64_t)blockIdx.x * WARP_ROWS + (threadIdx.x >> 5); row < a.M; row += (int64_t)gridDim.x * WARP_ROWS) {
        float v[NV][V];
        uint32_t mx = 0;
        float ss = 0.0f;
        load_row<T, V, NV>(a, row, lane, 32, v, mx, ss);
        reduce(mx, ss);
        finish_row<T, V, NV>(a, row, lane, 32, v, mx, ss, reduce);
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
            r = inv_rms(s2, K, eps * lift * lift);
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

// A block per row without a norm or a residual: the row waits for its maximum in the
// type it came in (2048 x 14336 in bf16 21.4 us in FP32 registers, 15.0 so).
template <typename T, int V, int NV>
__global__ void __launch_bounds__(512) q8_plain_kernel(int64_t K, const T *__restrict__ x, int64_t ldx,
                                                       int8_t *__restrict__ q, int64_t ldq, float *__restrict__ scale) {
    __shared__ uint32_t red[64];
    pdl_wait();
    const int nvec = (int)(K / V);
    const T *xr = x + (int64_t)blockIdx.x * ldx;
    Raw<T, V> r[NV] = {};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (int)(threadIdx.x + i * blockDim.x);
        if (c < nvec) r[i].load(xr + (int64_t)c * V);
    }
    uint32_t mx = raw_max<T, V, NV>(r);
    float none = 0.0f;
    block_max_sum(mx, none, red);
    const RowQuant rq(mx);
    if (threadIdx.x == 0) scale[blockIdx.x] = row_scale(rq, 1.0f, 1.0f);
    int8_t *qr = q + (int64_t)blockIdx.x * ldq;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (int)(threadIdx.x + i * blockDim.x);
        float v[V];
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = r[i][e];
        if (c < nvec) store_q<V>(qr + (int64_t)c * V, rq, v);
    }
}

template <typename K, typename... A>
cudaError_t launch_rows_pdl(K kern, dim3 grid, int threads, size_t smem, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <typename T>
Rows<T> rows_of(const Q8RowsArgs &a) {
    return {a.M, a.K, (const T *)a.x, a.ldx, (const T *)a.residual, a.ldr, a.weight, a.eps, (T *)a.h, a.ldh,
            (T *)a.y, a.ldy, a.q, a.ldq, a.scale};
}

// Vectors per thread: the fewest, from `from` on, that `most` threads a row allow; 0
// if it takes more than `last`.
int vectors_per_thread(int64_t nvec, int most, int from, int last) {
    for (int nv = from; nv <= last; nv *= 2)
        if (nvec <= (int64_t)most * nv) return nv;
    return 0;
}
// A block's share.  Few rows: as many threads as there are.  Otherwise a thread keeps
// several loads in flight, which counts for more than threads do, up to 32 words of
// input without a norm and 4 vectors with one.
//   vectors a thread          1     2     4     8    16
//   no norm, 8192 x 4096     24.2  17.8  16.0
//     2048 x 14336                       15.7  15.0  19.0
//     the same in FP32                   23.4  25.4  30.9
//   norm, 8192 x 2048        24.4  21.7
//     8192 x 4096 with y     51.6  46.9  48.2
//     1001 x 4092 in FP32          7.4   6.4   8.2
//     2048 x 14336                       38.9  50.9  68.6
// (us, bf16 unless said; with residual but for FP32)
int block_vectors(int64_t nvec, bool norm, bool few_rows, int words_of_vector) {
    if (few_rows) return vectors_per_thread(nvec, 512, 1, 16);
    const int cap = norm ? 4 : words_of_vector > 2 ? 32 / words_of_vector : 16;
    const int nv = norm ? vectors_per_thread(nvec, 256, 2, cap) : vectors_per_thread(nvec, 128, 1, cap);
    return nv ? nv : vectors_per_thread(nvec, 512, cap, 16);
}
int threads_for(int64_t nvec, int nv) {
    const int t = (int)(((nvec + nv - 1) / nv + 31) / 32 * 32);
    return t < 32 ? 32 : t;
}

template <typename T, int V>
cudaError_t launch_block(const Q8RowsArgs &a) {
    const int64_t nvec = a.K / V;
    const int nv = block_vectors(nvec, a.weight != nullptr, a.M <= 2 * (int64_t)a.sm_count, (V * (int)sizeof(T) + 3) / 4);
    const int threads = threads_for(nvec, nv);
    const dim3 grid((unsigned)a.M);
    if (a.weight == nullptr) {
        const T *x = (const T *)a.x;
        auto run = [&](auto kernel) {
            return launch_rows_pdl(kernel, grid, threads, 0, a.stream, a.K, x, a.ldx, a.q, a.ldq, a.scale);
        };
        switch (nv) {
            case 1: return run(q8_plain_kernel<T, V, 1>);
            case 2: return run(q8_plain_kernel<T, V, 2>);
            case 4: return run(q8_plain_kernel<T, V, 4>);
            default: break;
        }
        if constexpr (V * sizeof(T) <= 16) {
            if (nv == 8) return run(q8_plain_kernel<T, V, 8>);
        }
        if constexpr (V * sizeof(T) <= 8) {
            if (nv == 16) return run(q8_plain_kernel<T, V, 16>);
        }
        return cudaErrorInvalidValue;
    }
    const Rows<T> r = rows_of<T>(a);
    switch (nv) {
        case 1: return launch_rows_pdl(q8_rows_kernel<T, V, 1>, grid, threads, 0, a.stream, r);
        case 2: return launch_rows_pdl(q8_rows_kernel<T, V, 2>, grid, threads, 0, a.stream, r);
        case 4: return launch_rows_pdl(q8_rows_kernel<T, V, 4>, grid, threads, 0, a.stream, r);
        default: break;
    }
    if constexpr (V <= 4) {
        if (nv == 8) return launch_rows_pdl(q8_rows_kernel<T, V, 8>, grid, threads, 0, a.stream, r);
    }
    if constexpr (V == 1) {
        if (nv == 16) return launch_rows_pdl(q8_rows_kernel<T, V, 16>, grid, threads, 0, a.stream, r);
    }
    return cudaErrorInvalidValue;
}

template <typename T, int V>
cudaError_t launch_warp(const Q8RowsArgs &a) {
    const int64_t blocks = (a.M + WARP_ROWS - 1) / WARP_ROWS, most = (int64_t)a.sm_count * 8;
    const dim3 grid((unsigned)(blocks < most ? blocks : most));
    const Rows<T> r = rows_of<T>(a);
    switch (vectors_per_thread(a.K / V, 32, 1, 2)) {
        case 1: return launch_rows_pdl(q8_rows_warp_kernel<T, V, 1>, grid, WARP_ROWS * 32, 0, a.stream, r);
        default: return launch_rows_pdl(q8_rows_warp_kernel<T, V, 2>, grid, WARP_ROWS * 32, 0, a.stream, r);
    }
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
    constexpr int V16 = 16 / (int)sizeof(T);       // elements of a 16-byte access
    if (a.K > 0 && a.K <= 64 * V16 && fits(V16) && a.M > 2 * (int64_t)a.sm_count) return launch_warp<T, V16>(a);
    if (a.K <= 16384 && fits(8)) return launch_block<T, 8>(a);
    if (a.K <= 16384 && fits(4)) return launch_block<T, 4>(a);
    if (a.K <= 8192) return launch_block<T, 1>(a);
    return launch_rows_pdl(q8_rows_long_kernel<T>, dim3((unsigned)a.M), 1024, 0, a.stream, a.K,
                           (const T *)a.x, a.ldx, (const T *)a.residual, a.ldr, a.weight, a.eps,
                           (T *)a.h, a.ldh, (T *)a.y, a.ldy, a.q, a.ldq, a.scale);
}

}  // namespace

cudaError_t launch_q8_rows(const Q8RowsArgs &a) {
    return a.type == kTypeBf16 ? launch_t<__nv_bfloat16>(a) : launch_t<float>(a);
}

}  // namespace sgemm_gb300
