// q8_stream.cu -- 8-bit linear product by streaming W past a few token rows:
//
//     C[m][n] = act(xs[m] * ws[n] * sum_k X[m][k] * W[n][k] + bias[n])
//
// Bound by memory: every byte of W is read once per block of 16 tokens.  A
// warp takes 16 rows of W (see q8_stream.cuh); `kw` warps of a block divide K
// and their integer sums meet in shared memory, so the result does not depend
// on the division.  Any alignment and stride.
#include "q8_stream.cuh"

namespace sgemm_gb300 {
namespace {

constexpr int SWARPS = 8;

template <int NB, bool VEC, typename OutT>
__global__ void __launch_bounds__(SWARPS * 32)
q8_stream_kernel(int M, int N, int K, const int8_t *__restrict__ X, int64_t ldx,
                 const float *__restrict__ xs, const int8_t *__restrict__ W, int64_t ldw,
                 const float *__restrict__ ws, Epilogue ep, OutT *__restrict__ C, int64_t ldc, int kw) {
    constexpr int TOK = NB * 8;
    __shared__ int part[SWARPS][16][TOK + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const int rt = SWARPS / kw;                     // 16-row tiles per block
    const int tile = warp / kw, kpart = warp % kw;
    const int n0 = ((int)blockIdx.x * rt + tile) * 16;
    const int m0 = (int)blockIdx.y * TOK;
    pdl_wait();
    int sum[NB][4];
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[n][i] = 0;
    if (n0 < N) {
        // rows past N and tokens past M read the last one; their results are dropped
        const int ra = min(n0 + g, N - 1), rb = min(n0 + g + 8, N - 1);
        const int8_t *x[NB];
#pragma unroll
        for (int n = 0; n < NB; ++n) x[n] = X + (int64_t)min(m0 + 8 * n + g, M - 1) * ldx;
        const int steps = (K + kQ8Step - 1) / kQ8Step;
        const int per = (steps + kw - 1) / kw;
        const int s0 = min(kpart * per, steps), s1 = min(s0 + per, steps);
        q8_dot<NB, VEC, 4>(sum, W + (int64_t)ra * ldw, W + (int64_t)rb * ldw, x, K, s0, s1, W,
                           W + (int64_t)(N - 1) * ldw + K, X, X + (int64_t)(M - 1) * ldx + K);
    }
#pragma unroll
    for (int n = 0; n < NB; ++n) {
        part[warp][g][8 * n + 2 * t] = sum[n][0];
        part[warp][g][8 * n + 2 * t + 1] = sum[n][1];
        part[warp][g + 8][8 * n + 2 * t] = sum[n][2];
        part[warp][g + 8][8 * n + 2 * t + 1] = sum[n][3];
    }
    __syncthreads();
    for (int o = threadIdx.x; o < rt * 16 * TOK; o += SWARPS * 32) {
        const int row = o % 16, tl = (o / 16) % rt, tok = o / (16 * rt);
        const int n = ((int)blockIdx.x * rt + tl) * 16 + row, m = m0 + tok;
        if (n >= N || m >= M) continue;
        int s = 0;
        for (int w = 0; w < kw; ++w) s += part[tl * kw + w][row][tok];
        const float v = (float)s * xs[m] * ws[n];
        C[(int64_t)m * ldc + n] = from_f32<OutT>(epilogue_tail(ep, v, n));
    }
}

template <int NB, bool VEC, typename OutT>
cudaError_t launch_s(const Q8LinearArgs &a) {
    const int64_t steps = (a.K + kQ8Step - 1) / kQ8Step;
    int kw = 1;
    while (kw < SWARPS && steps >= 8 * kw) kw *= 2;   // at least 4 steps a warp
    const int64_t rows = 16 * (SWARPS / kw);
    const int64_t mb = (a.M + NB * 8 - 1) / (NB * 8);
    if (mb > 65535) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.N + rows - 1) / rows), (unsigned)mb, 1);
    cfg.blockDim = dim3(SWARPS * 32, 1, 1);
    cfg.stream = a.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const Epilogue ep{1.0f, 0.0f, a.bias, a.act};
    return cudaLaunchKernelEx(&cfg, q8_stream_kernel<NB, VEC, OutT>, (int)a.M, (int)a.N, (int)a.K, a.X,
                              a.ldx, a.xs, a.W, a.ldw, a.ws, ep, (OutT *)a.C, a.ldc, kw);
}

template <typename OutT>
cudaError_t launch_o(const Q8LinearArgs &a) {
    const bool vec = reinterpret_cast<uintptr_t>(a.X) % 16 == 0 && a.ldx % 16 == 0 &&
                     reinterpret_cast<uintptr_t>(a.W) % 16 == 0 && a.ldw % 16 == 0;
    if (a.M <= 8) return vec ? launch_s<1, true, OutT>(a) : launch_s<1, false, OutT>(a);
    return vec ? launch_s<2, true, OutT>(a) : launch_s<2, false, OutT>(a);
}

}  // namespace

cudaError_t launch_q8_stream(const Q8LinearArgs &a) {
    return a.type == kTypeBf16 ? launch_o<__nv_bfloat16>(a) : launch_o<float>(a);
}

}  // namespace sgemm_gb300
