// q8_stream.cu -- 8-bit linear product for a few tokens, by streaming W:
//
//     C[m][n] = act(xs[m] * ws[n] * sum_k X[m][k] * W[n][k] + bias[n])
//
// Bound by memory: every byte of W is read once per block of up to 16 tokens.
// Both kernels multiply with mma.sync (see q8_stream.cuh): the tensor rate
// that takes is well below what the kernel's bytes leave time for, so tensor
// memory would gain nothing here.
//
// q8_ring_kernel (W 16-byte aligned) is persistent, one block per SM: a
// producer warp keeps 130 to 200 KB of bulk copies in flight, across tile ends too,
// which no block-per-tile form does; sixteen warps share each stage and add
// their integer sums in shared memory.  q8_stream_kernel takes any alignment.
//
// Measured at 14336 x 4096 (58.7 MB of W): 12.6 us for one token (4.7 TB/s; the
// launch and the ring's filling are 4 of them: 57344 x 4096 streams at 6.0 TB/s),
// 13.8 up to 8 tokens, 17.9 for 16, where the expansion to FP16 and its MMAs
// have the same length as the copies.  With W at an odd address, q8_stream_kernel takes
// 29 us for one token (2.0 TB/s), 32 for 4 and 44 for 16; 1 x 4096 x 4095 9.5 us.
#include "q8_stream.cuh"

namespace sgemm_gb300 {
namespace {

constexpr int SWARPS = 8;

template <int NB, typename OutT>
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
    pdl_wait();
    // a grid has 65535 blocks in y at most: beyond, a block takes several blocks of tokens
    for (int64_t first = (int64_t)blockIdx.y * TOK; first < M; first += (int64_t)gridDim.y * TOK) {
        const int m0 = (int)first;
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
            q8_dot<NB, 4>(sum, W + (int64_t)ra * ldw, W + (int64_t)rb * ldw, x, K, s0, s1, W,
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
            const float v = K > 0 ? (float)s * xs[m] * ws[n] : 0.0f;
            C[(int64_t)m * ldc + n] = from_f32<OutT>(epilogue_tail(ep, v, n));
        }
        __syncthreads();   // `part` is written again
    }
}

// ---- the ring ------------------------------------------------------------------

constexpr uint64_t DRAIN_NS = 1000000000ull;
// NB blocks of 8 tokens; RT 16-row tiles per stage, RW of them per warp.  DP > 0: at
// most DP tokens, by dp4a.
template <int DP_, int NB_, int RT_, int RW_, int STEPS_, int RING_>
struct RingCfg {
    using S = Q8Stage<RT_, RW_, STEPS_>;
    static constexpr int DP = DP_, NB = NB_, RT = RT_, RW = RW_, RING = RING_;
    static constexpr int XN = DP > 0 ? DP : NB;                      // token rows a lane reads
    static_assert(DP == 0 || (NB == 1 && RW == 1 && DP <= 8), "dp4a takes one block of tokens");
    static constexpr int TOK = NB * 8, TILE = S::ROWS * TOK;
    static constexpr int THREADS = (kQ8Consumers + RT) * 32;         // RT producer warps
    static constexpr int PART = kQ8Consumers * RW * NB * 32;         // int4 of one tile's sums
    static constexpr size_t SMEM = 128 + (size_t)RING * S::BYTES + 2 * (size_t)PART * 16 + 256;
    static_assert(SMEM <= 227 * 1024, "shared memory per block");
};

template <typename C, typename OutT>
__global__ void __launch_bounds__(C::THREADS, 1)
q8_ring_kernel(int M, int N, int K, const int8_t *__restrict__ X,
               int64_t ldx, int xvec, const float *__restrict__ xs, const int8_t *__restrict__ W, int64_t ldw,
               const float *__restrict__ ws, Epilogue ep, OutT *__restrict__ out, int64_t ldc, unsigned *err,
               uint64_t wait_ns) {
    using S = typename C::S;
    constexpr int DP = C::DP, XN = C::XN, NB = C::NB, RT = C::RT, RW = C::RW, RING = C::RING;
    constexpr int TOK = C::TOK, ROWS = S::ROWS, KB = S::KB, KW = S::KW, STEPS = S::STEPS;
    extern __shared__ unsigned char smem_raw[];
    const uintptr_t base = (reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127);
    unsigned char *ring = reinterpret_cast<unsigned char *>(base);
    int4 *sums = reinterpret_cast<int4 *>(ring + (size_t)RING * S::BYTES);   // [2][warp][RW][NB][lane]
    uint64_t *full = reinterpret_cast<uint64_t *>(sums + 2 * C::PART);
    uint64_t *empty = full + RING;
    uint64_t *tdone = empty + RING;                       // [2] all warps have added their sums
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int blocks = K / kQ8Step;                       // whole steps; the rest is read directly
    const int stages = (blocks + KB - 1) / KB;            // per tile
    const int tiles = groups_of(N, ROWS);
    const int m0 = (int)blockIdx.y * TOK;

    if (threadIdx.x == 0) {
        for (int s = 0; s < RING; ++s) {
            mbar_init(smem_u32(&full[s]), RT);
            mbar_init(smem_u32(&empty[s]), kQ8Consumers);
        }
        mbar_init(smem_u32(&tdone[0]), kQ8Consumers);
        mbar_init(smem_u32(&tdone[1]), kQ8Consumers);
        mbar_fence_init();
    }
    __syncthreads();
    pdl_wait();

    if (warp >= kQ8Consumers) {
        const int first = (warp - kQ8Consumers) * 16;   // this producer's rows of the stage
        bool ok = true;
        uint32_t g = 0;
        for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x)
            for (int s = 0; s < stages; ++s, ++g) {
                const int r = (int)(g % RING);
                if (g >= (uint32_t)RING && !warp_wait(smem_u32(&empty[r]), (g / RING - 1) & 1, wait_ns)) {
                    ok = false;
                    break;
                }
                const uint32_t bar = smem_u32(&full[r]);
                const uint32_t bytes = (uint32_t)min(KB, blocks - s * KB) * kQ8Step;
                if (lane == 0) mbar_arrive_expect_tx(bar, bytes * 16);
                __syncwarp();
                // rows past N read the last one; their results are dropped
                if (lane < 16)
                    bulk_load(smem_u32(ring + (size_t)r * S::BYTES) + (uint32_t)(first + lane) * S::LD,
                              W + (int64_t)min(t * ROWS + first + lane, N - 1) * ldw + (int64_t)s * (KB * kQ8Step),
                              bytes, bar);
                __syncwarp();
            }
        // The block may not end before its copies have landed, whichever warp gave up.
        // (Otherwise they have been waited for already, or are about to be.)
        if (lane == 0) {
            if (!ok) record_error(err, kErrWaitTimeout);
            for (uint32_t q = g > (uint32_t)RING ? g - RING : 0; q < g; ++q)
                mbar_wait(smem_u32(&full[q % RING]), (q / RING) & 1, DRAIN_NS);
        }
        return;
    }

    const int g = lane >> 2, t4 = lane & 3;
    const int rt = warp / KW * RW, kpart = warp % KW;   // first row tile, share of the steps
    const int8_t *x[XN];
#pragma unroll
    for (int n = 0; n < XN; ++n) x[n] = X + (int64_t)min(m0 + (DP > 0 ? n : 8 * n + g), M - 1) * ldx + 16 * t4;
    const int8_t *xend = X + (int64_t)(M - 1) * ldx + K;
    // this lane's 16 bytes of rows g and g + 8 in the warp's first step
    const uint32_t wa = (uint32_t)(rt * 16 + g) * S::LD + (uint32_t)(kpart * STEPS * kQ8Step + 16 * t4);
    const uint32_t wb = wa + 8 * S::LD;
    // tokens do not depend on the tile: the same steps come round every time
    uint4 xnext[STEPS][XN];
    auto xload = [&](int u, int step) {
#pragma unroll
        for (int n = 0; n < XN; ++n) {
            const int8_t *p = x[n] + (int64_t)step * kQ8Step;
            if (step < blocks)
                xnext[u][n] = xvec ? __ldg(reinterpret_cast<const uint4 *>(p)) : load16_unaligned(p, X, xend);
        }
    };
#pragma unroll
    for (int u = 0; u < STEPS; ++u) {
#pragma unroll
        for (int n = 0; n < XN; ++n) xnext[u][n] = make_uint4(0u, 0u, 0u, 0u);
        xload(u, kpart * STEPS + u);
    }
    uint32_t used = 0;      // stages read
    uint32_t count = 0;     // tiles finished
    for (int t = blockIdx.x; t < tiles; t += gridDim.x, ++count) {
        int sum[RW][NB][4], dsum[XN][2];
        float acc[RW][NB][4];
#pragma unroll
        for (int r = 0; r < RW; ++r)
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    sum[r][n][i] = 0;
                    acc[r][n][i] = 0.0f;
                }
#pragma unroll
        for (int j = 0; j < XN; ++j) dsum[j][0] = dsum[j][1] = 0;
        auto flush = [&] {
#pragma unroll
            for (int r = 0; r < RW; ++r) q8_flush<NB>(sum[r], acc[r]);
        };
        // This thread's results of the tile: word e of the sums' layout, where
        // words follow the fragments (lane, then 4 words: rows g, g, g + 8, g + 8,
        // tokens 2 t4, + 1, 2 t4, + 1).  Their scales are asked for now.
        constexpr int OUTS = C::TILE, PER = (OUTS + kQ8Consumers * 32 - 1) / (kQ8Consumers * 32);
        const int n0 = t * ROWS;
        auto place = [&](int e, int &row, int &tok) {
            const int i = e & 3, l = (e >> 2) & 31, frag = e >> 7;      // frag: (tile of the stage, token block)
            row = frag / NB * 16 + (l >> 2) + 8 * (i >> 1);
            tok = frag % NB * 8 + 2 * (l & 3) + (i & 1);
        };
        float sx[PER], sw[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            int row, tok;
            const int e = (int)threadIdx.x + i * kQ8Consumers * 32;
            place(e, row, tok);
            sx[i] = sw[i] = 0.0f;
            if (e < OUTS && n0 + row < N && m0 + tok < M) {
                sx[i] = __ldg(xs + m0 + tok);
                sw[i] = __ldg(ws + n0 + row);
            }
        }
        bool ok = true;
        for (int s = 0; s < stages; ++s, ++used) {
            const int b0 = s * KB + kpart * STEPS;
            const int nb = blocks - b0;                            // steps there are, from this warp's first
            const int bn = b0 - s * KB + (s + 1 < stages ? s + 1 : 0) * KB;   // the next stage's first
            const int r = (int)(used % RING);
            if (!warp_wait(smem_u32(&full[r]), (used / RING) & 1, wait_ns)) {
                ok = false;
                break;
            }
            const uint32_t stage = smem_u32(ring + (size_t)r * S::BYTES);
#pragma unroll
            for (int u = 0; u < STEPS; ++u) {
                if (u < nb) {
                    uint4 a[RW], b[RW];
#pragma unroll
                    for (int w = 0; w < RW; ++w) {
                        a[w] = lds128(stage + wa + (uint32_t)w * 16 * S::LD + (uint32_t)u * kQ8Step);
                        b[w] = lds128(stage + wb + (uint32_t)w * 16 * S::LD + (uint32_t)u * kQ8Step);
                    }
                    if constexpr (DP > 0) q8_step_dp<XN>(dsum, a[0], b[0], xnext[u]);
                    else if constexpr (NB == 1) q8_step_s8(sum[0][0], a[0], b[0], xnext[u][0]);
                    else q8_step_rows<RW, NB>(acc, a, b, xnext[u]);
                }
                xload(u, bn + u);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&empty[r]));
            if (NB > 1 && s % (kQ8ExactSteps / STEPS) == kQ8ExactSteps / STEPS - 1) flush();
        }
        if (!ok) {
            if (lane == 0) record_error(err, kErrWaitTimeout);
            return;
        }
        if (K % kQ8Step != 0 && kpart == 0) {   // the last values of each row
            const int valid = min(16, max(0, K - blocks * kQ8Step - 16 * t4));
            const int64_t k = (int64_t)blocks * kQ8Step + 16 * t4;
            uint4 xt[XN], a[RW], b[RW];
#pragma unroll
            for (int n = 0; n < XN; ++n) xt[n] = load16_bytes(x[n] + (int64_t)blocks * kQ8Step, valid);
#pragma unroll
            for (int w = 0; w < RW; ++w) {
                const int row = n0 + (rt + w) * 16 + g;
                a[w] = load16_bytes(W + (int64_t)min(row, N - 1) * ldw + k, valid);
                b[w] = load16_bytes(W + (int64_t)min(row + 8, N - 1) * ldw + k, valid);
            }
            if constexpr (DP > 0) {
                q8_step_dp<XN>(dsum, a[0], b[0], xt);
            } else if constexpr (NB == 1) {
                q8_step_s8(sum[0][0], a[0], b[0], xt[0]);
            } else {
                flush();      // a chunk of its own
                q8_step_rows<RW, NB>(acc, a, b, xt);
            }
        }
        flush();
        int4 *tile = sums + (count & 1) * C::PART;
        if constexpr (DP > 0) {
#pragma unroll
            for (int j = 0; j < XN; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    int v = dsum[j][i];
                    v += __shfl_xor_sync(0xffffffffu, v, 1);
                    v += __shfl_xor_sync(0xffffffffu, v, 2);
                    // one lane of the quad: where the MMA would leave (row, token j)
                    if (t4 == (j >> 1)) reinterpret_cast<int *>(tile + warp * 32 + lane)[2 * i + (j & 1)] = v;
                }
        } else {
#pragma unroll
            for (int w = 0; w < RW; ++w)
#pragma unroll
                for (int n = 0; n < NB; ++n)
                    tile[((warp * RW + w) * NB + n) * 32 + lane] =
                        make_int4(sum[w][n][0], sum[w][n][1], sum[w][n][2], sum[w][n][3]);
        }
        __syncwarp();
        const uint32_t bar = smem_u32(&tdone[count & 1]);
        if (lane == 0) mbar_arrive(bar);
        if (!warp_wait(bar, (count >> 1) & 1, wait_ns)) {
            if (lane == 0) record_error(err, kErrWaitTimeout);
            return;
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            int row, tok;
            const int e = (int)threadIdx.x + i * kQ8Consumers * 32;
            place(e, row, tok);
            const int n = n0 + row, m = m0 + tok;
            if (e < OUTS && n < N && m < M) {
                // the KW warps that share this tile's steps (whole numbers: any order)
                const int frag = e >> 7, rtile = frag / NB;
                const int *v = reinterpret_cast<const int *>(tile) +
                               ((rtile / RW * KW * RW + rtile % RW) * NB + frag % NB) * 128 + (e & 127);
                int total = 0;
#pragma unroll
                for (int w = 0; w < KW; ++w) total += v[w * RW * NB * 128];
                out[(int64_t)m * ldc + n] = from_f32<OutT>(epilogue_tail(ep, (float)total * sx[i] * sw[i], n));
            }
        }
    }
}

template <int NB, typename OutT>
cudaError_t launch_s(const Q8LinearArgs &a) {
    const int64_t steps = (a.K + kQ8Step - 1) / kQ8Step;
    int kw = 1;
    while (kw < SWARPS && steps >= 8 * kw) kw *= 2;   // at least 4 steps a warp
    const int64_t rows = 16 * (SWARPS / kw);
    const int64_t mb = (a.M + NB * 8 - 1) / (NB * 8);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.N + rows - 1) / rows), (unsigned)(mb < 65535 ? mb : 65535), 1);
    cfg.blockDim = dim3(SWARPS * 32, 1, 1);
    cfg.stream = a.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const Epilogue ep{1.0f, 0.0f, a.bias, a.act};
    return cudaLaunchKernelEx(&cfg, q8_stream_kernel<NB, OutT>, (int)a.M, (int)a.N, (int)a.K, a.X,
                              a.ldx, a.xs, a.W, a.ldw, a.ws, ep, (OutT *)a.C, a.ldc, kw);
}

template <typename C, typename OutT>
cudaError_t launch_ring(const Q8LinearArgs &a) {
    auto kern = q8_ring_kernel<C, OutT>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
    if (e != cudaSuccess) return e;
    const int64_t tiles = (a.N + C::S::ROWS - 1) / C::S::ROWS, mb = (a.M + C::TOK - 1) / C::TOK;
    const int64_t sms = a.sm_count > 0 ? a.sm_count : 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles < sms ? tiles : sms), (unsigned)mb, 1);
    cfg.blockDim = dim3(C::THREADS, 1, 1);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = a.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const int xvec = reinterpret_cast<uintptr_t>(a.X) % 16 == 0 && a.ldx % 16 == 0;
    return cudaLaunchKernelEx(&cfg, kern, (int)a.M, (int)a.N, (int)a.K, a.X, a.ldx, xvec, a.xs, a.W, a.ldw, a.ws,
                              Epilogue{1.0f, 0.0f, a.bias, a.act}, (OutT *)a.C, a.ldc, a.err, a.wait_ns);
}

// Rows per stage: as many k as the row has, up to 4096 (1024 for 16 tokens).
template <int DP, typename OutT>
cudaError_t launch_8(const Q8LinearArgs &a) {
    if (a.K <= 1024) return launch_ring<RingCfg<DP, 1, 4, 1, 2, 5>, OutT>(a);
    if (a.K <= 2048) return launch_ring<RingCfg<DP, 1, 2, 1, 4, 3>, OutT>(a);
    return launch_ring<RingCfg<DP, 1, 1, 1, 4, 3>, OutT>(a);
}

template <typename OutT>
cudaError_t launch_r(const Q8LinearArgs &a) {
    if (a.M == 1) return launch_8<1, OutT>(a);
    if (a.M <= 8) return launch_8<0, OutT>(a);
    return launch_ring<RingCfg<0, 2, 2, 2, 1, 4>, OutT>(a);
}

template <typename OutT>
cudaError_t launch_o(const Q8LinearArgs &a) {
    const bool wvec = reinterpret_cast<uintptr_t>(a.W) % 16 == 0 && a.ldw % 16 == 0;
    if (wvec && a.K >= kQ8Step && (a.M + 7) / 8 <= 65535) return launch_r<OutT>(a);
    return a.M <= 8 ? launch_s<1, OutT>(a) : launch_s<2, OutT>(a);
}

}  // namespace

cudaError_t launch_q8_stream(const Q8LinearArgs &a) {
    return a.type == kTypeBf16 ? launch_o<__nv_bfloat16>(a) : launch_o<float>(a);
}

}  // namespace sgemm_gb300
