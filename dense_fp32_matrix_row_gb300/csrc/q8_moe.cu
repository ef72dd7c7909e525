// q8_moe.cu -- a whole mixture-of-experts layer for a few tokens, with 8-bit
// expert weights, in two kernels.
//
//   logits[t][e] = sum_h x[t][h] * router[e][h]                (FP32)
//   the top_k experts of each token by logit (ties: the lowest index), their
//   gates softmax over all experts, or over the chosen ones (renormalize)
//   xq, xs = 8-bit rows of x (as in q8_rows.cu)
//   g, u   = xs[t] * s_up[e][.] * (xq[t] . w_up[e][.])         rows [0, I), [I, 2I)
//   hid    = g / (1 + exp(-g)) * u,   hq, hs = 8-bit rows of hid
//   out[t] = sum_j gate_j * hs * s_down[e_j][.] * (hq . w_down[e_j][.])
//
// Bound by memory: the picked experts' weights, read once each (a block of up
// to 16 of an expert's tokens shares the read).
//
// The first kernel computes the logits and quantises the tokens.  The second
// is persistent: blocks draw work units from one counter, all gate/up units
// first, then all down units.  A down unit waits (bounded) until its expert's
// hidden rows are there; since every gate/up unit has been drawn by then, by
// a block that waits for nothing, that wait always ends, whatever else runs
// on the GPU.  The block that finishes an expert's last gate/up unit turns
// the hidden rows into 8 bits, and the one that finishes the last down unit
// of an output range adds the experts' results, in slot order: nothing
// depends on timing, and results repeat bit for bit.
#include "q8_stream.cuh"

namespace sgemm_gb300 {
namespace {

constexpr int RTHREADS = 256;
constexpr int MWARPS = 8, MTHREADS = MWARPS * 32;
constexpr int kMaxPairs = kMoeMaxTokens * kMoeMaxTopK;

// The layer's workspace: byte offsets of its arrays.
struct MoeLayout {
    int P, Hp, Ip, dmax;      // pairs (token, slot); row strides; down groups at most
    size_t logits, xs, xq, hidden, hs, hq, part, zero, total;
    int nzero;                // words to clear: ticket, ready[P], flag[P], hmax[P], done[dmax]
    __host__ __device__ MoeLayout(int T, int E, int top_k, int H, int I) {
        P = T * top_k;
        Hp = (H + kQ8Step - 1) / kQ8Step * kQ8Step;
        Ip = (I + kQ8Step - 1) / kQ8Step * kQ8Step;
        dmax = (H + 15) / 16;
        size_t at = 0;
        auto take = [&](size_t bytes) {
            const size_t o = at;
            at += (bytes + 255) / 256 * 256;
            return o;
        };
        logits = take((size_t)T * E * 4);
        xs = take((size_t)T * 4);
        xq = take((size_t)T * Hp);
        hidden = take((size_t)P * I * 4);
        hs = take((size_t)P * 4);
        hq = take((size_t)P * Ip);
        part = take((size_t)P * H * 4);
        nzero = 1 + 3 * P + dmax;
        zero = take((size_t)nzero * 4);
        total = at;
    }
};

// Blocks 0 .. E-1: one expert's logits for every token.  Blocks E .. E+T-1:
// one token's 8-bit row; the first of them also clears the second kernel's
// counters.
template <typename T>
__global__ void __launch_bounds__(RTHREADS)
q8_route_kernel(int ntok, int E, int top_k, int H, int I, const T *__restrict__ x, int64_t ldx,
                const float *__restrict__ router, int64_t ldr, unsigned char *__restrict__ ws) {
    __shared__ uint32_t red[64];
    __shared__ float lsum[RTHREADS / 32][8];
    const MoeLayout L(ntok, E, top_k, H, I);
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if ((int)blockIdx.x < E) {
        const int e = (int)blockIdx.x;
        const float *w = router + (int64_t)e * ldr;
        float *logits = reinterpret_cast<float *>(ws + L.logits);
        for (int t0 = 0; t0 < ntok; t0 += 8) {
            float acc[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
            for (int k = threadIdx.x; k < H; k += RTHREADS) {
                const float wk = __ldg(w + k);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (t0 + j < ntok) acc[j] = fmaf(to_f32<T>(x[(int64_t)(t0 + j) * ldx + k]), wk, acc[j]);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], o);
            __syncthreads();
            if (lane == 0)
#pragma unroll
                for (int j = 0; j < 8; ++j) lsum[warp][j] = acc[j];
            __syncthreads();
            if (threadIdx.x < 8 && t0 + (int)threadIdx.x < ntok) {
                float s = 0.0f;
#pragma unroll
                for (int v = 0; v < RTHREADS / 32; ++v) s += lsum[v][threadIdx.x];
                logits[(int64_t)(t0 + threadIdx.x) * E + e] = s;
            }
        }
        return;
    }
    const int t = (int)blockIdx.x - E;
    if (t == 0) {
        uint32_t *z = reinterpret_cast<uint32_t *>(ws + L.zero);
        for (int i = threadIdx.x; i < L.nzero; i += RTHREADS) z[i] = 0u;
    }
    const T *xr = x + (int64_t)t * ldx;
    uint32_t mx = 0;
    float none = 0.0f;
    for (int k = threadIdx.x; k < H; k += RTHREADS) mx = max(mx, abs_bits(to_f32<T>(xr[k])));
    block_max_sum(mx, none, red);
    const RowQuant rq(mx);
    int8_t *q = reinterpret_cast<int8_t *>(ws + L.xq) + (int64_t)t * L.Hp;
    for (int k = threadIdx.x; k < L.Hp; k += RTHREADS)
        q[k] = k < H ? (int8_t)rq(to_f32<T>(xr[k])) : (int8_t)0;
    if (threadIdx.x == 0) reinterpret_cast<float *>(ws + L.xs)[t] = rq.step * rq.unpre;
}

// Logits as unsigned numbers in the same order, every NaN above +inf and -0
// equal to +0; 0 is below all of them (a slot already taken).
__device__ __forceinline__ uint32_t logit_key(float v) {
    if (v != v) return 0xffffffffu;
    const uint32_t b = __float_as_uint(v + 0.0f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ uint32_t ld_acquire(const uint32_t *p) {
    uint32_t v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void st_release(uint32_t *p, uint32_t v) {
    asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

struct MoeShared {
    int ids[kMaxPairs];
    float gates[kMaxPairs];
    unsigned short list[kMaxPairs];      // pairs by expert, then by pair
    unsigned short chunk_e[kMaxPairs], chunk_at[kMaxPairs];
    unsigned char chunk_n[kMaxPairs];    // up to 16 pairs of one expert
    int count[kMoeMaxExperts];
    int first[kMoeMaxExperts], first_chunk[kMoeMaxExperts];
    int nchunks;
    int ticket[2];
    int flag;
    int part[MWARPS][16][17];
};

// The routing of all tokens, the same in every block: top_k experts and gates
// of each token, then each expert's pairs and their chunks of up to 16.
__device__ void moe_route(MoeShared &S, int ntok, int E, int top_k, int renorm, const float *logits) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int PER = kMoeMaxExperts / 32;
    for (int t = warp; t < ntok; t += MWARPS) {
        float l[PER];
        uint32_t key[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = lane + 32 * i;
            l[i] = e < E ? __ldg(logits + (int64_t)t * E + e) : 0.0f;
            key[i] = e < E ? logit_key(l[i]) : 0u;
        }
        float top = 0.0f, chosen = 0.0f, mine = 0.0f;
        int my_id = 0;
        for (int j = 0; j < top_k; ++j) {
            uint32_t best = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i) best = max(best, key[i]);
            best = __reduce_max_sync(0xffffffffu, best);
            uint32_t at = 0xffffffffu;     // the lowest index that holds it
#pragma unroll
            for (int i = PER - 1; i >= 0; --i)
                if (key[i] == best) at = (uint32_t)(lane + 32 * i);
            at = __reduce_min_sync(0xffffffffu, at);
            float v = 0.0f;
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if ((uint32_t)(lane + 32 * i) == at) {
                    v = l[i];
                    key[i] = 0u;
                }
            v = __shfl_sync(0xffffffffu, v, (int)(at & 31));
            if (j == 0) top = v;
            const float p = expf(v - top);
            chosen += p;
            if (lane == j) {
                my_id = (int)at;
                mine = p;
            }
        }
        float all = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (lane + 32 * i < E) all += expf(l[i] - top);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
        if (lane < top_k) {
            S.ids[t * top_k + lane] = my_id;
            S.gates[t * top_k + lane] = mine / (renorm ? chosen : all);
        }
    }
    __syncthreads();
    const int P = ntok * top_k;
    for (int e = threadIdx.x; e < E; e += MTHREADS) {
        int c = 0;
        for (int p = 0; p < P; ++p) c += S.ids[p] == e;
        S.count[e] = c;
    }
    __syncthreads();
    if (warp == 0) {    // running sums of pairs and of chunks
        int at = 0, chunks = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + lane;
            const int c = e < E ? S.count[e] : 0, k = (c + 15) / 16;
            int sc = c, sk = k;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int a = __shfl_up_sync(0xffffffffu, sc, o), b = __shfl_up_sync(0xffffffffu, sk, o);
                if (lane >= o) {
                    sc += a;
                    sk += b;
                }
            }
            if (e < E) {
                S.first[e] = at + sc - c;
                S.first_chunk[e] = chunks + sk - k;
            }
            at += __shfl_sync(0xffffffffu, sc, 31);
            chunks += __shfl_sync(0xffffffffu, sk, 31);
        }
        if (lane == 0) S.nchunks = chunks;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += MTHREADS) {
        int at = S.first[e];
        if (S.count[e])
            for (int p = 0; p < P; ++p)
                if (S.ids[p] == e) S.list[at++] = (unsigned short)p;
        for (int c = 0; c * 16 < S.count[e]; ++c) {
            S.chunk_e[S.first_chunk[e] + c] = (unsigned short)e;
            S.chunk_at[S.first_chunk[e] + c] = (unsigned short)(S.first[e] + 16 * c);
            S.chunk_n[S.first_chunk[e] + c] = (unsigned char)min(16, S.count[e] - 16 * c);
        }
    }
    __syncthreads();
}

// One block's sums for 16-row tiles `tile` of a weight matrix into S.part.
template <int NB, bool VEC, bool COHERENT>
__device__ __forceinline__ void moe_dot(MoeShared &S, const int8_t *wa, const int8_t *wb, const int8_t *xbase,
                                        const int (&xrow)[2], int64_t xld, int K, int kw, const int8_t *wbegin,
                                        const int8_t *wend, const int8_t *xend) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int kpart = warp % kw;
    const int8_t *x[NB];
#pragma unroll
    for (int n = 0; n < NB; ++n) x[n] = xbase + (int64_t)xrow[n] * xld;
    int sum[NB][4];
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[n][i] = 0;
    const int steps = (K + kQ8Step - 1) / kQ8Step;
    const int per = (steps + kw - 1) / kw;
    const int s0 = min(kpart * per, steps), s1 = min(s0 + per, steps);
    q8_dot<NB, VEC, 4, COHERENT>(sum, wa, wb, x, K, s0, s1, wbegin, wend, xbase, xend);
#pragma unroll
    for (int n = 0; n < NB; ++n) {
        S.part[warp][g][8 * n + 2 * t] = sum[n][0];
        S.part[warp][g][8 * n + 2 * t + 1] = sum[n][1];
        S.part[warp][g + 8][8 * n + 2 * t] = sum[n][2];
        S.part[warp][g + 8][8 * n + 2 * t + 1] = sum[n][3];
    }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(MTHREADS, 2)
q8_expert_kernel(int ntok, int E, int top_k, int H, int I, int renorm, const int8_t *__restrict__ w_up,
                 int64_t ldu, const float *__restrict__ s_up, const int8_t *__restrict__ w_down,
                 int64_t ldd, const float *__restrict__ s_down, T *__restrict__ out, int64_t ldo,
                 int *__restrict__ ids, float *__restrict__ gates, unsigned char *ws, int kw_up,
                 int kw_down, unsigned *err, uint64_t wait_ns) {
    __shared__ MoeShared S;
    const MoeLayout L(ntok, E, top_k, H, I);
    const float *xs = reinterpret_cast<const float *>(ws + L.xs);
    const int8_t *xq = reinterpret_cast<const int8_t *>(ws + L.xq);
    float *hidden = reinterpret_cast<float *>(ws + L.hidden);
    float *hs = reinterpret_cast<float *>(ws + L.hs);
    int8_t *hq = reinterpret_cast<int8_t *>(ws + L.hq);
    float *part = reinterpret_cast<float *>(ws + L.part);
    uint32_t *ticket = reinterpret_cast<uint32_t *>(ws + L.zero);
    uint32_t *ready = ticket + 1, *quantised = ready + L.P, *hmax = quantised + L.P, *done = hmax + L.P;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2;

    pdl_wait();
    if (tid == 0) S.ticket[0] = (int)atomicAdd(ticket, 1u);
    moe_route(S, ntok, E, top_k, renorm, reinterpret_cast<const float *>(ws + L.logits));
    if (blockIdx.x == 0) {
        for (int p = tid; p < L.P; p += MTHREADS) {
            if (ids) ids[p] = S.ids[p];
            if (gates) gates[p] = S.gates[p];
        }
    }
    const int rt_up = MWARPS / kw_up, rt_down = MWARPS / kw_down;
    const int ugroups = (I + 8 * rt_up - 1) / (8 * rt_up);
    const int dgroups = (H + 16 * rt_down - 1) / (16 * rt_down);
    const int up_units = S.nchunks * ugroups, units = up_units + S.nchunks * dgroups;
    const int8_t *up_end = w_up + ((int64_t)E * 2 * I - 1) * ldu + H;
    const int8_t *down_end = w_down + ((int64_t)E * H - 1) * ldd + I;

    for (int it = 0;; ++it) {
        const int u = S.ticket[it & 1];
        if (u >= units) break;
        if (tid == 0) S.ticket[(it + 1) & 1] = (int)atomicAdd(ticket, 1u);
        const bool up = u < up_units;
        const int c = up ? u / ugroups : (u - up_units) / dgroups;
        const int grp = up ? u - c * ugroups : (u - up_units) - c * dgroups;
        const int e = S.chunk_e[c], at = S.chunk_at[c], n = S.chunk_n[c];
        // this lane's token rows: its pair in each block of 8 (the last one past the end)
        const int pa = S.list[at + min(g, n - 1)], pb = S.list[at + min(g + 8, n - 1)];
        if (up) {
            const int i0 = (grp * rt_up + warp / kw_up) * 8;
            const int row = min(i0 + g, I - 1);
            const int8_t *wa = w_up + ((int64_t)e * 2 * I + row) * ldu;
            const int8_t *wb = wa + (int64_t)I * ldu;
            const int xrow[2] = {pa / top_k, pb / top_k};
            const int8_t *xend = xq + (int64_t)ntok * L.Hp;
            if (n <= 8) moe_dot<1, VEC, true>(S, wa, wb, xq, xrow, L.Hp, H, kw_up, w_up, up_end, xend);
            else moe_dot<2, VEC, true>(S, wa, wb, xq, xrow, L.Hp, H, kw_up, w_up, up_end, xend);
            __syncthreads();
            const int tok = n <= 8 ? 8 : 16;
            for (int o = tid; o < 8 * rt_up * tok; o += MTHREADS) {   // whole warps: 8 * tok * rt_up is a multiple of 32
                const int r = o & 7, tl = (o >> 3) % rt_up, j = (o >> 3) / rt_up;
                const int i = (grp * rt_up + tl) * 8 + r;
                uint32_t mb = 0;
                int p = 0;
                if (j < n && i < I) {
                    int sg = 0, su = 0;
                    for (int w = 0; w < kw_up; ++w) {
                        sg += S.part[tl * kw_up + w][r][j];
                        su += S.part[tl * kw_up + w][r + 8][j];
                    }
                    p = S.list[at + j];
                    const float s = __ldcg(xs + p / top_k);
                    const float gv = (float)sg * s * s_up[(int64_t)e * 2 * I + i];
                    const float uv = (float)su * s * s_up[(int64_t)e * 2 * I + I + i];
                    const float hv = __fdiv_rn(gv, 1.0f + expf(-gv)) * uv;
                    __stcg(hidden + (int64_t)p * I + i, hv);
                    mb = abs_bits(hv);
                }
#pragma unroll
                for (int d = 1; d < 8; d <<= 1) mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, d));
                if (r == 0 && j < n && mb != 0u) atomicMax(hmax + p, mb);
            }
            __threadfence();
            __syncthreads();
            if (tid == 0) S.flag = atomicAdd(ready + c, 1u) == (uint32_t)(ugroups - 1);
            __syncthreads();
            if (S.flag) {   // the expert's hidden rows are complete: 8 bits
                __threadfence();
                for (int j = 0; j < n; ++j) {
                    const int p = S.list[at + j];
                    const RowQuant rq(__ldcg(hmax + p));
                    for (int i = tid; i < L.Ip; i += MTHREADS)
                        hq[(int64_t)p * L.Ip + i] = i < I ? (int8_t)rq(__ldcg(hidden + (int64_t)p * I + i)) : (int8_t)0;
                    if (tid == 0) hs[p] = rq.step * rq.unpre;
                }
                __threadfence();
                __syncthreads();
                if (tid == 0) st_release(quantised + c, 1u);
            }
        } else {
            if (tid == 0) {
                bool ok = ld_acquire(quantised + c) != 0u;
                if (!ok) {
                    const uint64_t t0 = globaltimer_ns();
                    do {
                        ok = ld_acquire(quantised + c) != 0u;
                    } while (!ok && globaltimer_ns() - t0 <= wait_ns);
                }
                if (!ok) record_error(err, kErrWaitTimeout);
                S.flag = ok;
            }
            __syncthreads();
            if (!S.flag) break;
            const int n0 = (grp * rt_down + warp / kw_down) * 16;
            const int8_t *wa = w_down + ((int64_t)e * H + min(n0 + g, H - 1)) * ldd;
            const int8_t *wb = w_down + ((int64_t)e * H + min(n0 + g + 8, H - 1)) * ldd;
            const int xrow[2] = {pa, pb};
            const int8_t *xend = hq + (int64_t)L.P * L.Ip;
            if (n <= 8) moe_dot<1, VEC, true>(S, wa, wb, hq, xrow, L.Ip, I, kw_down, w_down, down_end, xend);
            else moe_dot<2, VEC, true>(S, wa, wb, hq, xrow, L.Ip, I, kw_down, w_down, down_end, xend);
            __syncthreads();
            for (int o = tid; o < 16 * rt_down * n; o += MTHREADS) {
                const int r = o & 15, tl = (o >> 4) % rt_down, j = (o >> 4) / rt_down;
                const int col = (grp * rt_down + tl) * 16 + r;
                if (col >= H) continue;
                int s = 0;
                for (int w = 0; w < kw_down; ++w) s += S.part[tl * kw_down + w][r][j];
                const int p = S.list[at + j];
                __stcg(part + (int64_t)p * H + col, (float)s * __ldcg(hs + p) * s_down[(int64_t)e * H + col]);
            }
            __threadfence();
            __syncthreads();
            if (tid == 0) S.flag = atomicAdd(done + grp, 1u) == (uint32_t)(S.nchunks - 1);
            __syncthreads();
            if (S.flag) {   // every expert's part of these columns is there
                __threadfence();
                const int cols = 16 * rt_down, c0 = grp * cols;
                for (int o = tid; o < cols * ntok; o += MTHREADS) {
                    const int col = c0 + o % cols, t = o / cols;
                    if (col >= H) continue;
                    float v = 0.0f;
                    for (int j = 0; j < top_k; ++j)
                        v = fmaf(S.gates[t * top_k + j], __ldcg(part + (int64_t)(t * top_k + j) * H + col), v);
                    out[(int64_t)t * ldo + col] = from_f32<T>(v);
                }
            }
        }
        __syncthreads();   // S.part, S.flag and the next ticket
    }
}

// Warps that share one 16-row tile's K: at least 4 steps each.
int warps_per_tile(int K) {
    const int steps = (K + kQ8Step - 1) / kQ8Step;
    int kw = 1;
    while (kw < MWARPS && steps >= 8 * kw) kw *= 2;
    return kw;
}

template <typename K, typename... A>
cudaError_t launch_pdl(K kern, int grid, int threads, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <typename T>
cudaError_t launch_t(const Q8MoeArgs &a, unsigned char *ws) {
    cudaError_t e = launch_pdl(q8_route_kernel<T>, a.E + a.T, RTHREADS, a.stream, a.T, a.E, a.top_k, a.H, a.I,
                               (const T *)a.x, a.ldx, a.router, a.ldr, ws);
    if (e != cudaSuccess) return e;
    const bool vec = reinterpret_cast<uintptr_t>(a.w_up) % 16 == 0 && a.ldu % 16 == 0 &&
                     reinterpret_cast<uintptr_t>(a.w_down) % 16 == 0 && a.ldd % 16 == 0;
    const int kw_up = warps_per_tile(a.H), kw_down = warps_per_tile(a.I);
    // no more blocks than units: at most one chunk per pair and one per expert and 16 pairs
    const int grid = 2 * (a.sm_count > 0 ? a.sm_count : 1);
    auto kern = vec ? q8_expert_kernel<T, true> : q8_expert_kernel<T, false>;
    return launch_pdl(kern, grid, MTHREADS, a.stream, a.T, a.E, a.top_k, a.H, a.I, a.renormalize, a.w_up, a.ldu,
                      a.s_up, a.w_down, a.ldd, a.s_down, (T *)a.out, a.ldo, a.ids, a.gates, ws, kw_up, kw_down,
                      a.err, a.wait_ns);
}

}  // namespace

size_t q8_moe_workspace_bytes(int T, int E, int top_k, int H, int I) {
    return MoeLayout(T, E, top_k, H, I).total;
}

cudaError_t launch_q8_moe(const Q8MoeArgs &a, void *workspace) {
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    return a.type == kTypeBf16 ? launch_t<__nv_bfloat16>(a, ws) : launch_t<float>(a, ws);
}

}  // namespace sgemm_gb300
