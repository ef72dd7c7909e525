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
// Bound by memory: the picked experts' weights, read once for each 16 of an
// expert's tokens.
//
// The first kernel computes the logits and quantises the tokens.  The second
// is persistent: blocks draw work units from one counter, all gate/up units
// first, then all down units.  A down unit waits (bounded) until its expert's
// hidden rows are there; since every gate/up unit has been drawn by then, by
// a block that waits for nothing, that wait always ends, whatever else runs
// on the GPU.  Between and after them, hidden rows are turned into 8 bits and the
// experts' results added, in slot order: by units of their own
// (q8_expert_ring_kernel) or by the block that finishes the last unit they need
// (q8_expert_kernel, for arrays of any alignment).  Nothing depends on timing, and
// results repeat bit for bit.
//
// Measured (bf16): one token, 2 of 8 experts of 4096 x 14336, 353 MB, 72 us, 4.9
// TB/s; 16 tokens, 6 of 64 experts of 2048 x 1408, 440 MB, 115 us, 3.8 TB/s; 5 FP32
// tokens, 4 of 16 experts of 1024 x 1000, 38 MB, 40 us; 64 tokens over the 64 experts
// 187 us.  (With weights at an odd address, q8_expert_kernel: 174, 280, 41 and 396 us.)  What is above memory's time
// is a chain of hand-overs that each take 1 to 4 us (logits, routing, the first
// weights, hidden rows, 8 bits, results, sums): 17 us for a layer without work.  A
// finisher's unit takes 7000 cycles, half of them the fence before its counter;
// several units to a fence gained nothing.
#include <type_traits>

#include "q8_stream.cuh"

namespace sgemm_gb300 {
namespace {

constexpr int RTHREADS = 256;
constexpr int kRouteTokens = 4;        // tokens of a router block
constexpr int MWARPS = 8, MTHREADS = MWARPS * 32;
constexpr int kMaxPairs = kMoeMaxTokens * kMoeMaxTopK;

// The layer's workspace: byte offsets of its arrays.
struct MoeLayout {
    int P, Hp, Ip, dmax;      // pairs (token, slot); row strides (whole cache lines); down groups at most
    size_t logits, xs, xq, hidden, hs, hq, part, zero, total;
    int nzero;                // words to clear: ticket, ready[P], flag[P], hmax[P], done[dmax]
    __host__ __device__ MoeLayout(int T, int E, int top_k, int H, int I) {
        P = T * top_k;
        Hp = (H + 127) / 128 * 128;
        Ip = (I + 127) / 128 * 128;
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
        hidden = take((size_t)P * I * 4);    // rows of I floats: 16-byte aligned where I % 4 == 0
        hs = take((size_t)P * 4);
        hq = take((size_t)P * Ip);
        part = take((size_t)P * H * 4);
        nzero = 1 + 3 * P + dmax;
        zero = take((size_t)nzero * 4);
        total = at;
    }
};

// The first E * ceil(T / 4) blocks: one expert's logits for four tokens (with all
// tokens in one block, 16 of them over 16 experts left most SMs idle and took 19 us
// cold).  The T blocks after them: one token's 8-bit row; the first of those also
// clears the second kernel's counters.
template <typename T>
__global__ void __launch_bounds__(RTHREADS)
q8_route_kernel(int ntok, int E, int top_k, int H, int I, const T *__restrict__ x, int64_t ldx,
                const float *__restrict__ router, int64_t ldr, int vec, unsigned char *__restrict__ ws) {
    __shared__ uint32_t red[64];
    __shared__ float lsum[RTHREADS / 32][kRouteTokens];
    const MoeLayout L(ntok, E, top_k, H, I);
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int chunks = (ntok + kRouteTokens - 1) / kRouteTokens;
    if ((int)blockIdx.x < E * chunks) {
        const int e = (int)blockIdx.x / chunks, t0 = ((int)blockIdx.x - e * chunks) * kRouteTokens;
        const float *w = router + (int64_t)e * ldr;
        float *logits = reinterpret_cast<float *>(ws + L.logits);
        const T *xr[kRouteTokens];      // tokens past the last read the last one
        float acc[kRouteTokens];
#pragma unroll
        for (int j = 0; j < kRouteTokens; ++j) {
            xr[j] = x + (int64_t)min(t0 + j, ntok - 1) * ldx;
            acc[j] = 0.0f;
        }
        if (vec) {
#pragma unroll 4
            for (int k = 4 * (int)threadIdx.x; k < H; k += 4 * RTHREADS) {
                const float4 w4 = __ldg(reinterpret_cast<const float4 *>(w + k));
#pragma unroll
                for (int j = 0; j < kRouteTokens; ++j) {
                    float v[4];
                    load_vec<T, 4>(xr[j] + k, v);
                    acc[j] = fmaf(v[0], w4.x, fmaf(v[1], w4.y, fmaf(v[2], w4.z, fmaf(v[3], w4.w, acc[j]))));
                }
            }
        } else {
            for (int k = threadIdx.x; k < H; k += RTHREADS) {
                const float wk = __ldg(w + k);
#pragma unroll
                for (int j = 0; j < kRouteTokens; ++j) acc[j] = fmaf(to_f32<T>(xr[j][k]), wk, acc[j]);
            }
        }
#pragma unroll
        for (int j = 0; j < kRouteTokens; ++j)
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], o);
        if (lane == 0)
#pragma unroll
            for (int j = 0; j < kRouteTokens; ++j) lsum[warp][j] = acc[j];
        __syncthreads();
        if (threadIdx.x < kRouteTokens && t0 + (int)threadIdx.x < ntok) {
            float s = 0.0f;
#pragma unroll
            for (int v = 0; v < RTHREADS / 32; ++v) s += lsum[v][threadIdx.x];
            logits[(int64_t)(t0 + threadIdx.x) * E + e] = s;
        }
        return;
    }
    const int t = (int)blockIdx.x - E * chunks;
    if (t == 0) {
        uint32_t *z = reinterpret_cast<uint32_t *>(ws + L.zero);
        for (int i = threadIdx.x; i < L.nzero; i += RTHREADS) z[i] = 0u;
    }
    const T *xr = x + (int64_t)t * ldx;
    uint32_t mx = 0;
    float none = 0.0f;
    int8_t *q = reinterpret_cast<int8_t *>(ws + L.xq) + (int64_t)t * L.Hp;
    if (vec) {
        for (int k = 4 * (int)threadIdx.x; k < H; k += 4 * RTHREADS) {
            float v[4];
            load_vec<T, 4>(xr + k, v);
#pragma unroll
            for (int i = 0; i < 4; ++i) mx = max(mx, abs_bits(v[i]));
        }
    } else {
        for (int k = threadIdx.x; k < H; k += RTHREADS) mx = max(mx, abs_bits(to_f32<T>(xr[k])));
    }
    block_max_sum(mx, none, red);
    const RowQuant rq(mx);
    if (vec) {
        for (int k = 4 * (int)threadIdx.x; k < L.Hp; k += 4 * RTHREADS) {
            float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (k < H) load_vec<T, 4>(xr + k, v);
            store_q<4>(q + k, rq, v);
        }
    } else {
        for (int k = threadIdx.x; k < L.Hp; k += RTHREADS)
            q[k] = k < H ? (int8_t)rq(to_f32<T>(xr[k])) : (int8_t)0;
    }
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
};

struct MoeBlock : MoeShared {
    int ticket[2];
    int flag;
    int part[MWARPS][16][17];
};

// top_k experts and gates of every token; E <= 32 * PER.
template <int PER>
__device__ void moe_choose(MoeShared &S, int ntok, int E, int top_k, int renorm, const float *logits) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int t = warp; t < ntok; t += (int)(blockDim.x >> 5)) {
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
}

// The routing of all tokens, the same in every block: top_k experts and gates
// of each token, then each expert's pairs and their chunks of up to 16.
__device__ void moe_route(MoeShared &S, int ntok, int E, int top_k, int renorm, const float *logits) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (E <= 32) moe_choose<1>(S, ntok, E, top_k, renorm, logits);
    else if (E <= 64) moe_choose<2>(S, ntok, E, top_k, renorm, logits);
    else if (E <= 128) moe_choose<4>(S, ntok, E, top_k, renorm, logits);
    else moe_choose<kMoeMaxExperts / 32>(S, ntok, E, top_k, renorm, logits);
    __syncthreads();
    const int P = ntok * top_k;
    for (int e = threadIdx.x; e < E; e += (int)blockDim.x) {
        int c = 0;
#pragma unroll 8
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
    for (int e = threadIdx.x; e < E; e += (int)blockDim.x) {
        int at = S.first[e];
        if (S.count[e])
#pragma unroll 8
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
template <int NB>
__device__ __forceinline__ void moe_dot(MoeBlock &S, const int8_t *wa, const int8_t *wb, const int8_t *xbase,
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
    q8_dot<NB, 4, true>(sum, wa, wb, x, K, s0, s1, wbegin, wend, xbase, xend);
#pragma unroll
    for (int n = 0; n < NB; ++n) {
        S.part[warp][g][8 * n + 2 * t] = sum[n][0];
        S.part[warp][g][8 * n + 2 * t + 1] = sum[n][1];
        S.part[warp][g + 8][8 * n + 2 * t] = sum[n][2];
        S.part[warp][g + 8][8 * n + 2 * t + 1] = sum[n][3];
    }
}

// ---- any alignment -------------------------------------------------------------

template <typename T>
__global__ void __launch_bounds__(MTHREADS, 2)
q8_expert_kernel(int ntok, int E, int top_k, int H, int I, int renorm, const int8_t *__restrict__ w_up,
                 int64_t ldu, const float *__restrict__ s_up, const int8_t *__restrict__ w_down,
                 int64_t ldd, const float *__restrict__ s_down, T *__restrict__ out, int64_t ldo,
                 int *__restrict__ ids, float *__restrict__ gates, unsigned char *ws, int kw_up,
                 int kw_down, unsigned *err, uint64_t wait_ns) {
    __shared__ MoeBlock S;
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
            if (n <= 8) moe_dot<1>(S, wa, wb, xq, xrow, L.Hp, H, kw_up, w_up, up_end, xend);
            else moe_dot<2>(S, wa, wb, xq, xrow, L.Hp, H, kw_up, w_up, up_end, xend);
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
            if (n <= 8) moe_dot<1>(S, wa, wb, hq, xrow, L.Ip, I, kw_down, w_down, down_end, xend);
            else moe_dot<2>(S, wa, wb, hq, xrow, L.Ip, I, kw_down, w_down, down_end, xend);
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

// ---- the persistent kernel for weights whose arrays are 16-byte aligned -----------
//
// Roles of a block (one per SM):
//   producer   one warp draws units from the counter and brings each unit's
//              weights into a ring of bulk copies (see q8_stream.cuh), running
//              ahead into later units, down projections too: weights depend on
//              the routing alone;
//   consumers  two groups of eight warps take units in turn, multiply (dp4a up
//              to 4 tokens, then 8-bit MMAs) and add their integer sums in a
//              buffer;
//   finishers  a warp for each group turns sums into hidden values, quantises
//              complete hidden rows and adds the experts' results (units of their
//              own after the gate/up and after the down projections).
// A unit is up to four 16-row tiles (of the gate/up projection, 8 gate and 8 up
// rows each), 33 to 70 KB: its chain of waits, token loads and hand-overs takes as
// long as 33 KB do at the memory's rate, hence the groups, the finishers and the
// size; larger units leave blocks idle at the end of a projection.
// Eight rows of a stage are one TMA box of 8-byte elements, 2 KB a row at most:
// as 16 bulk copies, a stage took its warp 2000 cycles to issue, 13 bytes a
// cycle.  (Rows then lie a multiple of 512 bytes apart; see unit_products on the
// bank conflicts that this would make.)  Rows whose
// length is no multiple of 16 (SHIFT) have no TMA map; they are copied one by one
// from the 16-byte boundary below and shifted as the fragments are read.
constexpr int FINISHERS = 2;                               // one per consumer group
constexpr int E_PRODUCER = kQ8Consumers + FINISHERS;
constexpr int ETHREADS = (E_PRODUCER + 1) * 32;
constexpr int ERING = 4, EBUFS = 4;                        // stages; buffers of sums, two per group
constexpr int EGROUP = kQ8Consumers / 2;                   // warps of a consumer group
constexpr int ESTEPS = 4;                                  // steps per consumer warp and stage
constexpr int ETILES = 4;                                  // 16-row tiles of a unit, at most
constexpr uint32_t ESTAGE = 64 * (2 * ESTEPS * kQ8Step + 80);  // the largest geometry (RT = 4)
constexpr int EPART = ETILES * 2 * 128;                    // one unit's sums: [tile][token block][word][lane]
constexpr int QSEG = 512;                                  // hidden values a quantising unit takes
constexpr int CSEG = 128;                                  // results an adding unit takes

struct EGeom {       // one projection's division
    int K, rt, kw, kb, blocks, stages;
    uint32_t ld;
    int tiles;       // groups of rt row tiles that the projection has
    int sub, groups; // groups of rt tiles to a unit (a power of two), units; set on the device
    EGeom() = default;
    // `rows` results, `per_tile` of them to a tile
    EGeom(int K_, int rows, int per_tile, bool shift) : K(K_) {
        const int steps = (K + kQ8Step - 1) / kQ8Step;
        rt = steps <= 8 ? 4 : steps <= 16 ? 2 : 1;
        kw = EGROUP / rt;
        kb = kw * ESTEPS;
        // whole steps that the ring brings; shifted rows leave 15 bytes at their end alone
        blocks = shift ? (K > 15 ? (K - 15) / kQ8Step : 0) : K / kQ8Step;
        stages = blocks > 0 ? (blocks + kb - 1) / kb : 1;
        ld = (uint32_t)(kb * kQ8Step + (shift ? 80 : 0));
        tiles = (rows + per_tile * rt - 1) / (per_tile * rt);
        sub = 1;
        groups = tiles;
    }
    // as many tiles to a unit as leave every block six units (at 8, 12 and 16 the
    // layer for one token took 74, 82 and 82 us, at 4 73).  Units of one tile at the end of a
    // projection, which would even out the blocks' ends, cost more than that (75 us).
    __device__ __forceinline__ void divide(int chunks, int blocks_of_grid) {
        const int64_t all = (int64_t)tiles * chunks;
        sub = rt == 1 ? 4 : rt == 2 ? 2 : 1;
        while (sub > 1 && all < (int64_t)6 * sub * blocks_of_grid) sub >>= 1;
        groups = (tiles + sub - 1) >> (sub == 4 ? 2 : sub == 2 ? 1 : 0);
    }
};
static_assert(ETILES == 4, "rt * sub tiles of a unit");

// What the roles work on; in shared memory, so that none of it occupies the
// registers of a role that does not need it (what they spill comes back from L2:
// next to 200 KB of shared memory L1 is small).
struct EArgs {
    const int8_t *w_up, *w_down;
    int64_t ldu, ldd;
    const float *s_up, *s_down;
    void *out;
    int64_t ldo;
    const float *xs;
    const int8_t *xq;
    float *hidden, *hs, *res;
    int8_t *hq;
    uint32_t *ticket, *ready, *quantised, *hmax, *done;
    unsigned *err;
    uint64_t wait_ns;
    int ntok, top_k, H, I, Hp, Ip;
    int segs, csegs;                          // quantising units of a pair, adding units of a token
    int up_units, quant_end, down_end, units; // units: gate/up, quantise, down, add

    // what unit u does: 0 gate/up, 1 quantise, 2 down, 3 add, -1 nothing (the end)
    __device__ __forceinline__ int kind(int u) const {
        return u < up_units ? 0 : u < quant_end ? 1 : u < down_end ? 2 : u < units ? 3 : -1;
    }
};

struct EShared {
    MoeShared route;
    EArgs a;
    EGeom geom[2];                    // gate/up, down
    int unit[ERING];                  // unit a stage belongs to
    int done[EBUFS];                  // unit a buffer of sums belongs to
    uint64_t full[ERING], empty[ERING], bfull[EBUFS], bempty[EBUFS];
};
constexpr size_t EOFF_PART = (size_t)ERING * ESTAGE;
constexpr size_t EOFF_SHARED = EOFF_PART + (size_t)EBUFS * EPART * 4;
constexpr size_t ESMEM = 128 + EOFF_SHARED + sizeof(EShared);
static_assert(ESMEM <= 227 * 1024, "shared memory per block");

// 16 bytes at any address of shared memory.
__device__ __forceinline__ uint4 lds_shifted(uint32_t addr) {
    const uint32_t a = addr & ~3u;
    const int sh = 8 * (int)(addr & 3);
    uint32_t w[5];
#pragma unroll
    for (int i = 0; i < 5; ++i) asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[i]) : "r"(a + 4 * i));
    return make_uint4(__funnelshift_r(w[0], w[1], sh), __funnelshift_r(w[1], w[2], sh),
                      __funnelshift_r(w[2], w[3], sh), __funnelshift_r(w[3], w[4], sh));
}

// Lane 0 polls a counter until it reaches `want` (bounded); the warp agrees.
__device__ __forceinline__ bool warp_poll(const uint32_t *p, uint32_t want, uint64_t wait_ns) {
    int ok = 1;
    if ((threadIdx.x & 31) == 0 && ld_acquire(p) < want) {
        const uint64_t t0 = globaltimer_ns();
        do {
            ok = ld_acquire(p) >= want;
        } while (!ok && globaltimer_ns() - t0 <= wait_ns);
    }
    ok = __shfl_sync(0xffffffffu, ok, 0);
    __syncwarp();
    return ok != 0;
}

// The same for `count` <= 32 counters, one a lane.
__device__ __forceinline__ bool warp_poll_all(const uint32_t *p, int count, uint32_t want, uint64_t wait_ns) {
    const int lane = threadIdx.x & 31;
    bool ok = lane >= count || ld_acquire(p + lane) >= want;
    if (!ok) {
        const uint64_t t0 = globaltimer_ns();
        do {
            ok = ld_acquire(p + lane) >= want;
        } while (!ok && globaltimer_ns() - t0 <= wait_ns);
    }
    // the vote orders no memory accesses: what one lane acquired is the others' from here
    ok = __all_sync(0xffffffffu, ok) != 0;
    __syncwarp();
    return ok;
}

// The products of one unit by one warp of a consumer group, into the buffer
// `sums`; false when a wait ran out.  DP: NT tokens by dp4a, each lane with every
// token's bytes; otherwise NT blocks of 8 tokens by MMA, lane row g with token g
// of each.
template <int NT, bool DP, bool SHIFT>
__device__ __forceinline__ bool unit_products(EShared &S, uint32_t ring, int *sums, int c, int grp, bool up,
                                           uint32_t used) {
    const EArgs &A = S.a;
    const MoeShared &R = S.route;
    const EGeom &G = S.geom[up ? 0 : 1];
    const int lane = threadIdx.x & 31, cw = (int)(threadIdx.x >> 5) % EGROUP;
    const int g = lane >> 2, t4 = lane & 3;
    const int kb = G.kb, blocks = G.blocks, stages = G.stages, sub = G.sub, rt = G.rt;
    const uint32_t ld = G.ld;
    const int tl = cw / G.kw, kpart = cw % G.kw;      // this warp's tile of a stage, its share of the steps
    const int step0 = kpart * ESTEPS;
    // Rows g and g + 1 lie in the same banks.  With dp4a every lane has its own sum, so
    // odd rows take their steps in the order 1, 0, 3, 2 and meet no conflict.
    static_assert(ESTEPS % 4 == 0 || ESTEPS == 2, "pairs of steps");
    const int odd = DP ? g & 1 : 0;
    const int8_t *xbase = (up ? A.xq : A.hq) + 16 * t4;
    int x[NT];                                        // offsets: at most 1024 rows of 131072 bytes
#pragma unroll
    for (int j = 0; j < NT; ++j) {                    // tokens past the chunk's end: the last one
        const int p = R.list[R.chunk_at[c] + min(DP ? j : 8 * j + g, (int)R.chunk_n[c] - 1)];
        x[j] = up ? p / A.top_k * A.Hp : p * A.Ip;
    }
    // The tokens of a batch of steps are asked for together, the first ahead of the
    // wait for the weights.  (A step past the last reads the last one's tokens and is
    // not used.)  Asked for a stage earlier still, or kept from tile to tile, they
    // gained nothing (125 against 125 us for 16 tokens, 72.5 against 71.7 for one).
    constexpr int BATCH = NT <= 2 || ESTEPS <= 2 ? ESTEPS : ESTEPS / 2;
    uint4 xv[BATCH][NT];
    auto xload = [&](int first) {
#pragma unroll
        for (int k = 0; k < BATCH; ++k)
#pragma unroll
            for (int j = 0; j < NT; ++j)
                xv[k][j] = *reinterpret_cast<const uint4 *>(xbase + (x[j] + max(0, min(first + (k ^ odd), blocks - 1)) * kQ8Step));
    };
    auto step = [&](auto &sum, const uint4 &a, const uint4 &d, const uint4 (&xs)[NT]) {
        if constexpr (DP) {
            q8_step_dp<NT>(sum, a, d, xs);
        } else {
#pragma unroll
            for (int j = 0; j < NT; ++j) q8_step_s8(sum[j], a, d, xs[j]);
        }
    };
    // this lane's two weight rows of a tile
    auto rows = [&](int t, const int8_t *&wa, const int8_t *&wb) {
        const int tile = (grp * sub + t) * rt + tl, e = R.chunk_e[c];
        if (up) {
            wa = A.w_up + ((int64_t)e * 2 * A.I + min(tile * 8 + g, A.I - 1)) * A.ldu;
            wb = wa + (int64_t)A.I * A.ldu;
        } else {
            wa = A.w_down + ((int64_t)e * A.H + min(tile * 16 + g, A.H - 1)) * A.ldd;
            wb = A.w_down + ((int64_t)e * A.H + min(tile * 16 + g + 8, A.H - 1)) * A.ldd;
        }
    };
    for (int t = 0; t < sub; ++t) {
        // where the rows lie in a stage
        uint32_t oa = (uint32_t)(tl * 16 + g) * ld + (uint32_t)(step0 * kQ8Step + 16 * t4), ob = oa + 8 * ld;
        if (SHIFT) {
            const int8_t *wa, *wb;
            rows(t, wa, wb);
            oa += (uint32_t)(reinterpret_cast<uintptr_t>(wa) & 15);
            ob += (uint32_t)(reinterpret_cast<uintptr_t>(wb) & 15);
        }
        int sum[NT][DP ? 2 : 4];
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < (DP ? 2 : 4); ++i) sum[j][i] = 0;
        for (int s = 0; s < stages; ++s, ++used) {
            const int r = (int)(used % ERING);
            const int first = s * kb + step0;
            const int here = min(ESTEPS, blocks - first);    // this warp's steps of the stage
            xload(first);
            if (s + t > 0 && !warp_wait(smem_u32(&S.full[r]), (used / ERING) & 1, A.wait_ns)) return false;
            const uint32_t stage = ring + (uint32_t)r * ESTAGE;
#pragma unroll
            for (int k0 = 0; k0 < ESTEPS; k0 += BATCH) {
                if (k0 > 0) xload(first + k0);
#pragma unroll
                for (int k = 0; k < BATCH; ++k)
                    if (((k0 + k) ^ odd) < here) {
                        const uint32_t o = stage + (uint32_t)((k0 + k) ^ odd) * kQ8Step;
                        step(sum, SHIFT ? lds_shifted(o + oa) : lds128(o + oa), SHIFT ? lds_shifted(o + ob) : lds128(o + ob), xv[k]);
                    }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&S.empty[r]));
        }
        if (kpart == 0 && blocks * kQ8Step < G.K) {   // the rows' last values
            const int8_t *wa, *wb;
            rows(t, wa, wb);
            for (int k0 = blocks * kQ8Step; k0 < G.K; k0 += kQ8Step) {
                const int valid = min(16, max(0, G.K - k0 - 16 * t4));
                uint4 xt[NT];
#pragma unroll
                for (int j = 0; j < NT; ++j) xt[j] = *reinterpret_cast<const uint4 *>(xbase + (x[j] + k0));
                step(sum, load16_bytes(wa + k0 + 16 * t4, valid), load16_bytes(wb + k0 + 16 * t4, valid), xt);
            }
        }
        // whole numbers: the order of these additions does not matter
        int *to = sums + (t * rt + tl) * 256;
        if constexpr (DP) {
            // The quad's four parts of every sum, each lane ending with row g + 8 i and
            // every second token; left where the MMA would leave them.
            const int i = t4 & 1, odd_tok = t4 >> 1;
            int m[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j)
                m[j] = (i ? sum[j][1] : sum[j][0]) + __shfl_xor_sync(0xffffffffu, i ? sum[j][0] : sum[j][1], 1);
            if constexpr (NT == 1) {
                const int v2 = m[0] + __shfl_xor_sync(0xffffffffu, m[0], 2);
                if (odd_tok == 0) atomicAdd(to + 64 * i + 4 * g, v2);
            } else {
#pragma unroll
                for (int h = 0; h < NT / 2; ++h) {
                    const int v2 = (odd_tok ? m[2 * h + 1] : m[2 * h]) +
                                   __shfl_xor_sync(0xffffffffu, odd_tok ? m[2 * h] : m[2 * h + 1], 2);
                    atomicAdd(to + 64 * i + 32 * odd_tok + 4 * g + h, v2);
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) atomicAdd(to + j * 128 + 32 * i + lane, sum[j][i]);
        }
    }
    return true;
}

template <bool SU, bool SD>
__device__ __noinline__ void produce(EShared &S, uint32_t ring, const CUtensorMap *map_up,
                                     const CUtensorMap *map_down, int next) {
    const EArgs &A = S.a;
    const int lane = threadIdx.x & 31;
    bool ok = true;
    uint32_t g = 0;
    auto slot = [&](int &r) {
        r = (int)(g % ERING);
        return g < (uint32_t)ERING || warp_wait(smem_u32(&S.empty[r]), (g / ERING - 1) & 1, A.wait_ns);
    };
    while (ok) {
        const int u = __shfl_sync(0xffffffffu, next, 0);
        if (lane == 0) next = (int)atomicAdd(A.ticket, 1u);   // on its way while this unit is brought
        const int kind = A.kind(u);
        if (kind & 1) {      // nothing to bring: a finisher's unit, or the end
            int r;
            if (!(ok = slot(r))) break;
            if (lane == 0) {
                S.unit[r] = u;
                mbar_arrive(smem_u32(&S.full[r]));
            }
            ++g;
            if (kind < 0) break;
            continue;
        }
        const bool up = kind == 0;
        const EGeom &G = S.geom[up ? 0 : 1];
        const int v = up ? u : u - A.quant_end;
        const int c = v / G.groups, grp = v - c * G.groups, e = S.route.chunk_e[c];
        const int rt = G.rt, stages = G.stages, kb = G.kb, blocks = G.blocks;
        const uint32_t ld = G.ld;
        for (int t = 0; t < G.sub && ok; ++t) {
            const int tile0 = (grp * G.sub + t) * rt;
            for (int s = 0; s < stages; ++s, ++g) {
                int r;
                if (!(ok = slot(r))) break;
                const uint32_t bar = smem_u32(&S.full[r]), base = ring + (uint32_t)r * ESTAGE;
                if (!(up ? SU : SD)) {
                    // lane q brings rows 8 (q % 2) .. + 7 of row tile q / 2 (rows past the
                    // projection's end are others' or zero; their results are dropped)
                    const int tile = tile0 + (lane >> 1);
                    const int row = up ? e * 2 * A.I + (lane & 1) * A.I + tile * 8 : e * A.H + tile * 16 + 8 * (lane & 1);
                    if (lane == 0) {
                        S.unit[r] = u;
                        if (blocks > 0) mbar_arrive_expect_tx(bar, 16u * rt * ld);
                        else mbar_arrive(bar);
                    }
                    __syncwarp();
                    if (lane < 2 * rt && blocks > 0)
                        tma_load_2d(base + (uint32_t)lane * 8 * ld, up ? map_up : map_down, bar, s * kb * (kQ8Step / 8), row);
                } else {
                    const int len = max(0, min(kb, blocks - s * kb)) * kQ8Step;
                    const int8_t *src[2];
                    uint32_t bytes[2], total = 0;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int q = lane + 32 * h, tile = tile0 + (q >> 4);
                        bytes[h] = 0;
                        src[h] = nullptr;
                        if (q < 16 * rt && len > 0) {   // rows past the end read the last one
                            const int64_t row = up ? (int64_t)e * 2 * A.I + min(tile * 8 + (q & 7), A.I - 1) + ((q >> 3) & 1) * A.I
                                                   : (int64_t)e * A.H + min(tile * 16 + (q & 15), A.H - 1);
                            src[h] = (up ? A.w_up + row * A.ldu : A.w_down + row * A.ldd) + (int64_t)s * kb * kQ8Step;
                            const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(src[h]) & 15);
                            src[h] -= off;
                            bytes[h] = ((uint32_t)len + off + 15) / 16 * 16;
                            total += bytes[h];
                        }
                    }
                    total = __reduce_add_sync(0xffffffffu, total);
                    if (lane == 0) {
                        S.unit[r] = u;
                        if (total > 0) mbar_arrive_expect_tx(bar, total);
                        else mbar_arrive(bar);
                    }
                    __syncwarp();
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        if (bytes[h] > 0) bulk_load(base + (uint32_t)(lane + 32 * h) * ld, src[h], bytes[h], bar);
                }
                __syncwarp();
            }
        }
    }
    // The block may not end before its copies have landed, whichever role gave up.
    if (lane == 0) {
        if (!ok) record_error(A.err, kErrWaitTimeout);
        for (uint32_t q = g > (uint32_t)ERING ? g - ERING : 0; q < g; ++q)
            mbar_wait(smem_u32(&S.full[q % ERING]), (q / ERING) & 1, 1000000000ull);
    }
}

template <bool SU, bool SD>
__device__ __noinline__ void consume(EShared &S, uint32_t ring, int *part) {
    const EArgs &A = S.a;
    const MoeShared &R = S.route;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = warp / EGROUP, cw = warp % EGROUP;
    int open_chunk = -1;              // the chunk whose hidden rows were last seen complete
    uint32_t used = 0;
    bool ok = true;
    for (uint32_t count = 0;; ++count) {
        int r = (int)(used % ERING);
        if (!(ok = warp_wait(smem_u32(&S.full[r]), (used / ERING) & 1, A.wait_ns))) break;
        const int u = S.unit[r];
        const int kind = A.kind(u);
        const bool mine = (int)(count & 1) == group, up = kind == 0;
        const EGeom &G = S.geom[up ? 0 : 1];
        if (!mine || (kind & 1)) {     // the other group's unit, or one without weights
            const int all = (kind & 1) ? 1 : G.stages * G.sub;
            for (int s = 0; s < all; ++s, ++used) {
                r = (int)(used % ERING);
                if (s > 0 && !(ok = warp_wait(smem_u32(&S.full[r]), (used / ERING) & 1, A.wait_ns))) break;
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&S.empty[r]));
            }
            if (!ok) break;
            if (!mine && kind >= 0) continue;
        } else {
            const int b = (int)(count % EBUFS);
            const int v = up ? u : u - A.quant_end;
            const int c = v / G.groups, grp = v - c * G.groups, n = R.chunk_n[c];
            // down: the chunk's hidden rows are there in 8 bits
            if (!up && c != open_chunk) {
                if (!(ok = warp_poll(A.quantised + c, (uint32_t)(n * A.segs), A.wait_ns))) break;
                open_chunk = c;
            }
            // the buffer is free (its finisher has read and cleared it)
            if (count >= (uint32_t)EBUFS &&
                !(ok = warp_wait(smem_u32(&S.bempty[b]), (count / EBUFS - 1) & 1, A.wait_ns)))
                break;
            int *sums = part + b * EPART;
            auto products = [&](auto shift) {
                constexpr bool SHIFT = decltype(shift)::value;
                if (n == 1) return unit_products<1, true, SHIFT>(S, ring, sums, c, grp, up, used);
                if (n == 2) return unit_products<2, true, SHIFT>(S, ring, sums, c, grp, up, used);
                if (n <= 4) return unit_products<4, true, SHIFT>(S, ring, sums, c, grp, up, used);
                if (n <= 8) return unit_products<1, false, SHIFT>(S, ring, sums, c, grp, up, used);
                return unit_products<2, false, SHIFT>(S, ring, sums, c, grp, up, used);
            };
            if (SU == SD || up) ok = products(std::bool_constant<SU>{});
            else ok = products(std::bool_constant<SD>{});
            if (!ok) break;
            used += (uint32_t)(G.stages * G.sub);
        }
        // hand the sums over; the end goes to every finisher, each group telling
        // the one whose buffers it fills (it alone knows their turn)
        const uint32_t last = kind >= 0 ? count : count + 1;
        for (uint32_t q = count; q <= last; ++q) {
            if ((int)(q & 1) != group) continue;
            const int o = (int)(q % EBUFS);
            if ((kind & 1) && q >= (uint32_t)EBUFS &&
                !(ok = warp_wait(smem_u32(&S.bempty[o]), (q / EBUFS - 1) & 1, A.wait_ns)))
                break;
            if (cw == 0 && lane == 0) S.done[o] = u;
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&S.bfull[o]));
        }
        if (!ok || kind < 0) break;
    }
    if (!ok && lane == 0) record_error(A.err, kErrWaitTimeout);
}

template <typename T>
__device__ __noinline__ void finish(EShared &S, int *part) {
    const EArgs &A = S.a;
    const MoeShared &R = S.route;
    const int lane = threadIdx.x & 31;
    const int H = A.H, I = A.I, top_k = A.top_k;
    bool ok = true;
    for (uint32_t count = (threadIdx.x >> 5) - kQ8Consumers;; count += FINISHERS) {
        const int b = (int)(count % EBUFS);       // one of this finisher's buffers
        if (!(ok = warp_wait(smem_u32(&S.bfull[b]), (count / EBUFS) & 1, A.wait_ns))) break;
        const int u = S.done[b];
        const int kind = A.kind(u);
        if (kind < 0) break;
        int *sums = part + b * EPART;
        auto sum_at = [&](int tile, int row, int tok) {
            return sums[tile * 256 + (tok >> 3) * 128 + (((row >> 3) << 1) + (tok & 1)) * 32 + (row & 7) * 4 + ((tok & 7) >> 1)];
        };
        if (kind & 1) {
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&S.bempty[b]));
        }
        if (kind == 1) {
            const int v = u - A.up_units, q = v / A.segs, seg = v - q * A.segs;
            const int p = R.list[q];            // pairs in the order of their chunks
            const int e = R.ids[p], c = R.first_chunk[e] + (q - R.first[e]) / 16;
            if (!(ok = warp_poll(A.ready + c, (uint32_t)S.geom[0].groups, A.wait_ns))) break;
            const int lo = seg * QSEG, hi = min(lo + QSEG, A.Ip);
            const float *hr = A.hidden + (int64_t)p * I;
            int8_t *qr = A.hq + (int64_t)p * A.Ip;
            float h4[QSEG / 128][4];        // all loads at once
#pragma unroll
            for (int q4 = 0; q4 < QSEG / 128; ++q4) {
                const int i = lo + 128 * q4 + 4 * lane;
                if (I % 4 == 0 && i < I) {
                    const float4 v4 = __ldcg(reinterpret_cast<const float4 *>(hr + i));
                    h4[q4][0] = v4.x; h4[q4][1] = v4.y; h4[q4][2] = v4.z; h4[q4][3] = v4.w;
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k) h4[q4][k] = i + k < I ? __ldcg(hr + i + k) : 0.0f;
                }
            }
            const RowQuant rq(__ldcg(A.hmax + p));
#pragma unroll
            for (int q4 = 0; q4 < QSEG / 128; ++q4) {
                const int i = lo + 128 * q4 + 4 * lane;
                if (i < hi)
                    *reinterpret_cast<uint32_t *>(qr + i) = pack4(rq(h4[q4][0]), rq(h4[q4][1]), rq(h4[q4][2]), rq(h4[q4][3]));
            }
            if (seg == 0 && lane == 0) A.hs[p] = rq.step * rq.unpre;
            __threadfence();
            __syncwarp();
            if (lane == 0) atomicAdd(A.quantised + c, 1u);
            continue;
        }
        if (kind == 3) {      // one token's sum over its experts, in slot order
            const int v = u - A.down_end, t = v / A.csegs, c0 = (v - t * A.csegs) * CSEG;
            const int cols = 16 * S.geom[1].rt * S.geom[1].sub, g0 = c0 / cols, g1 = (min(c0 + CSEG, H) - 1) / cols;
            if (!(ok = warp_poll_all(A.done + g0, g1 - g0 + 1, (uint32_t)R.nchunks, A.wait_ns))) break;
            const int col = c0 + 4 * lane;
            float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            const float *rr = A.res + (int64_t)t * top_k * H + col;
#pragma unroll 4
            for (int j = 0; j < top_k; ++j) {
                float w4[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) w4[k] = col + k < H ? __ldcg(rr + (int64_t)j * H + k) : 0.0f;
#pragma unroll
                for (int k = 0; k < 4; ++k) y[k] = fmaf(R.gates[t * top_k + j], w4[k], y[k]);
            }
            T *o = static_cast<T *>(A.out) + (int64_t)t * A.ldo + col;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (col + k < H) o[k] = from_f32<T>(y[k]);
            continue;
        }
        const bool up = kind == 0;
        const EGeom &G = S.geom[up ? 0 : 1];
        const int tiles = G.rt * G.sub, tsh = tiles == 4 ? 2 : tiles == 2 ? 1 : 0;     // of the unit
        const int v = up ? u : u - A.quant_end;
        const int c = v / G.groups, grp = v - c * G.groups;
        const int e = R.chunk_e[c], at = R.chunk_at[c], n = R.chunk_n[c];
        if (up) {
            const int all = 8 * tiles * n;
            for (int o0 = 0; o0 < all; o0 += 128) {     // four rounds' scales at once
                float sx[4], sg[4], su[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int o = o0 + 32 * q + lane, tl = (o >> 3) & (tiles - 1), j = (o >> 3) >> tsh;
                    const int i = (grp * tiles + tl) * 8 + (o & 7);
                    sx[q] = sg[q] = su[q] = 0.0f;
                    if (o < all && i < I) {
                        sx[q] = __ldg(A.xs + R.list[at + j] / top_k);
                        sg[q] = __ldg(A.s_up + (int64_t)e * 2 * I + i);
                        su[q] = __ldg(A.s_up + (int64_t)e * 2 * I + I + i);
                    }
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (o0 + 32 * q >= all) break;
                    const int o = o0 + 32 * q + lane, row = o & 7, tl = (o >> 3) & (tiles - 1), j = (o >> 3) >> tsh;
                    const int i = (grp * tiles + tl) * 8 + row;
                    uint32_t mb = 0;
                    int p = 0;
                    if (o < all && i < I) {
                        p = R.list[at + j];
                        const float gv = (float)sum_at(tl, row, j) * sx[q] * sg[q];
                        const float uv = (float)sum_at(tl, row + 8, j) * sx[q] * su[q];
                        const float hv = __fdiv_rn(gv, 1.0f + expf(-gv)) * uv;
                        __stcg(A.hidden + (int64_t)p * I + i, hv);
                        mb = abs_bits(hv);
                    }
#pragma unroll
                    for (int d = 1; d < 8; d <<= 1) mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, d));
                    if (row == 0 && mb != 0u) atomicMax(A.hmax + p, mb);
                }
            }
        } else {
            const int all = 16 * tiles * n;
#pragma unroll 4
            for (int o = lane; o < all; o += 32) {
                const int row = o & 15, tl = (o >> 4) & (tiles - 1), j = (o >> 4) >> tsh;
                const int col = (grp * tiles + tl) * 16 + row;
                if (col < H) {
                    const int p = R.list[at + j];
                    __stcg(A.res + (int64_t)p * H + col,
                           (float)sum_at(tl, row, j) * __ldcg(A.hs + p) * __ldg(A.s_down + (int64_t)e * H + col));
                }
            }
        }
        // the sums have been read: the buffer goes back empty
        __syncwarp();
        for (int i = lane; i < tiles * 64; i += 32) reinterpret_cast<int4 *>(sums)[i] = make_int4(0, 0, 0, 0);
        __threadfence();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(smem_u32(&S.bempty[b]));
            atomicAdd(up ? A.ready + c : A.done + grp, 1u);
        }
    }
    if (!ok && lane == 0) record_error(A.err, kErrWaitTimeout);
}

template <typename T, bool SU, bool SD>
__global__ void __launch_bounds__(ETHREADS, 1)
q8_expert_ring_kernel(const __grid_constant__ CUtensorMap map_up, const __grid_constant__ CUtensorMap map_down,
                      const EGeom g_up, const EGeom g_down, int ntok, int E, int top_k, int H, int I, int renorm, const int8_t *w_up, int64_t ldu,
                      const float *s_up, const int8_t *w_down, int64_t ldd, const float *s_down, T *out, int64_t ldo,
                      int *__restrict__ ids, float *__restrict__ gates, unsigned char *ws, unsigned *err,
                      uint64_t wait_ns) {
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
    int *part = reinterpret_cast<int *>(smem + EOFF_PART);
    EShared &S = *reinterpret_cast<EShared *>(smem + EOFF_SHARED);
    MoeShared &R = S.route;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const MoeLayout L(ntok, E, top_k, H, I);

    if (tid == 0) {
        for (int s = 0; s < ERING; ++s) {
            mbar_init(smem_u32(&S.full[s]), 1);
            mbar_init(smem_u32(&S.empty[s]), kQ8Consumers);
        }
        for (int b = 0; b < EBUFS; ++b) {
            mbar_init(smem_u32(&S.bfull[b]), EGROUP);
            mbar_init(smem_u32(&S.bempty[b]), 1);
        }
        mbar_fence_init();
    }
    for (int i = tid; i < EBUFS * EPART; i += ETHREADS) part[i] = 0;
    uint32_t *ticket = reinterpret_cast<uint32_t *>(ws + L.zero);
    if (tid == 32) {
        EArgs &A = S.a;
        A.w_up = w_up; A.w_down = w_down; A.ldu = ldu; A.ldd = ldd; A.s_up = s_up; A.s_down = s_down;
        A.out = out; A.ldo = ldo;
        A.xs = reinterpret_cast<const float *>(ws + L.xs);
        A.xq = reinterpret_cast<const int8_t *>(ws + L.xq);
        A.hidden = reinterpret_cast<float *>(ws + L.hidden);
        A.hs = reinterpret_cast<float *>(ws + L.hs);
        A.hq = reinterpret_cast<int8_t *>(ws + L.hq);
        A.res = reinterpret_cast<float *>(ws + L.part);
        A.ticket = ticket;
        A.ready = ticket + 1;
        A.quantised = A.ready + L.P;
        A.hmax = A.quantised + L.P;
        A.done = A.hmax + L.P;
        A.err = err; A.wait_ns = wait_ns;
        A.ntok = ntok; A.top_k = top_k; A.H = H; A.I = I; A.Hp = L.Hp; A.Ip = L.Ip;
    }
    pdl_wait();
    int next = 0;       // the producer's first unit, asked for before the routing
    if (warp == E_PRODUCER && lane == 0) next = (int)atomicAdd(ticket, 1u);
    moe_route(R, ntok, E, top_k, renorm, reinterpret_cast<const float *>(ws + L.logits));   // ends with a barrier
    EArgs &A = S.a;
    if (tid == 0) {
        S.geom[0] = g_up;
        S.geom[0].divide(R.nchunks, (int)gridDim.x);
        A.up_units = R.nchunks * S.geom[0].groups;
    } else if (tid == 32) {
        S.geom[1] = g_down;
        S.geom[1].divide(R.nchunks, (int)gridDim.x);
        A.csegs = (H + CSEG - 1) / CSEG;
    } else if (tid == 64) {
        A.segs = (L.Ip + QSEG - 1) / QSEG;
    }
    if (blockIdx.x == 0) {
        for (int p = tid; p < L.P; p += ETHREADS) {
            if (ids) ids[p] = R.ids[p];
            if (gates) gates[p] = R.gates[p];
        }
    }
    __syncthreads();
    if (tid == 0) {
        A.quant_end = A.up_units + L.P * A.segs;
        A.down_end = A.quant_end + R.nchunks * S.geom[1].groups;
        A.units = A.down_end + ntok * A.csegs;
    }
    __syncthreads();
    if (warp == E_PRODUCER) produce<SU, SD>(S, smem_u32(smem), &map_up, &map_down, next);
    else if (warp < kQ8Consumers) consume<SU, SD>(S, smem_u32(smem), part);
    else finish<T>(S, part);
}

// Map of rows of `K` bytes in 8-byte elements, for boxes of 8 rows as long as a
// stage is deep (K >= 64).
bool encode_rows8(EncodeTiledFn enc, CUtensorMap *map, const int8_t *base, int K, int64_t rows, int64_t ld) {
    if (enc == nullptr) return false;
    const EGeom g(K, 1, 1, false);
    const cuuint64_t dims[2] = {(cuuint64_t)(K / 8), (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)ld};
    const cuuint32_t box[2] = {(cuuint32_t)(g.kb * kQ8Step / 8), 8};
    const cuuint32_t estr[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT64, 2, const_cast<int8_t *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Warps that share one 16-row tile's K: at least 4 steps each.
int warps_per_tile(int K) {
    const int steps = (K + kQ8Step - 1) / kQ8Step;
    int kw = 1;
    while (kw < MWARPS && steps >= 8 * kw) kw *= 2;
    return kw;
}

template <typename K, typename... A>
cudaError_t launch_pdl(K kern, int grid, int threads, size_t smem, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
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
cudaError_t launch_t(const Q8MoeArgs &a, unsigned char *ws) {
    // four elements at a time: one aligned access of each array, H a multiple of 4
    const int vec = a.H % 4 == 0 && a.ldx % 4 == 0 && a.ldr % 4 == 0 &&
                    reinterpret_cast<uintptr_t>(a.x) % (4 * sizeof(T)) == 0 &&
                    reinterpret_cast<uintptr_t>(a.router) % 16 == 0;
    cudaError_t e = launch_pdl(q8_route_kernel<T>, a.E * ((a.T + kRouteTokens - 1) / kRouteTokens) + a.T, RTHREADS, 0, a.stream, a.T, a.E, a.top_k, a.H, a.I,
                               (const T *)a.x, a.ldx, a.router, a.ldr, vec, ws);
    if (e != cudaSuccess) return e;
    if (reinterpret_cast<uintptr_t>(a.w_up) % 16 == 0 && reinterpret_cast<uintptr_t>(a.w_down) % 16 == 0) {
        const bool su = a.ldu % 16 != 0, sd = a.ldd % 16 != 0;
        auto kern = su ? (sd ? q8_expert_ring_kernel<T, true, true> : q8_expert_ring_kernel<T, true, false>)
                       : (sd ? q8_expert_ring_kernel<T, false, true> : q8_expert_ring_kernel<T, false, false>);
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)ESMEM);
        if (e != cudaSuccess) return e;
        alignas(64) CUtensorMap up = {}, down = {};
        if ((!su && a.H >= kQ8Step && !encode_rows8(a.encode, &up, a.w_up, a.H, (int64_t)a.E * 2 * a.I, a.ldu)) ||
            (!sd && a.I >= kQ8Step && !encode_rows8(a.encode, &down, a.w_down, a.I, (int64_t)a.E * a.H, a.ldd)))
            return cudaErrorInvalidValue;
        return launch_pdl(kern, a.sm_count > 0 ? a.sm_count : 1, ETHREADS, ESMEM, a.stream, up, down,
                          EGeom(a.H, a.I, 8, su), EGeom(a.I, a.H, 16, sd), a.T, a.E, a.top_k, a.H,
                          a.I, a.renormalize, a.w_up, a.ldu, a.s_up, a.w_down, a.ldd, a.s_down, (T *)a.out, a.ldo,
                          a.ids, a.gates, ws, a.err, a.wait_ns);
    }
    const int kw_up = warps_per_tile(a.H), kw_down = warps_per_tile(a.I);
    const int grid = 2 * (a.sm_count > 0 ? a.sm_count : 1);
    return launch_pdl(q8_expert_kernel<T>, grid, MTHREADS, 0, a.stream, a.T, a.E, a.top_k, a.H, a.I, a.renormalize,
                      a.w_up, a.ldu, a.s_up, a.w_down, a.ldd, a.s_down, (T *)a.out, a.ldo, a.ids, a.gates, ws, kw_up,
                      kw_down, a.err, a.wait_ns);
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
