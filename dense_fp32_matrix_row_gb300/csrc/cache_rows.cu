// cache_rows.cu -- heads of queries, keys and values on their way to attention:
// RMS norm and position rotation, quantisation into the paged cache, and the
// cache's rows back as floats.
//
//     p = x * weight,  each pair (p_a, p_b) turned by its angle
//     r = 1 / sqrt(mean x^2 + eps)         y = p * r
//     q = rint(p * (127 / max|p|))         scale = (max|p| / 127) * r
//
// The norm's factor r is one number for the head and a rotation is linear, so r
// is applied last: q depends on no summation order.  Each product and difference
// of a rotation is rounded by itself (no fused multiply-add), which makes q the
// same whole numbers wherever they are computed.
//
// Bound by memory: every head is read and written once.  A group of 8, 16 or 32
// lanes holds a head, 8 elements a lane: four pairs, whose angles belong to the
// lane and serve all the heads that the group takes of a token.
#include "cache.cuh"

namespace sgemm_gb300 {
namespace {

constexpr int kThreads = 256;

// Element (t, h, d) at p[t*ld + h*hs + d].
struct Heads {
    void *p;
    int n;
    int64_t ld, hs;
    template <typename T>
    __device__ __forceinline__ T *at(int64_t t, int h) const { return static_cast<T *>(p) + t * ld + h * hs; }
};

struct RowsParams {
    int64_t T;
    int D, pairs;          // rotated pairs: 0 without a rotation
    bool interleaved;
    Heads q, q_out, k, k_out, v;
    const float *qw, *kw;
    float eps;
    const float *cos, *sin;
    int64_t rows, ldt;
    const int64_t *positions;
    const int64_t *slots;  // nullptr: no cache
    sgemm_q8_cache cache;
    int q_units, k_units, units;      // per token: groups of U heads of queries, keys, values
    int64_t first, count;             // units of this launch, over all tokens
    unsigned *err;
};

// Where slot s of the cache lies: page and row; false for one outside it.
__device__ __forceinline__ bool place(const sgemm_q8_cache &c, int64_t s, int64_t &page, int &row) {
    if ((uint64_t)s >= (uint64_t)(c.blocks * c.page)) return false;
    if (s <= 0xffffffffll) {
        page = (uint32_t)s / (uint32_t)c.page;
        row = (int)((uint32_t)s - (uint32_t)page * (uint32_t)c.page);
    } else {
        page = s / c.page;
        row = (int)(s - page * c.page);
    }
    return true;
}

// The elements of four pairs (a, b): both halves of a rotated head, or eight
// neighbours.
template <typename T, bool VEC>
__device__ __forceinline__ void load_pairs(const T *p, int a0, int b0, bool neighbours, float (&a)[4], float (&b)[4]) {
    if (neighbours) {
        if constexpr (VEC) {
            float u[4], w[4];
            load_vec<T, 4>(p + a0, u);
            load_vec<T, 4>(p + a0 + 4, w);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                a[i] = u[2 * i]; b[i] = u[2 * i + 1];
                a[i + 2] = w[2 * i]; b[i + 2] = w[2 * i + 1];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) { a[i] = to_f32<T>(p[a0 + 2 * i]); b[i] = to_f32<T>(p[a0 + 2 * i + 1]); }
        }
    } else if constexpr (VEC) {
        load_vec<T, 4>(p + a0, a);
        load_vec<T, 4>(p + b0, b);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) { a[i] = to_f32<T>(p[a0 + i]); b[i] = to_f32<T>(p[b0 + i]); }
    }
}

template <typename T, bool VEC>
__device__ __forceinline__ void store_pairs(T *p, int a0, int b0, bool neighbours, const float (&a)[4],
                                            const float (&b)[4]) {
    if (neighbours) {
        if constexpr (VEC) {
            const float u[4] = {a[0], b[0], a[1], b[1]}, w[4] = {a[2], b[2], a[3], b[3]};
            store_vec<T, 4>(p + a0, u);
            store_vec<T, 4>(p + a0 + 4, w);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) { p[a0 + 2 * i] = from_f32<T>(a[i]); p[a0 + 2 * i + 1] = from_f32<T>(b[i]); }
        }
    } else if constexpr (VEC) {
        store_vec<T, 4>(p + a0, a);
        store_vec<T, 4>(p + b0, b);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) { p[a0 + i] = from_f32<T>(a[i]); p[b0 + i] = from_f32<T>(b[i]); }
    }
}

// The same as whole numbers (the cache's rows are 16-byte aligned; the halves of
// a rotated part are 4-byte aligned where VEC says so).
template <bool VEC>
__device__ __forceinline__ void store_pairs_q(int8_t *p, int a0, int b0, bool neighbours, const RowQuant &rq,
                                              const float (&a)[4], const float (&b)[4]) {
    if (neighbours && VEC) {
        const float u[8] = {a[0], b[0], a[1], b[1], a[2], b[2], a[3], b[3]};
        store_q<8>(p + a0, rq, u);
    } else if (VEC) {
        store_q<4>(p + a0, rq, a);
        store_q<4>(p + b0, rq, b);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            p[a0 + (neighbours ? 2 * i : i)] = (int8_t)rq(a[i]);
            p[neighbours ? a0 + 2 * i + 1 : b0 + i] = (int8_t)rq(b[i]);
        }
    }
}

// LANES lanes to a head, U heads of one kind and token to a group.  Without VEC
// a lane's pairs may straddle the end of the rotated part, and are taken one by
// one (elem says where).
template <typename T, bool VEC, int LANES, int U>
__global__ void __launch_bounds__(kThreads) head_rows_kernel(const __grid_constant__ RowsParams a) {
    const int lane = threadIdx.x % LANES;
    const int64_t idx = (int64_t)blockIdx.x * (kThreads / LANES) + threadIdx.x / LANES;
    const bool here = idx < a.count;
    const uint32_t local = here ? (uint32_t)idx : 0u;
    const uint32_t tok = local / (uint32_t)a.units;
    const int64_t t = a.first + tok;
    int unit = (int)(local - tok * (uint32_t)a.units);
    // which heads: queries, keys or values
    const bool is_q = unit < a.q_units, is_k = !is_q && unit < a.q_units + a.k_units;
    if (!is_q) unit -= is_k ? a.q_units : a.q_units + a.k_units;
    const Heads in = is_q ? a.q : is_k ? a.k : a.v;
    const float *weight = is_q ? a.qw : is_k ? a.kw : nullptr;
    const int h0 = unit * U;
    const bool active = here && 8 * lane < a.D;

    // the lane's pairs
    const int p0 = 4 * lane;
    const bool turned = (is_q || is_k) && a.pairs > 0;
    const bool neighbours = !turned || a.interleaved || p0 >= a.pairs;
    int ea[4], eb[4];
    if constexpr (!VEC) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool nb = !turned || a.interleaved || p0 + i >= a.pairs;
            ea[i] = nb ? 2 * (p0 + i) : p0 + i;
            eb[i] = nb ? 2 * (p0 + i) + 1 : p0 + i + a.pairs;
        }
    }
    const int a0 = neighbours ? 2 * p0 : p0, b0 = p0 + a.pairs;

    float xa[U][4], xb[U][4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const bool on = active && h0 + u < in.n;
        if (on) {
            const T *src = in.at<T>(t, h0 + u);
            if constexpr (VEC) {
                load_pairs<T, true>(src, a0, b0, neighbours, xa[u], xb[u]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) { xa[u][i] = to_f32<T>(src[ea[i]]); xb[u][i] = to_f32<T>(src[eb[i]]); }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) xa[u][i] = xb[u][i] = 0.0f;
        }
    }

    // the token's place in the tables and in the cache
    bool fine = here;
    int64_t pos = t;
    if (a.pairs > 0) {
        if (here && a.positions) pos = a.positions[t];
        if ((uint64_t)pos >= (uint64_t)a.rows) {
            if (here && lane == 0) record_error(a.err, kErrBadIndex);
            fine = false;
        }
    }
    float c[4], s[4];
    if (turned && fine && active) {
        const float *pc = a.cos + pos * a.ldt, *ps = a.sin + pos * a.ldt;
        if constexpr (VEC) {
            if (p0 < a.pairs) {
                load_vec<float, 4>(pc + p0, c);
                load_vec<float, 4>(ps + p0, s);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (p0 + i < a.pairs) { c[i] = pc[p0 + i]; s[i] = ps[p0 + i]; }
        }
    }
    float wa[4], wb[4];
    if (weight && active) {
        if constexpr (VEC) {
            load_pairs<float, true>(weight, a0, b0, neighbours, wa, wb);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) { wa[i] = weight[ea[i]]; wb[i] = weight[eb[i]]; }
        }
    }
    const bool cached = a.slots != nullptr && !is_q;
    int64_t page = 0;
    int row = 0;
    bool stored = false;
    if (cached && fine) {
        const int64_t slot = a.slots[t];
        stored = place(a.cache, slot, page, row);
        if (!stored && slot >= 0 && lane == 0) record_error(a.err, kErrBadIndex);
    }

#pragma unroll
    for (int u = 0; u < U; ++u) {
        float ss = 0.0f;
        if (weight) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                ss = fmaf(xa[u][i], xa[u][i], ss);
                ss = fmaf(xb[u][i], xb[u][i], ss);
            }
        }
        float pa[4], pb[4];
        uint32_t mx = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            pa[i] = xa[u][i];
            pb[i] = xb[u][i];
            if (weight && active) {
                pa[i] = __fmul_rn(pa[i], wa[i]);
                pb[i] = __fmul_rn(pb[i], wb[i]);
            }
            if (turned && active && p0 + i < a.pairs) {
                const float x = pa[i], y = pb[i];
                pa[i] = __fsub_rn(__fmul_rn(x, c[i]), __fmul_rn(y, s[i]));
                pb[i] = __fadd_rn(__fmul_rn(y, c[i]), __fmul_rn(x, s[i]));
            }
            mx = max(mx, max(abs_bits(pa[i]), abs_bits(pb[i])));
        }
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) {
            ss += __shfl_xor_sync(0xffffffffu, ss, o);
            mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        }
        float r = 1.0f, lift = 1.0f;
        if (weight) {
            r = inv_rms(ss, a.D, a.eps);
            lift = norm_lift(ss, a.D, a.eps, mx);
        }
        if (__any_sync(0xffffffffu, lift != 1.0f)) {   // squares beyond FP32's range: rare
            float s2 = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float va = xa[u][i] * lift, vb = xb[u][i] * lift;
                s2 = fmaf(va, va, s2);
                s2 = fmaf(vb, vb, s2);
            }
#pragma unroll
            for (int o = LANES / 2; o > 0; o >>= 1) s2 += __shfl_xor_sync(0xffffffffu, s2, o);
            if (lift != 1.0f) r = inv_rms(s2, a.D, a.eps * lift * lift);
        }
        const int h = h0 + u;
        if (!active || !fine || h >= in.n) continue;
        if (cached) {
            if (!stored) continue;
            const RowQuant rq(mx);
            const int64_t at = (int64_t)h * a.cache.page + row;
            int8_t *dst = is_k ? a.cache.k + page * a.cache.k_stride : a.cache.v + page * a.cache.v_stride;
            dst += at * a.D;
            if constexpr (VEC) {
                store_pairs_q<true>(dst, a0, b0, neighbours, rq, pa, pb);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) { dst[ea[i]] = (int8_t)rq(pa[i]); dst[eb[i]] = (int8_t)rq(pb[i]); }
            }
            if (lane == 0) {
                float *scale = is_k ? a.cache.k_scale + page * a.cache.k_scale_stride
                                    : a.cache.v_scale + page * a.cache.v_scale_stride;
                scale[at] = row_scale(rq, lift, r);
            }
        } else {
            const Heads o = is_q ? a.q_out : a.k_out;
            T *dst = o.at<T>(t, h);
            if (weight) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    pa[i] = lift == 1.0f ? pa[i] * r : pa[i] * lift * r;
                    pb[i] = lift == 1.0f ? pb[i] * r : pb[i] * lift * r;
                }
            }
            if constexpr (VEC) {
                store_pairs<T, true>(dst, a0, b0, neighbours, pa, pb);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) { dst[ea[i]] = from_f32<T>(pa[i]); dst[eb[i]] = from_f32<T>(pb[i]); }
            }
        }
    }
}

struct ReadParams {
    int64_t N;
    int D;
    sgemm_q8_cache cache;
    const int64_t *slots;
    Heads k_out, v_out;
    int k_units, units;
    int64_t first, count;
    unsigned *err;
};

// LANES lanes to a row, 16 elements a lane; U heads of one token to a group.
template <typename T, bool VEC, int LANES, int U>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const __grid_constant__ ReadParams a) {
    const int lane = threadIdx.x % LANES;
    const int64_t idx = (int64_t)blockIdx.x * (kThreads / LANES) + threadIdx.x / LANES;
    if (idx >= a.count) return;
    const uint32_t tok = (uint32_t)idx / (uint32_t)a.units;
    const int64_t n = a.first + tok;
    int unit = (int)((uint32_t)idx - tok * (uint32_t)a.units);
    const bool is_k = unit < a.k_units;
    if (!is_k) unit -= a.k_units;
    const int64_t slot = a.slots[n];
    int64_t page;
    int row;
    if (!place(a.cache, slot, page, row)) {
        if (slot >= 0 && lane == 0) record_error(a.err, kErrBadIndex);
        return;
    }
    if (16 * lane >= a.D) return;
    const int h0 = unit * U, heads = (int)a.cache.heads;
    const int8_t *src = (is_k ? a.cache.k + page * a.cache.k_stride : a.cache.v + page * a.cache.v_stride);
    const float *scales = is_k ? a.cache.k_scale + page * a.cache.k_scale_stride
                               : a.cache.v_scale + page * a.cache.v_scale_stride;
    uint4 w[U];
    float sc[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (h0 + u < heads) {
            const int64_t at = (int64_t)(h0 + u) * a.cache.page + row;
            w[u] = *reinterpret_cast<const uint4 *>(src + at * a.D + 16 * lane);
            sc[u] = scales[at];
        }
    }
    const Heads out = is_k ? a.k_out : a.v_out;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (h0 + u >= heads) break;
        const uint32_t word[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = (float)(int8_t)(word[i / 4] >> (8 * (i % 4))) * sc[u];
        T *dst = out.at<T>(n, h0 + u) + 16 * lane;
        if constexpr (VEC) {
            constexpr int V = 16 / (int)sizeof(T);
#pragma unroll
            for (int i = 0; i < 16 / V; ++i) {
                float part[V];
#pragma unroll
                for (int e = 0; e < V; ++e) part[e] = v[V * i + e];
                store_vec<T, V>(dst + V * i, part);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) dst[i] = from_f32<T>(v[i]);
        }
    }
}

Heads heads_of(const sgemm_heads &h) { return Heads{h.p, h.p ? (int)h.heads : 0, h.ld, h.hs}; }

// Whether accesses of `bytes` to every head start on their boundary.
bool aligned(const Heads &h, int es, int bytes) {
    if (h.p == nullptr || h.n == 0) return true;
    return reinterpret_cast<uintptr_t>(h.p) % bytes == 0 && h.ld * es % bytes == 0 && (h.n == 1 || h.hs * es % bytes == 0);
}
bool aligned(const void *p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

// Tokens of one launch: its units are counted in 32 bits.
constexpr int64_t kMostUnits = int64_t(1) << 30;

template <typename T, bool VEC, int LANES, int U>
cudaError_t rows_launch(RowsParams p, cudaStream_t stream) {
    const int64_t step = kMostUnits / p.units;
    for (int64_t t = 0; t < p.T; t += step) {
        const int64_t n = p.T - t < step ? p.T - t : step;
        p.first = t;
        p.count = n * p.units;
        const int64_t per = kThreads / LANES;
        head_rows_kernel<T, VEC, LANES, U><<<(unsigned)((p.count + per - 1) / per), kThreads, 0, stream>>>(p);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <typename T, bool VEC, int U>
cudaError_t rows_lanes(const RowsParams &p, cudaStream_t stream) {
    if (p.D <= 64) return rows_launch<T, VEC, 8, U>(p, stream);
    if (p.D <= 128) return rows_launch<T, VEC, 16, U>(p, stream);
    return rows_launch<T, VEC, 32, U>(p, stream);
}

template <typename T>
cudaError_t rows_type(RowsParams p, cudaStream_t stream, int sm_count) {
    constexpr int es = sizeof(T), bytes = 4 * es;
    const bool vec = p.pairs % 4 == 0 && aligned(p.q, es, bytes) && aligned(p.k, es, bytes) && aligned(p.v, es, bytes) &&
                     aligned(p.q_out, es, bytes) && aligned(p.k_out, es, bytes) && aligned(p.cos, 16) &&
                     aligned(p.sin, 16) && p.ldt % 4 == 0 && aligned(p.qw, 16) && aligned(p.kw, 16);
    auto split = [&](int u) {
        p.q_units = (p.q.n + u - 1) / u;
        p.k_units = (p.k.n + u - 1) / u;
        p.units = p.q_units + p.k_units + (p.v.n + u - 1) / u;
    };
    if (!vec) {
        split(1);
        return rows_lanes<T, false, 1>(p, stream);
    }
    // Four heads to a group once single ones would fill every SM: a token's angles
    // are then loaded once for four heads, and four heads' loads are under way together.
    const int lanes = p.D <= 64 ? 8 : p.D <= 128 ? 16 : 32;
    split(1);
    if (p.T * p.units * lanes <= (int64_t)sm_count * 2048) return rows_lanes<T, true, 1>(p, stream);
    split(4);
    return rows_lanes<T, true, 4>(p, stream);
}

template <typename T, bool VEC, int LANES, int U>
cudaError_t read_launch(ReadParams p, cudaStream_t stream) {
    const int per_kind = ((int)p.cache.heads + U - 1) / U;
    p.k_units = p.k_out.n > 0 ? per_kind : 0;
    p.units = p.k_units + (p.v_out.n > 0 ? per_kind : 0);
    const int64_t step = kMostUnits / p.units;
    for (int64_t t = 0; t < p.N; t += step) {
        const int64_t n = p.N - t < step ? p.N - t : step;
        p.first = t;
        p.count = n * p.units;
        const int64_t per = kThreads / LANES;
        cache_read_kernel<T, VEC, LANES, U><<<(unsigned)((p.count + per - 1) / per), kThreads, 0, stream>>>(p);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <typename T>
cudaError_t read_type(const ReadParams &p, cudaStream_t stream) {
    const bool vec = aligned(p.k_out, sizeof(T), 16) && aligned(p.v_out, sizeof(T), 16);
    if (p.D <= 64) return vec ? read_launch<T, true, 4, 2>(p, stream) : read_launch<T, false, 4, 1>(p, stream);
    if (p.D <= 128) return vec ? read_launch<T, true, 8, 2>(p, stream) : read_launch<T, false, 8, 1>(p, stream);
    return vec ? read_launch<T, true, 16, 2>(p, stream) : read_launch<T, false, 16, 1>(p, stream);
}

}  // namespace

cudaError_t launch_head_rows(const HeadRowsArgs &a) {
    RowsParams p{};
    p.T = a.T;
    p.D = a.D;
    p.pairs = (int)(a.rotary.dims / 2);
    p.interleaved = a.rotary.interleaved != 0;
    p.q = heads_of(a.q); p.q_out = heads_of(a.q_out);
    p.k = heads_of(a.k); p.k_out = heads_of(a.k_out);
    p.v = heads_of(a.v);
    p.qw = a.q_weight; p.kw = a.k_weight; p.eps = a.eps;
    p.cos = a.rotary.cos; p.sin = a.rotary.sin;
    p.rows = a.rotary.rows; p.ldt = a.rotary.ld; p.positions = a.rotary.positions;
    p.slots = a.slots; p.cache = a.cache;
    p.err = a.err;
    return a.type == kTypeBf16 ? rows_type<__nv_bfloat16>(p, a.stream, a.sm_count)
                               : rows_type<float>(p, a.stream, a.sm_count);
}

cudaError_t launch_cache_read(const CacheReadArgs &a) {
    ReadParams p{};
    p.N = a.N;
    p.D = (int)a.cache.dim;
    p.cache = a.cache; p.slots = a.slots;
    p.k_out = heads_of(a.k_out); p.v_out = heads_of(a.v_out);
    p.err = a.err;
    return a.type == kTypeBf16 ? read_type<__nv_bfloat16>(p, a.stream) : read_type<float>(p, a.stream);
}

}  // namespace sgemm_gb300
