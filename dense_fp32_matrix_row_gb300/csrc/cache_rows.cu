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
// Every head is read and written once.  FP32 is bound by memory; in bf16 neither memory
// nor the issue slots are full (67% of them taken, a quarter of a warp's time spent
// waiting for loads, and a quarter ready behind another warp).  A group of 8, 16 or 32 lanes holds a head, 8 elements a lane: four
// pairs, whose angles belong to the lane and serve all the heads that the group
// takes of a token.
//
// Measured: 8192 tokens of 32 + 8 heads of 128, bf16, 172 MB, 31.5 us, 5.5 TB/s (82% of
// a copy's); in FP32, 340 MB, 51.2 us, 6.6 TB/s.  With keys and 8 heads of values into
// the cache, 189 MB, 41.2 us, 4.6 TB/s (69%; FP32, 357 MB, 61.5 us, 87%): its blocks hold
// more registers, eight to an SM instead of nine.  Keys and values alone, 32768 tokens of
// 8 + 8 heads, 204 MB, 58.3 us (52%).  18432 tokens of 8 + 8 heads read back, 114 MB, 20.1
// us, 5.7 TB/s (85%).  One token 1.5 us.  Not kept (first case): 16 elements
// a lane 40 us, eight heads to a group one half after the other 44, one kernel for
// floats and cache 33.0, a question for each load whether its head is there 34.8.
#include "cache.cuh"

namespace sgemm_gb300 {
namespace {

constexpr int kThreads = 128;     // 256: 3% longer, 512: 8%

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
    float eps, over_dim;   // 1 / D
    float least;           // sums of squares below it may have lost some
    const float *cos, *sin;
    int64_t rows, ldt;
    const int64_t *positions;
    const int64_t *slots;  // nullptr: no cache
    sgemm_q8_cache cache;
    // units: groups of U heads; per token, and of this launch over all its tokens
    int q_units, k_units, float_units, cache_units;
    int64_t first, float_count, cache_count;
    unsigned cache_begin, cache_blocks;
    int sms;
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

// Four elements as they come from memory.
template <typename T>
struct Quad {
    uint32_t w[sizeof(T)];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T); ++i) w[i] = 0;
    }
    __device__ __forceinline__ void load(const T *p) {
        if constexpr (sizeof(T) == 4) {
            const uint4 u = *reinterpret_cast<const uint4 *>(p);
            w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
        } else {
            const uint2 u = *reinterpret_cast<const uint2 *>(p);
            w[0] = u.x; w[1] = u.y;
        }
    }
    // From four places, one by one.
    __device__ __forceinline__ void gather(const T *p, const int (&at)[4]) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(p[at[i]]);
        } else {
            const unsigned short *h = reinterpret_cast<const unsigned short *>(p);
#pragma unroll
            for (int i = 0; i < 2; ++i) w[i] = (uint32_t)h[at[2 * i]] | (uint32_t)h[at[2 * i + 1]] << 16;
        }
    }
    // Elements 2i and 2i + 1.
    __device__ __forceinline__ float2 pair(int i) const {
        if constexpr (sizeof(T) == 4) return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
        else return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    }
};

// 1 / sqrt(mean square + eps) from a head's sum of squares: rsqrtf, good to 2 units in
// the last place.
__device__ __forceinline__ float norm_factor(float ss, float over_dim, float eps) { return rsqrtf(fmaf(ss, over_dim, eps)); }

// What a head's squares are lifted by, with its bit in `huge` or `tiny`.
__device__ __forceinline__ float lift_of(uint32_t huge, uint32_t tiny, int u) {
    return huge >> u & 1 ? kTwoM100 : tiny >> u & 1 ? kTwo100 : 1.0f;
}

// x * c - y * s and y * c + x * s, each product and sum rounded by itself.  (Not two
// elements at a time: such products came out fused with the sum, whatever their
// form, which moved one whole number in a million.)
__device__ __forceinline__ void rotate(float &x, float &y, float c, float s) {
    const float px = x, py = y;
    x = __fsub_rn(__fmul_rn(px, c), __fmul_rn(py, s));
    y = __fadd_rn(__fmul_rn(py, c), __fmul_rn(px, s));
}

// LANES lanes to a head, U heads of one kind and token to a group.  A lane has two
// quads of a head's elements.  INTER false: the first elements of four rotated
// pairs, and the second ones; true: four pairs, one behind another.  Lanes behind
// the rotated part have eight neighbours.  Without VEC the rotated part may end
// within a quad, and elements are taken one by one.  FULL: no lane is without
// elements, and heads that are not there are loaded as the last one, rather than
// asked for one by one.  CACHED: keys and values into the cache; otherwise queries
// and keys to floats.
template <typename T, bool VEC, bool FULL, bool INTER, bool CACHED, int LANES, int U>
__device__ __forceinline__ void head_rows(const RowsParams &a, uint32_t idx, uint32_t count, int units, int first_units) {
    constexpr uint32_t ALL = 0xffffffffu;
    const int lane = threadIdx.x % LANES;
    const bool here = idx < count;
    const uint32_t tok = here ? idx / (uint32_t)units : 0u;
    const int64_t t = a.first + tok;
    int unit = here ? (int)(idx - tok * (uint32_t)units) : 0;
    // the first kind: queries, or keys for the cache; the second: keys, or values
    const bool one = unit < first_units;
    if (!one) unit -= first_units;
    const int h0 = unit * U;
    const bool active = FULL || (here && 8 * lane < a.D);

    // the token's places, asked for first
    int64_t pos = t, slot = -1;
    if (a.pairs > 0 && a.positions && here) pos = a.positions[t];
    if (CACHED && here) slot = a.slots[t];

    // where the lane's elements are, and whether they are rotated
    const int p0 = 4 * lane;
    const bool rotates = (one || !CACHED) && a.pairs > 0;
    int at0[4], at1[4];         // VEC: the quads' first elements alone
    bool turn[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (INTER || VEC) {
            turn[i] = rotates && p0 + (VEC ? 0 : i) < a.pairs;
            const bool halves = !INTER && turn[i];
            at0[i] = (halves ? p0 : 2 * p0) + i;
            at1[i] = (halves ? p0 + a.pairs : 2 * p0 + 4) + i;
        } else {                // a pair of neighbours stands for a pair behind the rotated part
            turn[i] = rotates && p0 + i < a.pairs;
            at0[i] = turn[i] ? p0 + i : 2 * (p0 + i);
            at1[i] = turn[i] ? p0 + i + a.pairs : 2 * (p0 + i) + 1;
        }
    }

    const Heads &in = CACHED ? (one ? a.k : a.v) : (one ? a.q : a.k);
    const int heads = here ? min(in.n - h0, U) : 0;
    Quad<T> x0[U], x1[U];
    {
        const T *src = in.at<T>(t, h0);
        const int64_t hs = in.hs;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if constexpr (FULL) {
                const T *from = src + min(u, max(heads - 1, 0)) * hs;
                x0[u].load(from + at0[0]);
                x1[u].load(from + at1[0]);
            } else if (active && u < heads) {
                if constexpr (VEC) {
                    x0[u].load(src + u * hs + at0[0]);
                    x1[u].load(src + u * hs + at1[0]);
                } else {
                    x0[u].gather(src + u * hs, at0);
                    x1[u].gather(src + u * hs, at1);
                }
            } else {
                x0[u].clear();
                x1[u].clear();
            }
        }
    }
    bool fine = here;
    if (a.pairs > 0 && (uint64_t)pos >= (uint64_t)a.rows) {
        if (here && lane == 0) record_error(a.err, kErrBadIndex);
        fine = false;
    }
    Quad<float> c, s;
    if (rotates && fine && active) {
        const float *pc = a.cos + pos * a.ldt + p0, *ps = a.sin + pos * a.ldt + p0;
        if constexpr (VEC) {
            if (turn[0]) {
                c.load(pc);
                s.load(ps);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (turn[i]) { c.w[i] = __float_as_uint(pc[i]); s.w[i] = __float_as_uint(ps[i]); }
        }
    }
    const float *weight = CACHED ? (one ? a.kw : nullptr) : (one ? a.qw : a.kw);
    Quad<float> w0, w1;
    if (weight && active) {
        if constexpr (VEC) {
            w0.load(weight + at0[0]);
            w1.load(weight + at1[0]);
        } else {
            w0.gather(weight, at0);
            w1.gather(weight, at1);
        }
    }

    // the norms' factors
    float r[U];
    bool lifted = false;
    uint32_t huge = 0, tiny = 0;        // of `lifted`: heads, a bit each
    if (__any_sync(ALL, weight != nullptr)) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            r[u] = 0.0f;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                r[u] = fmaf(x0[u].pair(i).x, x0[u].pair(i).x, r[u]);
                r[u] = fmaf(x0[u].pair(i).y, x0[u].pair(i).y, r[u]);
                r[u] = fmaf(x1[u].pair(i).x, x1[u].pair(i).x, r[u]);
                r[u] = fmaf(x1[u].pair(i).y, x1[u].pair(i).y, r[u]);
            }
        }
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1)
#pragma unroll
            for (int u = 0; u < U; ++u) r[u] += __shfl_xor_sync(ALL, r[u], o);
        bool odd = false;
#pragma unroll
        for (int u = 0; u < U; ++u) odd |= r[u] > kLargest || r[u] < a.least;
        lifted = __any_sync(ALL, odd && weight != nullptr);
        if (lifted) {           // squares beyond FP32's range: rare
#pragma unroll
            for (int u = 0; u < U; ++u) {
                huge |= (uint32_t)(weight && r[u] > kLargest) << u;
                tiny |= (uint32_t)(weight && r[u] < a.least) << u;
                const float lift = lift_of(huge, tiny, u);
                float s2 = 0.0f;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float2 v0 = x0[u].pair(i), v1 = x1[u].pair(i);
                    s2 = fmaf(v0.x * lift, v0.x * lift, s2);
                    s2 = fmaf(v0.y * lift, v0.y * lift, s2);
                    s2 = fmaf(v1.x * lift, v1.x * lift, s2);
                    s2 = fmaf(v1.y * lift, v1.y * lift, s2);
                }
#pragma unroll
                for (int o = LANES / 2; o > 0; o >>= 1) s2 += __shfl_xor_sync(ALL, s2, o);
                r[u] = norm_factor(s2, a.over_dim, a.eps * lift * lift);
            }
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u) r[u] = norm_factor(r[u], a.over_dim, a.eps);
        }
    }

    // where the results go
    bool stored = active && fine;
    int8_t *rows = nullptr;
    float *scales = nullptr;
    T *dst = nullptr;
    if constexpr (CACHED) {
        if (fine) {
            int64_t page = 0;
            int row = 0;
            if (place(a.cache, slot, page, row)) {
                const int64_t at = (int64_t)h0 * a.cache.page + row;
                rows = (one ? a.cache.k + page * a.cache.k_stride : a.cache.v + page * a.cache.v_stride) + at * a.D;
                scales = (one ? a.cache.k_scale + page * a.cache.k_scale_stride
                              : a.cache.v_scale + page * a.cache.v_scale_stride) + at;
            } else {
                stored = false;
                if (slot >= 0 && lane == 0) record_error(a.err, kErrBadIndex);
            }
        }
    } else {
        dst = (one ? a.q_out : a.k_out).at<T>(t, h0);
    }
    const int64_t step = CACHED ? a.cache.page * a.D : (one ? a.q_out : a.k_out).hs;

#pragma unroll
    for (int u = 0; u < U; ++u) {
        float2 f0[2], f1[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            f0[i] = x0[u].pair(i);
            f1[i] = x1[u].pair(i);
        }
        if (weight) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                f0[i] = __fmul2_rn(f0[i], w0.pair(i));
                f1[i] = __fmul2_rn(f1[i], w1.pair(i));
            }
        }
        if constexpr (INTER) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (turn[i]) rotate(f0[i].x, f0[i].y, __uint_as_float(c.w[i]), __uint_as_float(s.w[i]));
                if (turn[i + 2]) rotate(f1[i].x, f1[i].y, __uint_as_float(c.w[i + 2]), __uint_as_float(s.w[i + 2]));
            }
        } else if constexpr (VEC) {
            if (turn[0]) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    rotate(f0[i].x, f1[i].x, c.pair(i).x, s.pair(i).x);
                    rotate(f0[i].y, f1[i].y, c.pair(i).y, s.pair(i).y);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (turn[2 * i]) rotate(f0[i].x, f1[i].x, c.pair(i).x, s.pair(i).x);
                if (turn[2 * i + 1]) rotate(f0[i].y, f1[i].y, c.pair(i).y, s.pair(i).y);
            }
        }
        if constexpr (CACHED) {
            uint32_t mx = 0;
            if (active) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    mx = max(max(mx, max(abs_bits(f0[i].x), abs_bits(f0[i].y))), max(abs_bits(f1[i].x), abs_bits(f1[i].y)));
            }
#pragma unroll
            for (int o = LANES / 2; o > 0; o >>= 1) mx = max(mx, __shfl_xor_sync(ALL, mx, o));
            if (stored && u < heads) {
                const RowQuant rq(mx);
                const float v0[4] = {f0[0].x, f0[0].y, f0[1].x, f0[1].y};
                const float v1[4] = {f1[0].x, f1[0].y, f1[1].x, f1[1].y};
                int8_t *to = rows + u * step;
                if constexpr (VEC) {
                    store_q<4>(to + at0[0], rq, v0);
                    store_q<4>(to + at1[0], rq, v1);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) { to[at0[i]] = (int8_t)rq(v0[i]); to[at1[i]] = (int8_t)rq(v1[i]); }
                }
                if (lane == 0) scales[u * a.cache.page] = row_scale(rq, lifted ? lift_of(huge, tiny, u) : 1.0f, weight ? r[u] : 1.0f);
            }
        } else {
            if (lifted) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float lift = lift_of(huge, tiny, u);
                    f0[i] = __fmul2_rn(f0[i], make_float2(lift, lift));
                    f1[i] = __fmul2_rn(f1[i], make_float2(lift, lift));
                }
            }
            if (weight) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    f0[i] = __fmul2_rn(f0[i], make_float2(r[u], r[u]));
                    f1[i] = __fmul2_rn(f1[i], make_float2(r[u], r[u]));
                }
            }
            if (stored && u < heads) {
                const float v0[4] = {f0[0].x, f0[0].y, f0[1].x, f0[1].y};
                const float v1[4] = {f1[0].x, f1[0].y, f1[1].x, f1[1].y};
                T *to = dst + u * step;
                if constexpr (VEC) {
                    store_vec<T, 4>(to + at0[0], v0);
                    store_vec<T, 4>(to + at1[0], v1);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) { to[at0[i]] = from_f32<T>(v0[i]); to[at1[i]] = from_f32<T>(v1[i]); }
                }
            }
        }
    }
}

// With MIXED, cache_blocks blocks from cache_begin on write the cache, the others floats:
// those alone without it.  The cache first where there is more than a wave, as its blocks
// take longer and the end is short (8192 tokens 40.6 us, floats first 43.1, both kinds mixed
// 42.2), otherwise last (777 FP32 tokens of 20 heads of 96, read back as well: 6.8 us, first 7.7).
template <typename T, bool VEC, bool FULL, bool INTER, bool MIXED, int LANES, int U>
__global__ void __launch_bounds__(kThreads, MIXED ? 8 : 9) head_rows_kernel(const __grid_constant__ RowsParams a) {
    pdl_wait();
    pdl_trigger();
    const uint32_t group = threadIdx.x / LANES, per = kThreads / LANES;
    if (!MIXED || blockIdx.x - a.cache_begin >= a.cache_blocks) {
        const uint32_t at = MIXED && a.cache_begin == 0 ? blockIdx.x - a.cache_blocks : blockIdx.x;
        head_rows<T, VEC, FULL, INTER, false, LANES, U>(a, at * per + group, (uint32_t)a.float_count, a.float_units, a.q_units);
    } else if constexpr (MIXED) {
        head_rows<T, VEC, FULL, INTER, true, LANES, U>(a, (blockIdx.x - a.cache_begin) * per + group,
                                                       (uint32_t)a.cache_count, a.cache_units, a.k_units);
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

// Four bytes times sc, rounded once: a byte in the last bits of 2^23 makes 2^23 + itself.
__device__ __forceinline__ void bytes_to_f32(uint32_t w, float sc, float *v) {
    const uint32_t u = w ^ 0x80808080u;
    const float2 back = make_float2(-8388736.0f, -8388736.0f), by = make_float2(sc, sc);
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        float2 x = make_float2(__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440 + i)),
                               __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7441 + i)));
        x = __fmul2_rn(__fadd2_rn(x, back), by);
        v[i] = x.x;
        v[i + 1] = x.y;
    }
}

// LANES lanes to a row, 16 bytes of result a lane (IT times); U heads of one token to
// a group.
template <typename T, bool VEC, int LANES, int IT, int U>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const __grid_constant__ ReadParams a) {
    constexpr int V = 16 / (int)sizeof(T);
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x % LANES;
    const uint32_t idx = blockIdx.x * (uint32_t)(kThreads / LANES) + threadIdx.x / LANES;
    if (idx >= (uint32_t)a.count) return;
    // 16 tokens, then the next heads of the same 16: a page's rows of one head lie together
    const uint32_t tile = idx / 16 / (uint32_t)a.units;
    const int64_t n = a.first + tile * 16 + idx % 16;
    int unit = (int)(idx / 16 - tile * (uint32_t)a.units);
    if (n >= a.N) return;
    const int64_t slot = a.slots[n];
    const bool is_k = unit < a.k_units;
    if (!is_k) unit -= a.k_units;
    int64_t page;
    int row;
    if (!place(a.cache, slot, page, row)) {
        if (slot >= 0 && lane == 0) record_error(a.err, kErrBadIndex);
        return;
    }
    const int h0 = unit * U, heads = (int)a.cache.heads;
    const int8_t *src = (is_k ? a.cache.k + page * a.cache.k_stride : a.cache.v + page * a.cache.v_stride);
    const float *scales = is_k ? a.cache.k_scale + page * a.cache.k_scale_stride
                               : a.cache.v_scale + page * a.cache.v_scale_stride;
    uint32_t w[U][IT][V / 4];
    float sc[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (h0 + u >= heads) continue;
        const int64_t at = (int64_t)(h0 + u) * a.cache.page + row;
        sc[u] = scales[at];
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int e = (lane + i * LANES) * V;
            if (e >= a.D) continue;
            const int8_t *p = src + at * a.D + e;
            if constexpr (V == 8) {
                const uint2 x = *reinterpret_cast<const uint2 *>(p);
                w[u][i][0] = x.x;
                w[u][i][1] = x.y;
            } else {
                w[u][i][0] = *reinterpret_cast<const uint32_t *>(p);
            }
        }
    }
    const Heads out = is_k ? a.k_out : a.v_out;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (h0 + u >= heads) continue;
        T *dst = out.at<T>(n, h0 + u);
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int e = (lane + i * LANES) * V;
            if (e >= a.D) continue;
            float v[V];
#pragma unroll
            for (int k = 0; k < V / 4; ++k) bytes_to_f32(w[u][i][k], sc[u], v + 4 * k);
            if constexpr (VEC) {
                store_vec<T, V>(dst + e, v);
            } else {
#pragma unroll
                for (int k = 0; k < V; ++k) dst[e + k] = from_f32<T>(v[k]);
            }
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

template <typename T, bool VEC, bool FULL, bool INTER, int LANES, int U>
cudaError_t rows_launch(RowsParams p, cudaStream_t stream) {
    const bool cached = p.slots != nullptr;
    p.q_units = (p.q.n + U - 1) / U;
    p.k_units = (p.k.n + U - 1) / U;
    p.float_units = p.q_units + (cached ? 0 : p.k_units);
    p.cache_units = cached ? 2 * p.k_units : 0;         // as many values as keys
    const int64_t step = kMostUnits / (p.float_units > p.cache_units ? p.float_units : p.cache_units);
    for (int64_t t = 0; t < p.T; t += step) {
        const int64_t n = p.T - t < step ? p.T - t : step, per = kThreads / LANES;
        p.first = t;
        p.float_count = n * p.float_units;
        p.cache_count = n * p.cache_units;
        const unsigned float_blocks = (unsigned)((p.float_count + per - 1) / per);
        p.cache_blocks = (unsigned)((p.cache_count + per - 1) / per);
        const unsigned blocks = float_blocks + p.cache_blocks;
        p.cache_begin = blocks > 8u * p.sms ? 0 : float_blocks;
        const cudaError_t e =
            launch_dependent(cached ? head_rows_kernel<T, VEC, FULL, INTER, true, LANES, U>
                                    : head_rows_kernel<T, VEC, FULL, INTER, false, LANES, U>, blocks, kThreads, 0, stream, p);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <typename T, bool VEC, bool INTER, int U, int LANES>
cudaError_t rows_full(const RowsParams &p, cudaStream_t stream) {
    if constexpr (U > 1) {      // for a few heads it makes no difference
        if (p.D == 8 * LANES) return rows_launch<T, VEC, true, INTER, LANES, U>(p, stream);
    }
    return rows_launch<T, VEC, false, INTER, LANES, U>(p, stream);
}

template <typename T, bool VEC, bool INTER, int U>
cudaError_t rows_lanes(const RowsParams &p, cudaStream_t stream) {
    if (p.D <= 64) return rows_full<T, VEC, INTER, U, 8>(p, stream);
    if (p.D <= 128) return rows_full<T, VEC, INTER, U, 16>(p, stream);
    return rows_full<T, VEC, INTER, U, 32>(p, stream);
}

template <typename T, bool INTER>
cudaError_t rows_type(const RowsParams &p, cudaStream_t stream) {
    constexpr int es = sizeof(T), bytes = 4 * es;
    const bool vec = p.pairs % 4 == 0 && aligned(p.q, es, bytes) && aligned(p.k, es, bytes) && aligned(p.v, es, bytes) &&
                     aligned(p.q_out, es, bytes) && aligned(p.k_out, es, bytes) && aligned(p.cos, 16) &&
                     aligned(p.sin, 16) && p.ldt % 4 == 0 && aligned(p.qw, 16) && aligned(p.kw, 16);
    if (!vec) return rows_lanes<T, false, INTER, 1>(p, stream);
    // Several heads to a group once there are lanes for half of every SM: a token's angles
    // are then loaded once for them, and four loads of a lane are under way together
    // (tokens of 32 + 8 heads of 128 in bf16: 128 tokens 2.3 us against 2.0 with single heads,
    // 256 2.5 and 2.7, 1024 4.7 and 6.9, 4096 17.7 and 26.7).
    const int lanes = p.D <= 64 ? 8 : p.D <= 128 ? 16 : 32;
    if (p.T * (p.q.n + p.k.n + p.v.n) * lanes <= (int64_t)p.sms * 1024) return rows_lanes<T, true, INTER, 1>(p, stream);
    return rows_lanes<T, true, INTER, 8 / es>(p, stream);
}

template <typename T>
cudaError_t rows_of(const RowsParams &p, cudaStream_t stream) {
    return p.interleaved && p.pairs > 0 ? rows_type<T, true>(p, stream) : rows_type<T, false>(p, stream);
}

template <typename T, bool VEC, int LANES, int IT, int U>
cudaError_t read_launch(ReadParams p, cudaStream_t stream) {
    const int per_kind = ((int)p.cache.heads + U - 1) / U;
    p.k_units = p.k_out.n > 0 ? per_kind : 0;
    p.units = p.k_units + (p.v_out.n > 0 ? per_kind : 0);
    const int64_t step = kMostUnits / p.units / 16 * 16;
    for (int64_t t = 0; t < p.N; t += step) {
        const int64_t n = p.N - t < step ? p.N - t : step;
        p.first = t;
        p.count = (n + 15) / 16 * 16 * p.units;
        const int64_t per = kThreads / LANES;
        const cudaError_t e = launch_dependent(cache_read_kernel<T, VEC, LANES, IT, U>, (unsigned)((p.count + per - 1) / per),
                                               kThreads, 0, stream, p);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <typename T, bool VEC>
cudaError_t read_lanes(const ReadParams &p, cudaStream_t stream) {
    const int chunks = p.D * (int)sizeof(T) / 16;
    if (chunks <= 8) return read_launch<T, VEC, 4, 2, 2>(p, stream);
    if (chunks <= 16) return read_launch<T, VEC, 8, 2, 2>(p, stream);
    if (chunks <= 32) return read_launch<T, VEC, 16, 2, 2>(p, stream);
    return read_launch<T, VEC, 32, 2, 2>(p, stream);
}

template <typename T>
cudaError_t read_type(const ReadParams &p, cudaStream_t stream) {
    const bool vec = aligned(p.k_out, sizeof(T), 16) && aligned(p.v_out, sizeof(T), 16);
    return vec ? read_lanes<T, true>(p, stream) : read_lanes<T, false>(p, stream);
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
    p.over_dim = 1.0f / (float)a.D;
    p.least = a.eps < kTwoM100 ? kTwoM100 * (float)a.D : 0.0f;      // see norm_lift
    p.cos = a.rotary.cos; p.sin = a.rotary.sin;
    p.rows = a.rotary.rows; p.ldt = a.rotary.ld; p.positions = a.rotary.positions;
    p.slots = a.slots; p.cache = a.cache;
    p.sms = a.sm_count;
    p.err = a.err;
    return a.type == kTypeBf16 ? rows_of<__nv_bfloat16>(p, a.stream)
                               : rows_of<float>(p, a.stream);
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
