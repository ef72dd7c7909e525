// attend.cuh -- attention of one new token per sequence over the 8-bit paged
// cache, as a template over the heads' size (instantiated in attend_*.cu).
//
//     s_t = scale * q . k_t        p_t = 2^(s_t*log2(e) - m)        m: about the largest so far
//     out = sum_t p_t v_t / sum_t p_t
//
// One pass over the cache.  Keys and values are whole numbers times a scale per
// row, exact in FP16; the keys' scale multiplies the score, the values' the
// probability, so that both products are FP16 MMAs of whole numbers with FP32
// sums.  A warp takes strips of 16 tokens:
//
//     S^T (tokens x heads) = K (16 x D) . Q^T (D x 8)      K's rows are the MMA's A as they lie
//     O^T (dims x heads) += V^T (D x 16) . P^T (16 x 8)    A: bytes of two tokens paired
//
// up to 8 heads that share a key head as the MMA's 8 columns (NT of those).  The
// order of an MMA's inner index is free as long as A and B agree, so every lane
// reads 16 consecutive bytes of a row.  S^T comes out as P^T goes in except for a
// transposition of 8 x 8, one instruction (movmatrix).
//
// Strips travel through shared memory with cp.async, a ring for each warp, so that
// no barrier stands between a warp and its data.  The work of all sequences is
// one list of rounds (a strip for each of the block's warps), divided evenly over
// the blocks from the lengths as they are on the device: ragged batches balance,
// and one long sequence spreads over every SM.  A sequence's head that several
// blocks share is joined by the last of them to finish, in a fixed order.
#pragma once

#include "cache.cuh"

namespace sgemm_gb300 {

constexpr int kAttendWarps = 4;
constexpr int kStrip = 16;                 // tokens
constexpr int kJoin = 16;                  // parts joined at a time

struct AttendParams {
    int B, Hk, G, D, groups;               // groups: of 8*NT query heads to a key head
    int page, width;
    uint32_t page_mul, page_shift;         // t / page = (t * page_mul) >> page_shift (host: divider())
    int whole;                             // a strip lies within a page
    int window;
    float scale_log2;                      // scale * log2(e)
    const void *q; int64_t q_ld, q_hs;
    void *out; int64_t o_ld, o_hs;
    int q_vec, o_vec;                      // 16-byte accesses
    const int8_t *k, *v;
    const float *ks, *vs;
    int64_t k_stride, v_stride, ks_stride, vs_stride;
    int64_t blocks;
    const int32_t *table; int64_t ld_table;
    const int32_t *lens;
    float *lse;
    float *parts;                          // 2 * gridDim.x parts
    unsigned *tickets;                     // 2 * gridDim.x for parts, gridDim.x for groups of parts
    unsigned *err;
};

cudaError_t launch_attend_64(const AttendParams &p, int type, int nt, int sms, cudaStream_t stream);
cudaError_t launch_attend_128(const AttendParams &p, int type, int nt, int sms, cudaStream_t stream);
cudaError_t launch_attend_256(const AttendParams &p, int type, int nt, int sms, cudaStream_t stream);
// Blocks on an SM, which the workspace is sized by.
constexpr int attend_blocks(int dt, int nt) { return dt == 64 ? 4 : dt == 128 ? (nt == 1 ? 4 : 3) : 2; }
// Floats of one part: sums of 8*nt heads, then each head's m and sum of p.
constexpr int attend_part(int dt, int nt) { return 8 * nt * (dt + 2); }

#ifdef __CUDACC__

namespace {

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ uint4 lds16(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t lds4(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Lane l's pair of row l/4 becomes the pair of column l/4.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ float exp2_fast(float x) {      // 2 units in the last place; 0 below 2^-126
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t half_pair(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
// What half_pair leaves of the two.
__device__ __forceinline__ uint32_t half_pair_rest(float lo, float hi, uint32_t taken) {
    const float2 t = __half22float2(*reinterpret_cast<const __half2 *>(&taken));
    return half_pair(lo - t.x, hi - t.y);
}

// Words of four bytes of two tokens as FP16 pairs (token a, token b), one for each
// byte: the expansion of q8_to_f16 on interleaved bytes.
__device__ __forceinline__ void pair_tokens(uint32_t a, uint32_t b, uint32_t (&r)[4]) {
    const uint32_t ua = a ^ 0x80808080u, ub = b ^ 0x80808080u;
    const uint32_t lo = __byte_perm(ua, ub, 0x5140), hi = __byte_perm(ua, ub, 0x7362);
    const __half2 bias = __half2half2(__ushort_as_half((unsigned short)0x6480));   // 1152
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t x = __byte_perm(i < 2 ? lo : hi, 0x64646464u, (i & 1) ? 0x4342 : 0x4140);
        const __half2 h = __hsub2(*reinterpret_cast<const __half2 *>(&x), bias);
        r[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
}

// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
// e with 2^e <= v < 2^(e+1) for a finite v >= 2^-118; -118 below, 128 beyond.
__device__ __forceinline__ int exponent(float v) { return max(-118, (int)((__float_as_uint(v) >> 23) & 0xff) - 127); }

template <int DT, int NT, int TERMS>
struct Shape {
    static constexpr int CH = DT / 16;                 // 16-byte chunks of a row
    static constexpr int STEPS = DT / 16;              // MMAs along the head, and dim tiles of O^T
    static constexpr int ROWS = kStrip * DT;           // bytes of a strip's keys
    static constexpr int STAGE = 2 * ROWS + 256;       // keys, values, 16 + 16 scales, the mask
    static constexpr int HEADS = 8 * NT;
    static constexpr int BLOCKS = attend_blocks(DT, NT);
    // merge: every warp's sums of DM dims of all heads, padded against bank conflicts
    static constexpr int DM = (DT * NT > 128) ? 128 / NT : DT;
    static constexpr int MERGE = kAttendWarps * HEADS * (DM + 4) * 4;
    // the queries' operands: in registers as long as they take at most 32
    static constexpr bool Q_SHARED = NT * TERMS * STEPS * 2 > 32;
    static constexpr int QUERIES = Q_SHARED ? NT * TERMS * STEPS * 256 : 0;
    static constexpr int FIXED = MERGE + kAttendWarps * HEADS * 8 + 64 + QUERIES;
    static constexpr int ROOM = (227 * 1024) / BLOCKS - 1024 - 128 - FIXED;
    static constexpr int MOST = ROOM / (kAttendWarps * STAGE);
    static constexpr int STAGES = MOST > 6 ? 6 : MOST;
    static constexpr int SMEM = kAttendWarps * STAGES * STAGE + FIXED + 128;
    static_assert(STAGES >= 2, "a ring has two strips at least");
};

// Byte offset of chunk c of row r in a strip, chunks exchanged within 128 bytes so
// that neither the keys' reads (8 lanes: 2 rows, 4 chunks of each) nor the values'
// (8 lanes: 4 rows, 2 chunks) meet in a bank.
template <int DT>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
    if constexpr (DT == 64) return (uint32_t)((r >> 1) * 128 + ((((r & 1) * 4 + c) ^ (r & 6)) << 4));
    else return (uint32_t)(r * DT + (c >> 3) * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// 16 values of a query head from element d on, zeros past the head's end.
template <typename T>
__device__ __forceinline__ void load_q16(const T *q, int d, int D, bool vec, float (&x)[16]) {
    if (q == nullptr || d >= D) {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = 0.0f;
    } else if (vec) {
        constexpr int V = 16 / (int)sizeof(T);
#pragma unroll
        for (int i = 0; i < 16 / V; ++i) {
            float part[V];
            load_vec<T, V>(q + d + V * i, part);
#pragma unroll
            for (int e = 0; e < V; ++e) x[V * i + e] = part[e];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = to_f32<T>(q[d + i]);
    }
}

// The strips of a sequence that its new token attends to.
struct Span {
    int first, last;       // tokens [first, last)
    int strip0, strips;    // strips of 16 from token 16*strip0 on
    __device__ __forceinline__ int rounds() const { return (strips + kAttendWarps - 1) / kAttendWarps; }
};

__device__ __forceinline__ Span span_of(const AttendParams &p, int b) {
    const int most = p.width * p.page;
    int n = __ldg(p.lens + b);
    n = n < 0 ? 0 : n > most ? most : n;
    Span s;
    s.last = n;
    s.first = p.window > 0 && n > p.window ? n - p.window : 0;
    s.strip0 = s.first / kStrip;
    s.strips = n > 0 ? (n + kStrip - 1) / kStrip - s.strip0 : 0;
    return s;
}

// A place in the list of rounds: sequence, key head and group of query heads, round.
struct Cursor {
    int b, item, round;
    Span span;
    __device__ __forceinline__ void step(const AttendParams &p) {
        if (++round < span.rounds()) return;
        round = 0;
        if (++item < p.Hk * p.groups) return;
        item = 0;
        do {
            if (++b >= p.B) { b = p.B - 1; return; }    // past the end: nothing follows
            span = span_of(p, b);
        } while (span.strips == 0);
    }
};

// The first round of block c among `blocks`.
__device__ __forceinline__ int64_t block_start(int64_t total, int c, int blocks) { return total * c / blocks; }

template <int DT, int NT, typename T>
struct Attend {
    static constexpr bool SPLIT = sizeof(T) == 4;      // FP32: operands in two FP16 terms
    static constexpr int TERMS = SPLIT ? 2 : 1;
    using S = Shape<DT, NT, TERMS>;

    const AttendParams &p;
    uint32_t ring;          // this warp's stages
    uint32_t queries;       // Q_SHARED: the block's
    int warp, lane, g, j;

    // the strip to be loaded next: its page number is on its way
    Cursor next;
    int64_t left;           // rounds not yet loaded
    int next_page;
    bool next_on;

    __device__ __forceinline__ Attend(const AttendParams &pp, uint32_t smem, uint32_t q) : p(pp), queries(q) {
        warp = threadIdx.x >> 5;
        lane = threadIdx.x & 31;
        g = lane >> 2;
        j = lane & 3;
        ring = smem + warp * (S::STAGES * S::STAGE);
    }

    __device__ __forceinline__ int page_of(int t) const {
        return (int)(((uint64_t)(uint32_t)t * p.page_mul) >> p.page_shift);
    }

    // Asks for the page number of the strip at `next` (of this lane's token of it
    // where a strip may reach over several pages).
    __device__ __forceinline__ void look_up() {
        const int strip = next.round * kAttendWarps + warp;
        next_on = left > 0 && strip < next.span.strips;
        next_page = -1;
        if (next_on) {
            int t = (next.span.strip0 + strip) * kStrip;
            if (!p.whole) t = max(min(t + (lane & 15), next.span.last - 1), next.span.first);
            next_page = __ldg(p.table + next.b * p.ld_table + page_of(t));
        }
    }

    // Starts the copies of the strip at `next` into stage s, and moves on.
    __device__ __forceinline__ void load(int s) {
        if (next_on) {
            const uint32_t at = ring + s * S::STAGE;
            const int h = next.item / p.groups;
            const int t0 = (next.span.strip0 + next.round * kAttendWarps + warp) * kStrip;
            const int t = t0 + (lane & 15);
            const bool known = next_page >= 0 && next_page < p.blocks;
            if (!known && lane < 16) record_error(p.err, kErrBadIndex);
            const bool fine = known && t >= next.span.first && t < next.span.last;
            const uint32_t mask = __ballot_sync(0xffffffffu, fine) & 0xffffu;
            const int chunks = p.D >> 4;
            const int64_t page = next_page;
            if (p.whole) {
                if (known) {
                    const int64_t row = (int64_t)h * p.page + (t0 - page_of(t0) * p.page);
                    const int8_t *k = p.k + page * p.k_stride + row * p.D;
                    const int8_t *v = p.v + page * p.v_stride + row * p.D;
#pragma unroll
                    for (int i = 0; i < S::CH / 2; ++i) {
                        const int q = lane + 32 * i, r = q / S::CH, c = q % S::CH;
                        if (c < chunks) {
                            cp_async16(at + chunk_at<DT>(r, c), k + r * p.D + c * 16);
                            cp_async16(at + S::ROWS + chunk_at<DT>(r, c), v + r * p.D + c * 16);
                        }
                    }
                    const float *scale = lane < 16 ? p.ks + page * p.ks_stride : p.vs + page * p.vs_stride;
                    cp_async4(at + 2 * S::ROWS + 4 * lane, scale + row + (lane & 15));
                }
            } else {
                const int row = h * p.page + (t - page_of(t) * p.page);    // of this lane's token
#pragma unroll
                for (int i = 0; i < S::CH / 2; ++i) {
                    const int q = lane + 32 * i, r = q / S::CH, c = q % S::CH;
                    const int64_t rp = __shfl_sync(0xffffffffu, next_page, r);
                    const int64_t rr = __shfl_sync(0xffffffffu, row, r);
                    if (c < chunks && (mask >> r & 1)) {
                        cp_async16(at + chunk_at<DT>(r, c), p.k + rp * p.k_stride + rr * p.D + c * 16);
                        cp_async16(at + S::ROWS + chunk_at<DT>(r, c), p.v + rp * p.v_stride + rr * p.D + c * 16);
                    }
                }
                if (fine) {
                    const float *scale = lane < 16 ? p.ks + page * p.ks_stride : p.vs + page * p.vs_stride;
                    cp_async4(at + 2 * S::ROWS + 4 * lane, scale + row);
                }
            }
            if (lane == 0) asm volatile("st.shared.u32 [%0], %1;" ::"r"(at + 2 * S::ROWS + 128), "r"(mask) : "memory");
        }
        cp_commit();
        if (left > 0 && --left > 0) next.step(p);
        look_up();
    }

    // ---- one key head's running state -------------------------------------------------
    uint32_t qf[S::Q_SHARED ? 1 : NT][TERMS][S::STEPS][2];
    float qmul[NT][2];                  // turns a product into a score in base 2, without the key's scale
    float m[NT][2], sum[NT][2];         // of heads 2j and 2j + 1; sum: of this lane's tokens
    float vmul, vcap;                   // a power of two that the probabilities carry; the largest scale it is for
    float acc[S::STEPS][NT][4];

    // Queries of group `item` of sequence b as the MMA's B, scaled by a power of two
    // into FP16's range (below 2^15, so a BF16 query is exact).
    __device__ __forceinline__ void begin(int b, int item) {
        const int h = item / p.groups, first = (item % p.groups) * S::HEADS;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int head = first + nt * 8 + g;
            const T *q = head < p.G ? static_cast<const T *>(p.q) + b * p.q_ld + (h * (int64_t)p.G + head) * p.q_hs : nullptr;
            float x[S::CH / 4][16];
            float most = 0.0f;
#pragma unroll
            for (int i = 0; i < S::CH / 4; ++i) {
                load_q16<T>(q, key_chunk(i) * 16, p.D, p.q_vec != 0, x[i]);
#pragma unroll
                for (int e = 0; e < 16; ++e) most = fmaxf(most, fabsf(x[i][e]));
            }
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
            const int e = min(exponent(most), 127);
            const float up = pow2(min(14 - e, 127));
            const float mul = p.scale_log2 / up;
#pragma unroll
            for (int i = 0; i < S::CH / 4; ++i)
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const float a = x[i][4 * w] * up, bb = x[i][4 * w + 1] * up, c = x[i][4 * w + 2] * up,
                                d = x[i][4 * w + 3] * up;
                    const uint32_t lo = half_pair(a, bb), hi = half_pair(c, d);
                    put_query(nt, 0, 4 * i + w, lo, hi);
                    if constexpr (SPLIT) put_query(nt, 1, 4 * i + w, half_pair_rest(a, bb, lo), half_pair_rest(c, d, hi));
                }
            qmul[nt][0] = __shfl_sync(0xffffffffu, mul, 8 * j);
            qmul[nt][1] = __shfl_sync(0xffffffffu, mul, 8 * j + 4);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                m[nt][k] = -1e30f;
                sum[nt][k] = 0.0f;
            }
#pragma unroll
            for (int i = 0; i < S::STEPS; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[i][nt][k] = 0.0f;
        }
        vmul = 1.0f;
        vcap = -1.0f;
        if constexpr (S::Q_SHARED) __syncthreads();
    }

    // Where they are shared, every warp has computed them and stores a part.
    __device__ __forceinline__ void put_query(int nt, int term, int step, uint32_t lo, uint32_t hi) {
        if constexpr (S::Q_SHARED) {
            if (step % kAttendWarps == warp)
                asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(queries + ((nt * TERMS + term) * S::STEPS + step) * 256 + 8 * lane),
                             "r"(lo), "r"(hi)
                             : "memory");
        } else {
            qf[nt][term][step][0] = lo;
            qf[nt][term][step][1] = hi;
        }
    }
    __device__ __forceinline__ uint2 query(int nt, int term, int step) const {
        if constexpr (S::Q_SHARED) return lds8(queries + ((nt * TERMS + term) * S::STEPS + step) * 256 + 8 * lane);
        else return make_uint2(qf[nt][term][step][0], qf[nt][term][step][1]);
    }

    // The i-th chunk of a key row that this lane reads.
    __device__ __forceinline__ int key_chunk(int i) const {
        if constexpr (DT == 64) return j;
        else return (i >> 1) * 8 + 2 * j + (i & 1);
    }

    __device__ __forceinline__ void consume(int s) {
        const uint32_t at = ring + s * S::STAGE;
        const uint32_t mask = lds4(at + 2 * S::ROWS + 128);
        float sc[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 4; ++k) sc[nt][k] = 0.0f;
#pragma unroll
        for (int i = 0; i < S::CH / 4; ++i) {
            const int c = key_chunk(i);
            const uint4 lo = lds16(at + chunk_at<DT>(g, c)), hi = lds16(at + chunk_at<DT>(g + 8, c));
            const uint32_t wl[4] = {lo.x, lo.y, lo.z, lo.w}, wh[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                uint32_t a0, a1, a2, a3;
                q8_to_f16(wl[w], a0, a2);
                q8_to_f16(wh[w], a1, a3);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int t = 0; t < TERMS; ++t) {
                        const uint2 q = query(nt, t, 4 * i + w);
                        mma_f16(sc[nt], a0, a1, a2, a3, q.x, q.y);
                    }
            }
        }
        const uint32_t scales = at + 2 * S::ROWS;
        const float k0 = __uint_as_float(lds4(scales + 4 * g)), k1 = __uint_as_float(lds4(scales + 4 * g + 32));
        float v0 = __uint_as_float(lds4(scales + 64 + 4 * g)), v1 = __uint_as_float(lds4(scales + 64 + 4 * g + 32));
        bool grown = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            sc[nt][0] *= k0 * qmul[nt][0];
            sc[nt][1] *= k0 * qmul[nt][1];
            sc[nt][2] *= k1 * qmul[nt][0];
            sc[nt][3] *= k1 * qmul[nt][1];
        }
        if (mask != 0xffffu) {      // the same for the whole warp
            const bool on0 = mask >> g & 1, on1 = mask >> (g + 8) & 1;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                if (!on0) sc[nt][0] = sc[nt][1] = -INFINITY;
                if (!on1) sc[nt][2] = sc[nt][3] = -INFINITY;
            }
            if (!on0) v0 = 0.0f;
            if (!on1) v1 = 0.0f;
        }
        // The scaling by m and vmul is kept until a score passes m + 5 or a value's
        // scale vcap: probabilities stay below 2^5 and their products with the scales,
        // which vmul takes to [2^8, 2^10], below 2^15, in FP16's range.  FP16 rounds
        // such a product to 11 bits, or to 2^-24 where it is below 2^-14: 2^-33 of the
        // largest scale (p = 1), a token.
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            grown |= fmaxf(sc[nt][0], sc[nt][2]) > m[nt][0] + 5.0f || fmaxf(sc[nt][1], sc[nt][3]) > m[nt][1] + 5.0f;
        const float vm = fmaxf(fabsf(v0), fabsf(v1));
        grown |= vm > vcap;
        if (__any_sync(0xffffffffu, grown)) rescale(sc, vm);
        const float u0 = v0 * vmul, u1 = v1 * vmul;
        uint32_t pf[NT][TERMS][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const float p0 = exp2_fast(sc[nt][0] - m[nt][0]), p1 = exp2_fast(sc[nt][1] - m[nt][1]);
            const float p2 = exp2_fast(sc[nt][2] - m[nt][0]), p3 = exp2_fast(sc[nt][3] - m[nt][1]);
            sum[nt][0] += p0 + p2;
            sum[nt][1] += p1 + p3;
            const float x0 = p0 * u0, x1 = p1 * u0, x2 = p2 * u1, x3 = p3 * u1;
            const uint32_t a = half_pair(x0, x1), b = half_pair(x2, x3);
            pf[nt][0][0] = transpose8(a);
            pf[nt][0][1] = transpose8(b);
            if constexpr (SPLIT) {
                pf[nt][1][0] = transpose8(half_pair_rest(x0, x1, a));
                pf[nt][1][1] = transpose8(half_pair_rest(x2, x3, b));
            }
        }
        const uint32_t vals = at + S::ROWS;
        if constexpr (DT == 64) {
            // 8 dims a lane: half a chunk of each of its four tokens
            uint2 r[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) r[k] = lds8(vals + chunk_at<DT>(2 * j + (k & 1) + (k >> 1) * 8, g >> 1) + (g & 1) * 8);
            values(0, r[0].x, r[1].x, r[2].x, r[3].x, pf);
            values(1, r[0].y, r[1].y, r[2].y, r[3].y, pf);
        } else {
#pragma unroll
            for (int i = 0; i < S::CH / 8; ++i) {
                uint4 r[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) r[k] = lds16(vals + chunk_at<DT>(2 * j + (k & 1) + (k >> 1) * 8, g + 8 * i));
                values(4 * i, r[0].x, r[1].x, r[2].x, r[3].x, pf);
                values(4 * i + 1, r[0].y, r[1].y, r[2].y, r[3].y, pf);
                values(4 * i + 2, r[0].z, r[1].z, r[2].z, r[3].z, pf);
                values(4 * i + 3, r[0].w, r[1].w, r[2].w, r[3].w, pf);
            }
        }
    }

    // Word `word` of this lane's dims (four of them, of tokens 2j, 2j+1, 2j+8, 2j+9):
    // two dim tiles of O^T.
    __device__ __forceinline__ void values(int word, uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3,
                                           const uint32_t (&pf)[NT][TERMS][2]) {
        uint32_t lo[4], hi[4];
        pair_tokens(w0, w1, lo);
        pair_tokens(w2, w3, hi);
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int t = 0; t < TERMS; ++t)
                    mma_f16(acc[2 * word + half][nt], lo[2 * half], lo[2 * half + 1], hi[2 * half], hi[2 * half + 1],
                            pf[nt][t][0], pf[nt][t][1]);
    }

    __device__ __forceinline__ void rescale(const float (&sc)[NT][4], float vm) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) vm = fmaxf(vm, __shfl_xor_sync(0xffffffffu, vm, o));
        float f = 1.0f;
        if (vm > vcap) {
            const int e = min(exponent(vm), 127);
            const float to = pow2(8 - e);
            f = vcap < 0.0f ? 1.0f : to / vmul;
            vmul = to;
            vcap = e < 126 ? pow2(e + 2) : INFINITY;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float x = fmaxf(sc[nt][k], sc[nt][k + 2]);
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
                const float to = fmaxf(x, m[nt][k]);
                const float d = exp2_fast(m[nt][k] - to);
                m[nt][k] = to;
                sum[nt][k] *= d;
#pragma unroll
                for (int i = 0; i < S::STEPS; ++i) {
                    acc[i][nt][k] *= d * f;
                    acc[i][nt][k + 2] *= d * f;
                }
            }
    }

    // The dim of acc[i][.][0 or 1]; [2 or 3] is the next one.
    __device__ __forceinline__ int dim_of(int i) const {
        const int word = i >> 1, base = DT == 64 ? 8 * g : 16 * (g + 8 * (word >> 2));
        return base + 4 * (DT == 64 ? word : word & 3) + 2 * (i & 1);
    }
};

// Four dims of a head's result; with d == 0 its lse too.
template <int DT, int NT, typename T>
__device__ __forceinline__ void finish(const AttendParams &p, int b, int h, int head, int d, float4 o, float top, float total) {
    if (head >= p.G || d >= p.D) return;
    const float inv = total != 0.0f ? 1.0f / total : 0.0f;
    const float v[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
    T *to = static_cast<T *>(p.out) + b * p.o_ld + ((int64_t)h * p.G + head) * p.o_hs + d;
    if (p.o_vec) {
        store_vec<T, 4>(to, v);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) to[i] = from_f32<T>(v[i]);
    }
    if (d == 0 && p.lse)
        p.lse[((int64_t)b * p.Hk + h) * p.G + head] = total != 0.0f ? (top + log2f(total)) * 0.69314718055994531f : -INFINITY;
}

// Counts this block in at a ticket; true in all its threads if it is the last of n.
__device__ __forceinline__ bool last_of(unsigned *ticket, int n, int *note) {
    __syncthreads();            // all parts of this block are written
    if (threadIdx.x == 0) {
        __threadfence();
        const bool last = atomicAdd(ticket, 1u) == (unsigned)(n - 1);
        if (last) *ticket = 0;
        __threadfence();
        note[0] = last;
    }
    __syncthreads();
    return note[0] != 0;
}

// Sums n parts (part i at where(i)) for four dims of a head.
template <int DT, int NT, typename Where>
__device__ __forceinline__ void sum_parts(int n, Where where, int head, int d, float4 &o, float &top, float &total) {
    top = -1e30f;
    for (int i = 0; i < n; ++i)
        top = fmaxf(top, __ldcg(reinterpret_cast<const float2 *>(where(i) + 8 * NT * DT + 2 * head)).x);
    o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    total = 0.0f;
    for (int i = 0; i < n; ++i) {
        const float2 y = __ldcg(reinterpret_cast<const float2 *>(where(i) + 8 * NT * DT + 2 * head));
        const float4 x = __ldcg(reinterpret_cast<const float4 *>(where(i) + head * DT + d));
        const float f = exp2_fast(y.x - top);
        total += y.y * f;
        o.x += x.x * f; o.y += x.y * f; o.z += x.z * f; o.w += x.w * f;
    }
}

// Joins the parts of one key head that blocks c0 to c1 have written: the last of
// each kJoin blocks sums their parts into the first one's place, the last of
// those sums the sums.
template <int DT, int NT, typename T>
__device__ __forceinline__ void join(const AttendParams &p, int b, int h, int head0, int c0, int c1, bool is_first, int *note) {
    constexpr int PART = attend_part(DT, NT), HEADS = 8 * NT;
    const int n = c1 - c0 + 1, group = (int)(blockIdx.x - c0) / kJoin, groups = (n + kJoin - 1) / kJoin;
    auto where = [&](int i) { return p.parts + (int64_t)(2 * (c0 + i) + (i == 0 ? 1 : 0)) * PART; };
    const int g0 = group * kJoin, gn = min(kJoin, n - g0);
    if (!last_of(p.tickets + 2 * (c0 + g0) + (g0 == 0 ? 1 : 0), gn, note)) return;
    float4 o[(HEADS * DT / 4 + kAttendWarps * 32 - 1) / (kAttendWarps * 32)];
    if (groups > 1) {
        // read everything before the first part is written over
        float2 y[sizeof(o) / sizeof(o[0])];
#pragma unroll
        for (int k = 0; k < (int)(sizeof(o) / sizeof(o[0])); ++k) {
            const int i = threadIdx.x + k * kAttendWarps * 32, head = i / (DT / 4), d = (i % (DT / 4)) * 4;
            sum_parts<DT, NT>(gn, [&](int q) { return where(g0 + q); }, head, d, o[k], y[k].x, y[k].y);
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < (int)(sizeof(o) / sizeof(o[0])); ++k) {
            const int i = threadIdx.x + k * kAttendWarps * 32, head = i / (DT / 4), d = (i % (DT / 4)) * 4;
            *reinterpret_cast<float4 *>(where(g0) + head * DT + d) = o[k];
            if (d == 0) *reinterpret_cast<float2 *>(where(g0) + HEADS * DT + 2 * head) = y[k];
        }
        if (!last_of(p.tickets + 2 * gridDim.x + c0, groups, note)) return;
    }
    for (int i = threadIdx.x; i < HEADS * (DT / 4); i += kAttendWarps * 32) {
        const int head = i / (DT / 4), d = (i % (DT / 4)) * 4;
        float4 x;
        float top, total;
        if (groups > 1) sum_parts<DT, NT>(groups, [&](int q) { return where(q * kJoin); }, head, d, x, top, total);
        else sum_parts<DT, NT>(n, where, head, d, x, top, total);
        finish<DT, NT, T>(p, b, h, head0 + head, d, x, top, total);
    }
}

template <int DT, int NT, typename T>
__global__ void __launch_bounds__(kAttendWarps * 32, attend_blocks(DT, NT))
attend_kernel(const __grid_constant__ AttendParams p) {
    using S = typename Attend<DT, NT, T>::S;
    extern __shared__ uint8_t raw[];
    uint8_t *smem = raw + ((128 - (smem_u32(raw) & 127)) & 127);
    float *merge = reinterpret_cast<float *>(smem + kAttendWarps * S::STAGES * S::STAGE);
    float2 *ml = reinterpret_cast<float2 *>(merge + S::MERGE / 4);      // [warp][head]: m, sum of p
    int *note = reinterpret_cast<int *>(ml + kAttendWarps * S::HEADS);
    uint32_t *queries = reinterpret_cast<uint32_t *>(note + 16);
    const int tid = threadIdx.x;
    const int items = p.Hk * p.groups;

    // Rounds of all sequences, and where this block's begin.  A thread counts `per`
    // consecutive sequences.
    Cursor start{};
    int64_t total, mine, r0;
    int blocks;
    {
        int64_t *sums = reinterpret_cast<int64_t *>(merge);             // one per thread, then the warps'
        const int per = (p.B + kAttendWarps * 32 - 1) / (kAttendWarps * 32);
        const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
        int64_t count = 0;
        for (int b = b0; b < b1; ++b) {
            const Span s = span_of(p, b);
            count += s.rounds();
            if (blockIdx.x == 0) {
                const int n = p.lens[b];
                if (n < 0 || n > p.width * p.page) record_error(p.err, kErrBadIndex);
            }
        }
        count *= items;
        int64_t before = count;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, before, o);
            if ((tid & 31) >= o) before += x;
        }
        if ((tid & 31) == 31) sums[tid >> 5] = before;
        __syncthreads();
        before -= count;
        total = 0;
#pragma unroll
        for (int w = 0; w < kAttendWarps; ++w) {
            if (w < (tid >> 5)) before += sums[w];
            total += sums[w];
        }
        blocks = (int)(total < (int64_t)gridDim.x ? (total > 0 ? total : 1) : gridDim.x);
        r0 = (int)blockIdx.x < blocks ? block_start(total, blockIdx.x, blocks) : total;
        mine = (int)blockIdx.x < blocks ? block_start(total, blockIdx.x + 1, blocks) - r0 : 0;
        if (mine > 0 && r0 >= before && r0 < before + count) {
            int64_t off = r0 - before;
            int b = b0;
            int64_t n = (int64_t)span_of(p, b).rounds() * items;
            while (off >= n) {
                off -= n;
                n = (int64_t)span_of(p, ++b).rounds() * items;
            }
            const int rounds = (int)(n / items);
            note[0] = b;
            note[1] = (int)(off / rounds);
            note[2] = (int)(off % rounds);
        }
        // rows of sequences without tokens
        for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
            if (span_of(p, b).strips > 0) continue;
            for (int i = tid; i < p.Hk * p.G * p.D; i += blockDim.x)
                static_cast<T *>(p.out)[b * p.o_ld + (i / p.D) * p.o_hs + i % p.D] = from_f32<T>(0.0f);
            if (p.lse)
                for (int i = tid; i < p.Hk * p.G; i += blockDim.x) p.lse[(int64_t)b * p.Hk * p.G + i] = -INFINITY;
        }
        __syncthreads();
        if (mine == 0) return;
        start.b = note[0];
        start.item = note[1];
        start.round = note[2];
        start.span = span_of(p, start.b);
    }

    Attend<DT, NT, T> a(p, smem_u32(smem), smem_u32(queries));
    if (p.D < DT) {     // chunks past the head's end are never written: zeros in the products
        uint4 *z = reinterpret_cast<uint4 *>(smem + a.warp * (S::STAGES * S::STAGE));
        for (int i = a.lane; i < S::STAGES * S::STAGE / 16; i += 32) z[i] = make_uint4(0, 0, 0, 0);
        __syncwarp();
    }
    a.next = start;
    a.left = mine;
    a.look_up();
#pragma unroll
    for (int s = 0; s < S::STAGES - 1; ++s) a.load(s);

    Cursor cur = start;
    int stage = 0, fill = S::STAGES - 1;
    int64_t todo = mine, at_round = r0;
    while (todo > 0) {
        // one piece: the rounds of one sequence's key head that are this block's
        const int rounds = cur.span.rounds();
        const int n = (int)(todo < rounds - cur.round ? todo : rounds - cur.round);
        a.begin(cur.b, cur.item);
        for (int i = 0; i < n; ++i) {
            cp_wait<S::STAGES - 2>();
            __syncwarp();       // every lane's copies have landed, and the stage filled next has been read
            a.load(fill);
            if ((cur.round + i) * kAttendWarps + a.warp < cur.span.strips) a.consume(stage);
            stage = stage + 1 == S::STAGES ? 0 : stage + 1;
            fill = fill + 1 == S::STAGES ? 0 : fill + 1;
        }

        // the warps' results together
        const int64_t item0 = at_round - cur.round;         // the key head's rounds in the list
        const bool whole = n == rounds;
        const int first_block = (int)(((item0 + 1) * blocks - 1) / total);
        const int last_block = (int)(((item0 + rounds) * blocks - 1) / total);
        const bool is_first = first_block == (int)blockIdx.x;
        float *part = p.parts + (int64_t)(2 * blockIdx.x + (is_first ? 1 : 0)) * attend_part(DT, NT);
        const int h = cur.item / p.groups, head0 = (cur.item % p.groups) * S::HEADS;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float x = a.sum[nt][k];
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
                if (a.g == 0) ml[a.warp * S::HEADS + nt * 8 + 2 * a.j + k] = make_float2(a.m[nt][k], x);
            }
        __syncthreads();
        const float unscale = 1.0f / a.vmul;
        float factor[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float top = -1e30f;
#pragma unroll
                for (int w = 0; w < kAttendWarps; ++w) top = fmaxf(top, ml[w * S::HEADS + nt * 8 + 2 * a.j + k].x);
                factor[nt][k] = exp2_fast(a.m[nt][k] - top) * unscale;
            }
        constexpr int PITCH = S::DM + 4;
#pragma unroll
        for (int d0 = 0; d0 < DT; d0 += S::DM) {
            if (d0 > 0) __syncthreads();
#pragma unroll
            for (int i = 0; i < S::STEPS; ++i) {
                const int dim = a.dim_of(i) - d0;
                if (dim < 0 || dim >= S::DM) continue;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float *to = merge + (a.warp * S::HEADS + nt * 8 + 2 * a.j + k) * PITCH + dim;
                        *reinterpret_cast<float2 *>(to) =
                            make_float2(a.acc[i][nt][k] * factor[nt][k], a.acc[i][nt][k + 2] * factor[nt][k]);
                    }
            }
            __syncthreads();
            for (int i = tid; i < S::HEADS * (S::DM / 4); i += kAttendWarps * 32) {
                const int head = i / (S::DM / 4), d = (i % (S::DM / 4)) * 4;
                float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                float top = -1e30f;
                float total_p = 0.0f;
#pragma unroll
                for (int w = 0; w < kAttendWarps; ++w) top = fmaxf(top, ml[w * S::HEADS + head].x);
#pragma unroll
                for (int w = 0; w < kAttendWarps; ++w) {
                    const float4 x = *reinterpret_cast<const float4 *>(merge + (w * S::HEADS + head) * PITCH + d);
                    o.x += x.x; o.y += x.y; o.z += x.z; o.w += x.w;
                    const float2 y = ml[w * S::HEADS + head];
                    total_p += y.y * exp2_fast(y.x - top);
                }
                if (!whole) {
                    *reinterpret_cast<float4 *>(part + head * DT + d0 + d) = o;
                    if (d0 + d == 0) *reinterpret_cast<float2 *>(part + S::HEADS * DT + 2 * head) = make_float2(top, total_p);
                } else {
                    finish<DT, NT, T>(p, cur.b, h, head0 + head, d0 + d, o, top, total_p);
                }
            }
        }
        if (!whole) join<DT, NT, T>(p, cur.b, h, head0, first_block, last_block, is_first, note);
        __syncthreads();        // ml, merge and note are free again
        at_round += n;
        todo -= n;
        if (todo > 0) {
            cur.round += n - 1;
            cur.step(p);
        }
    }
}

template <int DT, int NT, typename T>
cudaError_t attend_launch(const AttendParams &p, int sms, cudaStream_t stream) {
    using S = typename Attend<DT, NT, T>::S;
    const cudaError_t e =
        cudaFuncSetAttribute(attend_kernel<DT, NT, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
    if (e != cudaSuccess) return e;
    attend_kernel<DT, NT, T><<<sms * S::BLOCKS, kAttendWarps * 32, S::SMEM, stream>>>(p);
    return cudaGetLastError();
}

template <int DT>
cudaError_t attend_of_dim(const AttendParams &p, int type, int nt, int sms, cudaStream_t stream) {
    if (type == kTypeBf16)
        return nt == 1 ? attend_launch<DT, 1, __nv_bfloat16>(p, sms, stream) : attend_launch<DT, 2, __nv_bfloat16>(p, sms, stream);
    return nt == 1 ? attend_launch<DT, 1, float>(p, sms, stream) : attend_launch<DT, 2, float>(p, sms, stream);
}

}  // namespace

#endif  // __CUDACC__

}  // namespace sgemm_gb300
