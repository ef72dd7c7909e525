// q8_stream.cuh -- one warp's share of an 8-bit product that streams 16 weight
// rows past a few token rows (used by the linear product at few tokens and by
// the expert layer).
//
// mma.sync m16n8k16 on FP16 operands expanded from the 8-bit values in
// registers (exact, see q8_to_f16), FP32 accumulation flushed into 32-bit
// integers every 1024 k: up to there |sum| <= 1024 * 128 * 128 = 2^24, so
// every FP32 partial sum is exact.
//
// The order of k inside an MMA is free as long as both operands share it.
// Lane t of a quad therefore takes 16 consecutive bytes of its row per step of
// 64 k (one 128-bit load each of weight rows g and g + 8 and of token g), and
// word s of those bytes feeds MMA s of the step: no shared memory, no shuffles.
#pragma once

#include "q8.cuh"

namespace sgemm_gb300 {

constexpr int kQ8Step = 64;          // k per step

#ifdef __CUDACC__

constexpr int kQ8ExactSteps = 16;    // steps per exact FP32 chunk (1024 k)

// Up to 16 bytes from p, byte by byte; bytes at and past `valid` are 0.
__device__ __forceinline__ uint4 load16_bytes(const int8_t *p, int valid) {
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (i < valid) w[i >> 2] |= (uint32_t)(uint8_t)p[i] << (8 * (i & 3));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// 16 bytes from p of any alignment, all of them inside [.., end): the five
// aligned words around them, shifted together, where those lie inside
// [begin, end) as well; byte by byte at the two ends of the array.
__device__ __forceinline__ uint4 load16_unaligned(const int8_t *p, const int8_t *begin,
                                                  const int8_t *end) {
    const int8_t *a = reinterpret_cast<const int8_t *>(reinterpret_cast<uintptr_t>(p) & ~uintptr_t(3));
    if (a < begin || a + 20 > end) return load16_bytes(p, 16);
    const uint32_t *w = reinterpret_cast<const uint32_t *>(a);
    const int sh = 8 * (int)(reinterpret_cast<uintptr_t>(p) & 3);
    const uint32_t w0 = __ldg(w), w1 = __ldg(w + 1), w2 = __ldg(w + 2), w3 = __ldg(w + 3), w4 = __ldg(w + 4);
    return make_uint4(__funnelshift_r(w0, w1, sh), __funnelshift_r(w1, w2, sh),
                      __funnelshift_r(w2, w3, sh), __funnelshift_r(w3, w4, sh));
}

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Products of one step: weight rows g (wa) and g + 8 (wb), tokens x[0..NB).
template <int NB>
__device__ __forceinline__ void q8_step(float (&acc)[NB][4], const uint4 &wa, const uint4 &wb,
                                        const uint4 (&x)[NB]) {
    const uint32_t ra[4] = {wa.x, wa.y, wa.z, wa.w}, rb[4] = {wb.x, wb.y, wb.z, wb.w};
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        uint32_t a[4];
        q8_to_f16(ra[s], a[0], a[2]);
        q8_to_f16(rb[s], a[1], a[3]);
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            const uint32_t w = s == 0 ? x[n].x : s == 1 ? x[n].y : s == 2 ? x[n].z : x[n].w;
            uint32_t b0, b1;
            q8_to_f16(w, b0, b1);
            mma_f16(acc[n], a, b0, b1);
        }
    }
}

// The same for RW pairs of weight rows that share the tokens.
template <int RW, int NB>
__device__ __forceinline__ void q8_step_rows(float (&acc)[RW][NB][4], const uint4 (&wa)[RW], const uint4 (&wb)[RW],
                                             const uint4 (&x)[NB]) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        uint32_t b[NB][2];
#pragma unroll
        for (int n = 0; n < NB; ++n)
            q8_to_f16(s == 0 ? x[n].x : s == 1 ? x[n].y : s == 2 ? x[n].z : x[n].w, b[n][0], b[n][1]);
#pragma unroll
        for (int r = 0; r < RW; ++r) {
            uint32_t a[4];
            q8_to_f16(s == 0 ? wa[r].x : s == 1 ? wa[r].y : s == 2 ? wa[r].z : wa[r].w, a[0], a[2]);
            q8_to_f16(s == 0 ? wb[r].x : s == 1 ? wb[r].y : s == 2 ? wb[r].z : wb[r].w, a[1], a[3]);
#pragma unroll
            for (int n = 0; n < NB; ++n) mma_f16(acc[r][n], a, b[n][0], b[n][1]);
        }
    }
}

template <int NB>
__device__ __forceinline__ void q8_flush(int (&sum)[NB][4], float (&acc)[NB][4]) {
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            sum[n][i] += __float2int_rn(acc[n][i]);
            acc[n][i] = 0.0f;
        }
}

// Adds into `sum` the dot products over steps [s0, s1) of a row of K values.
//   wa, wb     this lane's two weight rows (g and g + 8 of the 16), at k = 0, of
//              any alignment; wbegin/wend bound their array
//   x[n]       this lane's token row of block n (token 8n + g), at k = 0, of any
//              alignment; xbegin/xend bound their array
//   COHERENT   the token rows were written by other blocks of this kernel: they
//              are read from L2, are 16-byte aligned and padded with zeros to
//              whole steps (xbegin/xend unused)
// sum[n][0..3]: rows g, g, g+8, g+8 and tokens 8n + 2t, +1, 2t, +1.
template <int NB, int U, bool COHERENT = false>
__device__ __forceinline__ void q8_dot(int (&sum)[NB][4], const int8_t *wa, const int8_t *wb,
                                       const int8_t *const (&x)[NB], int64_t K, int s0, int s1,
                                       const int8_t *wbegin, const int8_t *wend,
                                       const int8_t *xbegin, const int8_t *xend) {
    const int t = (int)(threadIdx.x & 3);
    const int full = (int)(K / kQ8Step);
    const int sf = s1 < full ? s1 : full;
    float acc[NB][4];
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[n][i] = 0.0f;
    auto wload = [&](const int8_t *row, int s) {
        const int8_t *p = row + (int64_t)s * kQ8Step + 16 * t;
        return load16_unaligned(p, wbegin, wend);
    };
    auto xload = [&](const int8_t *row, int s) {
        const int8_t *p = row + (int64_t)s * kQ8Step + 16 * t;
        if (COHERENT) return __ldcg(reinterpret_cast<const uint4 *>(p));
        return load16_unaligned(p, xbegin, xend);
    };
    int s = s0, since = 0;
    static_assert(kQ8ExactSteps % U == 0, "an exact chunk is whole unrolled rounds");
    for (; s + U <= sf; s += U) {
        uint4 a[U], b[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            a[u] = wload(wa, s + u);
            b[u] = wload(wb, s + u);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            uint4 xv[NB];
#pragma unroll
            for (int n = 0; n < NB; ++n) xv[n] = xload(x[n], s + u);
            q8_step<NB>(acc, a[u], b[u], xv);
        }
        since += U;
        if (since == kQ8ExactSteps) {
            q8_flush<NB>(sum, acc);
            since = 0;
        }
    }
    for (; s < sf; ++s) {   // at most U - 1 steps, in the chunk the last round left open
        uint4 xv[NB];
        const uint4 a = wload(wa, s), b = wload(wb, s);
#pragma unroll
        for (int n = 0; n < NB; ++n) xv[n] = xload(x[n], s);
        q8_step<NB>(acc, a, b, xv);
    }
    q8_flush<NB>(sum, acc);
    if (s < s1) {   // the row's last K % 64 values
        const int64_t k = (int64_t)s * kQ8Step + 16 * t;
        const int valid = (int)(K - k < 0 ? 0 : K - k > 16 ? 16 : K - k);
        uint4 xv[NB];
        const uint4 a = load16_bytes(wa + k, valid), b = load16_bytes(wb + k, valid);
#pragma unroll
        for (int n = 0; n < NB; ++n)
            xv[n] = COHERENT ? __ldcg(reinterpret_cast<const uint4 *>(x[n] + k)) : load16_bytes(x[n] + k, valid);
        q8_step<NB>(acc, a, b, xv);
        q8_flush<NB>(sum, acc);
    }
}

// ---- the same product from a ring of bulk copies ----------------------------------
//
// One stage is RT 16-row tiles of KB steps (64 k each).  A row's share of it is
// one bulk copy (4 KB at RT = 1: a 64-byte-wide TMA box ran at half the rate), a
// tile's are issued by a warp of their own.  Rows lie 64 bytes further apart
// than they are long, so that the 128-bit reads of a fragment, rows g and g + 1
// together, meet no bank conflict.  Sixteen consumer warps take STEPS steps
// each, of RW tiles.  Their sums of a tile, integers, meet in shared memory: a
// 16-byte store per fragment and lane, and one pass of reads (added there by
// atomics, 4 tokens took 15.8 us instead of 13.8 at 14336 x 4096).
//
// Up to 8 tokens the products are 8-bit MMAs (mma.sync m16n8k32 s8): exact
// without any expansion, and although sm_103a runs them at a sixteenth of the
// FP16 rate per byte, 31 bytes of W per cycle and SM is more than memory brings
// (23).  For 16 tokens that halves, and the FP16 form takes over (alternate steps
// by one and the other ran 35% slower than FP16 alone).  There a warp takes RW = 2
// row tiles, so that the tokens' bytes, which would otherwise be as many as W's,
// are fetched half as often.  For one token dp4a is cheaper still (12.6 against 13.7
// us at 14336 x 4096; for two 14.2 against 13.8).
constexpr int kQ8Consumers = 16;
template <int RT, int RW, int STEPS_>
struct Q8Stage {
    static constexpr int STEPS = STEPS_, ROWS = 16 * RT;
    static constexpr int KW = kQ8Consumers / (RT / RW);   // warps that divide a tile's steps
    static constexpr int KB = KW * STEPS;
    static constexpr uint32_t LD = KB * kQ8Step + 64;
    static constexpr uint32_t BYTES = ROWS * LD;
    static_assert(RT % RW == 0 && kQ8ExactSteps % STEPS == 0, "the warps cover the stage");
};

__device__ __forceinline__ void mma_s8(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// q8_step with 8-bit MMAs: as there, words of the 16 bytes are fed in pairs.
__device__ __forceinline__ void q8_step_s8(int (&sum)[4], const uint4 &wa, const uint4 &wb, const uint4 &x) {
    mma_s8(sum, wa.x, wb.x, wa.y, wb.y, x.x, x.y);
    mma_s8(sum, wa.z, wb.z, wa.w, wb.w, x.z, x.w);
}

// The same for NT single tokens without an MMA: sum[j][0], sum[j][1] take this
// lane's 16 bytes of rows g and g + 8 times token j's; the four lanes of a quad
// hold parts of one sum.  8 NT dp4a a step (half rate) against two 8-bit MMAs at
// 17 cycles of the SM each: the cheaper way up to 4 tokens.
template <int NT>
__device__ __forceinline__ void q8_step_dp(int (&sum)[NT][2], const uint4 &wa, const uint4 &wb, const uint4 (&x)[NT]) {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        sum[j][0] = __dp4a((int)wa.x, (int)x[j].x, sum[j][0]);
        sum[j][1] = __dp4a((int)wb.x, (int)x[j].x, sum[j][1]);
        sum[j][0] = __dp4a((int)wa.y, (int)x[j].y, sum[j][0]);
        sum[j][1] = __dp4a((int)wb.y, (int)x[j].y, sum[j][1]);
        sum[j][0] = __dp4a((int)wa.z, (int)x[j].z, sum[j][0]);
        sum[j][1] = __dp4a((int)wb.z, (int)x[j].z, sum[j][1]);
        sum[j][0] = __dp4a((int)wa.w, (int)x[j].w, sum[j][0]);
        sum[j][1] = __dp4a((int)wb.w, (int)x[j].w, sum[j][1]);
    }
}

// Bulk copy into shared memory: 16-byte aligned addresses and size.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}

// One lane of the converged warp, the same on every call.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// The whole warp waits, and agrees on whether the phase completed.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, limit_ns)) != 0;
}

#endif  // __CUDACC__

}  // namespace sgemm_gb300
