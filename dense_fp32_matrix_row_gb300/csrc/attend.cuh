// attend.cuh -- attention of one new token per sequence over the 8-bit paged
// cache, as a template over the heads' size (instantiated in attend_*.cu).
//
//     s_t = scale * q . k_t        p_t = 2^(s_t*log2(e) - m)        m: see consume()
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
// up to 8 heads that share a key head as the MMA's 8 columns (NT sets of those).  The
// order of an MMA's inner index is free as long as A and B agree, so every lane
// reads 16 consecutive bytes of a row.  S^T comes out as P^T goes in except for a
// transposition of 8 x 8, one instruction (movmatrix).
//
// Work: the strips of all sequences' key heads are one list, divided evenly over
// the blocks (one on an SM) from the lengths as they are on the device, and over
// a block's warps: ragged batches balance, and one long sequence spreads over
// every SM.  A warp streams its strips through a ring of its own in shared memory
// (cp.async) and meets no barrier until its last: what a key head costs besides
// its strips (queries, results) is latency that the other warps cover.  A key
// head that several warps share is summed at the end, first within the block,
// then by the last of the blocks that share it, always in the same order.
//
// Bound by memory as long as sequences are long, by latency where they are short, and by
// issue slots with many query heads to a key head.  Measured (bf16, 8 key heads of 128, 8
// query heads to each; copies alone, without any arithmetic, stream at 7.0 TB/s):
//   64 sequences of 16384 tokens, 2.2 GB, 328 us, 6.8 TB/s;
//   64 of 1024 to 8192, 602 MB, 107 us: 3 us until the first copies, 5 to 8 of sums
//     at the end, while other SMs still load memory;
//   one of 131072 (4 heads to each), 277 MB, 52 us, the same; one of 8192, 17 MB, 14 us;
//   one of 500, 8.2 us: two strips a warp (1.1 us each), four dependent loads before
//     them (length, page number, queries, strip), two sums behind them.
#pragma once

#include <atomic>

#include "cache.cuh"

namespace sgemm_gb300 {

constexpr int kStrip = 16;                 // tokens
constexpr int kJoin = 48;                  // blocks' parts summed at a time
// A block boundary within so many strips of a key head's first or last strip moves
// there: joining blocks costs about as long as reading twice as many.  So does one
// anywhere in a key head of at most kFew strips or, where there is too little work
// for all SMs, kUnshared (half as many of FP32, whose strips take twice as long): a
// block takes those alone in about the time that joining would add.
constexpr int kSnap = 16, kFew = 48, kUnshared = 96;
constexpr int kLeast = 1;                  // strips to a warp, before work goes to another block
// A key head of at most so many strips is one warp's: summing two warps' parts costs
// about as long as four strips.
constexpr int kWhole = 10;

struct AttendParams {
    int B, Hk, G, D, groups;               // groups: of 8*NT query heads to a key head
    int page, width;
    uint32_t page_mul, page_shift;         // t / page = (t * page_mul) >> page_shift (host: divider())
    uint32_t chunk_mul;                    // q / chunks of a row = (q * chunk_mul) >> 16 for q < 192
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
    float *parts;                          // attend_parts() for each block
    unsigned *tickets;                     // 2 * gridDim.x for parts, gridDim.x for groups of parts
    unsigned *err;
};

cudaError_t launch_attend_64(const AttendParams &p, int type, int nt, int sms, cudaStream_t stream);
cudaError_t launch_attend_96(const AttendParams &p, int type, int nt, int sms, cudaStream_t stream);
cudaError_t launch_attend_128(const AttendParams &p, int type, int nt, int sms, cudaStream_t stream);
cudaError_t launch_attend_192(const AttendParams &p, int type, int nt, int sms, cudaStream_t stream);
cudaError_t launch_attend_256(const AttendParams &p, int type, int nt, int sms, cudaStream_t stream);
// The most sets of 8 query heads that a form takes (see attend.cu).
constexpr int attend_sets(int dt, bool bf16) { return dt <= 128 ? (bf16 ? 4 : 3) : dt == 192 ? 2 : bf16 ? 2 : 1; }
// Warps of a block, as many as 65536 registers hold, as many on each quarter of an SM
// (terms: 2 for FP32; 16 sequences of 16384, 8 key heads: 3 sets of heads of 64 with 8 warps 205
// us, with 12 173; of 128 with 8 150, with 10 178.  FP32 heads of 128 with 12 109, with 16 106,
// but 7 short sequences 12.7 and 13.5).
constexpr int attend_warps(int dt, int nt, int terms) {
    const int n = nt * terms;
    return dt == 64 ? (nt > 2 ? 12 : 16) : dt == 96 ? (n == 1 ? 16 : n <= 3 || nt == 2 ? 12 : 8)
         : dt == 128 ? (n == 1 ? 16 : nt <= 2 ? 12 : 8) : dt == 192 && n == 1 ? 12 : 8;
}
// Floats of one part: sums of 8*nt heads, then each head's m and sum of p.
constexpr int attend_part(int dt, int nt) { return 8 * nt * (dt + 2); }
// Parts in the workspace: two of each block, one of each warp.
constexpr int attend_parts(int dt, int nt, int terms) { return 2 + attend_warps(dt, nt, terms); }

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

__device__ __forceinline__ float log2_fast(float x) {      // -infinity for 0
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
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
// 1 / v for a power of two from 2^-126 to 2^126.
__device__ __forceinline__ float inverse_pow2(float v) { return __uint_as_float(0x7f000000u - __float_as_uint(v)); }
// e with 2^e <= v < 2^(e+1) for a finite v >= 2^-118; -118 below, 128 beyond.
__device__ __forceinline__ int exponent(float v) { return max(-118, (int)((__float_as_uint(v) >> 23) & 0xff) - 127); }

template <int DT, int NT, int TERMS>
struct Shape {
    static constexpr int WARPS = attend_warps(DT, NT, TERMS);
    static constexpr int THREADS = 32 * WARPS;
    static constexpr int CH = DT / 16;                 // 16-byte chunks of a row
    static constexpr int STEPS = DT / 16;              // MMAs along the head, and dim tiles of O^T
    static constexpr int ROWS = kStrip * (DT == 96 ? 128 : DT);        // bytes of a strip's keys
    // What a lane reads of a key row, as the MMAs' inner index: 16 bytes of each 64, and
    // 8 of the last 32 of 96.
    static constexpr int PIECES = (CH + 3) / 4;
    static constexpr int words(int piece) { return DT / 16 - 4 * piece < 4 ? DT / 16 - 4 * piece : 4; }
    static constexpr int STAGE = 2 * ROWS + 256;       // keys, values, 16 + 16 scales, the mask
    static constexpr int HEADS = 8 * NT;
    static constexpr int PART = attend_part(DT, NT);
    // The queries' operands: in registers as long as they leave room for the sums (16 sequences
    // of 16384, registers against shared memory: bf16 heads of 128, 16 to a key head, 115 and 112
    // us, of 256, 8, 174 and 177; FP32 heads of 64, 16, 108 and 94, of 128, 8, 111 and 108; 96: sums
    // take less, heads of 80, 16, 99 and 106).
    static constexpr bool Q_SHARED = NT * TERMS > 1 && !(DT == 96 && NT * TERMS == 2);
    // Where a strip's chunks go is kept, rather than found for each strip, where registers
    // are left for it (heads of 96 78 -> 75 us, of 128, 16 to a key head, 109 -> 107, FP32, 8, 107 -> 104,
    // but bf16, 8, 91 -> 94).
    static constexpr bool PLACES = DT < 256 && (DT != 128 || NT * TERMS > 1);
    static constexpr int QUERIES = Q_SHARED ? NT * TERMS * STEPS * 256 : 0;       // a warp
    static constexpr int NOTES = WARPS * (72 + 8) + 128;      // see the kernel
    static constexpr int ROOM = 227 * 1024 - 128 - NOTES - WARPS * QUERIES;
    static constexpr int MOST = ROOM / (WARPS * STAGE);
    static constexpr int STAGES = MOST > 6 ? 6 : MOST;
    static constexpr int SMEM = WARPS * (STAGES * STAGE + QUERIES) + NOTES + 128;
    static_assert(STAGES >= 2, "a ring has two strips at least");
    static_assert(PART * 4 <= STAGES * STAGE, "a ring holds its warp's sums");
};

// Byte offset of chunk c of row r in a strip, chunks exchanged within 128 bytes so
// that neither the keys' reads (8 lanes: 2 rows, 4 chunks of each) nor the values'
// (8 lanes: 4 rows, 2 chunks) meet in a bank.  96: rows lie as 128 do; 16 lanes read
// halves of chunks (keys: 4 rows, 2 chunks of each; values: every other of 8 rows).
// 192: eight chunks of each row as 128, then four as 64.
// Packed closer, with one more stage, four chunks of a row apart from its other two: 75 -> 79 us.
template <int DT>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
    if constexpr (DT == 64) return (uint32_t)((r >> 1) * 128 + ((((r & 1) * 4 + c) ^ (r & 6)) << 4));
    else if constexpr (DT == 96) return (uint32_t)(r * 128 + ((c ^ (((r ^ r >> 2) & 1) << 2 | (r & 2))) << 4));
    else if constexpr (DT == 192) return c < 8 ? chunk_at<128>(r, c) : 2048 + chunk_at<64>(r, c - 8);
    else return (uint32_t)(r * DT + (c >> 3) * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// The strips of a sequence that its new token attends to.
struct Span {
    int first, last;       // tokens [first, last)
    int strip0, strips;    // strips of 16 from token 16*strip0 on
};

// Of a sequence of n tokens, 0 <= n.
__device__ __forceinline__ Span span_of(const AttendParams &p, int n) {
    Span s;
    s.last = n;
    s.first = p.window > 0 && n > p.window ? n - p.window : 0;
    s.strip0 = s.first / kStrip;
    s.strips = n > 0 ? (n - 1) / kStrip + 1 - s.strip0 : 0;
    return s;
}
// A sequence's length, within what its pages hold.  (Read by plain loads, as page
// numbers are: a load through the read-only path might be moved before pdl_wait.)
__device__ __forceinline__ int tokens_of(const AttendParams &p, int b) {
    return max(0, min(p.lens[b], p.width * p.page));
}

// A place in the list: sequence, key head, group of its query heads, strip.
struct Cursor {
    int b, h, group, strip;
    Span span;
    // Only where another strip follows in the list, by the whole warp.
    __device__ __forceinline__ void step(const AttendParams &p) {
        if (++strip < span.strips) return;
        strip = 0;
        if (++group < p.groups) return;
        group = 0;
        if (++h < p.Hk) return;
        h = 0;
        // the next sequence with tokens: the warp looks at 32 at a time
        const int lane = threadIdx.x & 31;
        for (++b;; b += 32) {
            const int n = b + lane < p.B ? tokens_of(p, b + lane) : 0;
            const uint32_t some = __ballot_sync(0xffffffffu, n > 0);
            if (some == 0 && b + 32 < p.B) continue;
            const int k = max(__ffs(some) - 1, 0);
            b += k;
            span = span_of(p, __shfl_sync(0xffffffffu, n, k));
            return;
        }
    }
};

// Begins of even shares of n: the first n % shares of them are one longer.
struct Shares {
    int q, r;
    __device__ __forceinline__ Shares(int n, int shares) : q((int)((unsigned)n / (unsigned)shares)), r(n - q * shares) {}
    __device__ __forceinline__ int begin(int i) const { return q * i + min(i, r); }
    // The first share that begins behind `at`.
    __device__ __forceinline__ int behind(int at) const {
        return 1 + (at < (q + 1) * r ? at / (q + 1) : (at - r) / max(q, 1));
    }
};

// Finds places in the list, by a whole warp: it keeps 32 sequences, a lane each.
// Where there are more, `sums` has the strips of each of a block's warps' runs of
// `run` sequences, a multiple of 32.
struct Locator {
    int from, base;             // the first of the 32 sequences, and its place in the list
    int tokens;                 // of this lane's sequence
    int before, upto;           // its strips: [base + before, base + upto) of the list
    const int *sums;
    int run;

    __device__ __forceinline__ void load(const AttendParams &p, int first, int at) {
        const int lane = threadIdx.x & 31;
        from = first;
        base = at;
        tokens = from + lane < p.B ? tokens_of(p, from + lane) : 0;
        const int count = span_of(p, tokens).strips * (p.Hk * p.groups);
        upto = count;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += x;
        }
        before = upto - count;
    }
    __device__ __forceinline__ int all() const { return __shfl_sync(0xffffffffu, upto, 31); }

    // The strip at `at`, which is less than the list's length.
    __device__ __forceinline__ Cursor find(const AttendParams &p, int at) {
        if (p.B > 32 && (at < base || at >= base + all())) {
            int here = 0, w = 0;
            while (at >= here + sums[w]) here += sums[w++];
            load(p, w * run, here);
            while (at >= base + all()) load(p, from + 32, base + all());
        }
        const int k = __ffs(__ballot_sync(0xffffffffu, base + upto > at)) - 1;
        const int off = at - base - __shfl_sync(0xffffffffu, before, k);
        Cursor c;
        c.b = from + k;
        c.span = span_of(p, __shfl_sync(0xffffffffu, tokens, k));
        const int item = (int)((unsigned)off / (unsigned)c.span.strips);
        c.strip = off - item * c.span.strips;
        c.h = p.groups == 1 ? item : item / p.groups;
        c.group = item - c.h * p.groups;
        return c;
    }
};

// The list's division: block c begins at the c-th even share, unless that is within
// kSnap strips of a key head's begin or end.
struct Division {
    int total, blocks, unshared;
    __device__ __forceinline__ Division(int strips, int per_block, int terms)
        : total(strips), blocks(min((int)gridDim.x, max(1, (strips - 1) / per_block + 1))),
          unshared((blocks < (int)gridDim.x ? kUnshared : kFew) / terms) {}
    // A boundary at `at`, off strips into a key head of n strips, moved to its nearer end.
    static __device__ __forceinline__ int moved(int at, int off, int n) { return 2 * off < n ? at - off : at + (n - off); }
    __device__ __forceinline__ int start(const AttendParams &p, Locator &list, int c) const {
        if (c == blocks) return total;
        if (c == 0) return 0;
        const int at = Shares(total, blocks).begin(c);
        const Cursor x = list.find(p, at);
        const int off = x.strip, n = x.span.strips;
        return n > unshared && off > kSnap && n - off > kSnap ? at : moved(at, off, n);
    }
    // Of a key head at [at, at + n): the blocks first..last that share it, by the
    // boundaries that lie within it.  first >= last: one block alone.
    __device__ __forceinline__ void blocks_of(int at, int n, int &first, int &last) const {
        const Shares s(total, blocks);
        first = s.behind(at + kSnap) - 1;
        last = n > unshared ? s.behind(at + n - kSnap - 1) - 1 : first;
    }
};

// A part holds unnormalised sums of all heads, then each head's m and sum of p.  Four
// dims stay together; they are exchanged within a head so that a warp's stores meet
// in no bank of shared memory.
template <int DT>
__device__ __forceinline__ int part_at(int head, int d) { return head * DT + (d ^ ((head >> 1 & 3) << 2)); }

template <typename T>
__device__ __forceinline__ void store_out(const AttendParams &p, T *to, const float (&v)[4]) {
    if (p.o_vec) {
        store_vec<T, 4>(to, v);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) to[i] = from_f32<T>(v[i]);
    }
}
// (The logarithm of the mantissa alone: top may lie far from it.)
__device__ __forceinline__ float lse_of(float top, float total) {
    if (total == 0.0f) return -INFINITY;
    const int e = min(exponent(total), 126);
    return ((top + (float)e) + log2f(total * pow2(-e))) * 0.69314718055994531f;
}

// Four dims of a head's result; with d == 0 its lse too.
template <typename T>
__device__ __forceinline__ void finish_head(const AttendParams &p, int b, int h, int head, int d, float4 o, float top,
                                            float total) {
    if (head >= p.G || d >= p.D) return;
    const float inv = total != 0.0f ? 1.0f / total : 0.0f;
    const float v[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
    store_out<T>(p, static_cast<T *>(p.out) + b * p.o_ld + ((int64_t)h * p.G + head) * p.o_hs + d, v);
    if (d == 0 && p.lse) p.lse[((int64_t)b * p.Hk + h) * p.G + head] = lse_of(top, total);
}

// Four dims of a head summed over parts.
struct Sum {
    float4 o;
    float top, total;
    __device__ __forceinline__ Sum() : o(make_float4(0.0f, 0.0f, 0.0f, 0.0f)), top(-kLargest), total(0.0f) {}
    __device__ __forceinline__ void rise(float to) {
        const float f = exp2_fast(top - to);
        top = to;
        total *= f;
        o.x *= f; o.y *= f; o.z *= f; o.w *= f;
    }
    // A part's m and sum of p, and its dims; m is at most `top`.
    __device__ __forceinline__ void add(float2 y, float4 x) {
        const float f = exp2_fast(y.x - top);
        total += y.y * f;
        o.x += x.x * f; o.y += x.y * f; o.z += x.z * f; o.w += x.w * f;
    }
};

template <int DT, int NT, typename T>
struct Attend {
    static constexpr bool SPLIT = sizeof(T) == 4;      // FP32: operands in two FP16 terms
    static constexpr int TERMS = SPLIT ? 2 : 1;
    using S = Shape<DT, NT, TERMS>;

    const AttendParams &p;
    uint32_t ring;          // this warp's stages
    uint32_t queries;       // Q_SHARED: this warp's
    int warp, lane, g, j;
    uint32_t places[S::PLACES ? (S::CH + 3) / 4 : 1];     // find_place() of 2 * i and 2 * i + 1

    // the strip to be loaded next
    Cursor next;
    int left;               // strips not yet loaded
    // its page number (that of this lane's token, where strips reach over pages), asked
    // for when the strip before is loaded
    int next_page;

    __device__ __forceinline__ Attend(const AttendParams &pp, uint32_t smem) : p(pp) {
        warp = threadIdx.x >> 5;
        lane = threadIdx.x & 31;
        g = lane >> 2;
        j = lane & 3;
        ring = smem + warp * (S::STAGES * S::STAGE);
        if constexpr (S::PLACES) {
#pragma unroll
            for (int i = 0; i < (S::CH + 3) / 4; ++i) places[i] = find_place(2 * i) | find_place(2 * i + 1) << 16;
        }
        queries = smem + S::WARPS * (S::STAGES * S::STAGE) + warp * S::QUERIES;
    }

    // Where the strip's chunk number lane + 32 * i goes.
    __device__ __forceinline__ uint32_t find_place(int i) const {
        const int q = lane + 32 * i, r = (int)((uint32_t)q * p.chunk_mul >> 16) & (kStrip - 1);
        return chunk_at<DT>(r, q - r * (p.D >> 4));
    }
    __device__ __forceinline__ uint32_t place_of(int i) const {
        if constexpr (S::PLACES) return places[i / 2] >> 16 * (i % 2) & 0xffff;
        else return find_place(i);
    }

    __device__ __forceinline__ int page_of(int t) const {
        return (int)(((uint64_t)(uint32_t)t * p.page_mul) >> p.page_shift);
    }

    __device__ __forceinline__ void look_up() {
        const int32_t *row = p.table + next.b * p.ld_table;
        int t = (next.span.strip0 + next.strip) * kStrip;
        if (!p.whole) t = max(min(t + (lane & 15), next.span.last - 1), next.span.first);
        next_page = row[page_of(t)];
    }

    // Starts the copies of the strip at `next` into stage s, and moves on.
    __device__ __forceinline__ void load(int s) {
        if (left > 0) {
            const uint32_t at = ring + s * S::STAGE;
            const int h = next.h;
            const int t0 = (next.span.strip0 + next.strip) * kStrip;
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
                        // one chunk behind another, whatever the rows' size (16 sequences of 16384,
                        // heads of 64: 64 -> 61 us, of 112: 101 -> 98; 256, with twice the divisions,
                        // 175 -> 178)
                        const int q = lane + 32 * i, r = q / S::CH, c = q % S::CH;
                        if (DT == 256 ? c < chunks : q < 16 * chunks) {
                            const uint32_t to = at + (DT == 256 ? chunk_at<DT>(r, c) : place_of(i));
                            const int from = DT == 256 ? r * p.D + c * 16 : q * 16;
                            cp_async16(to, k + from);
                            cp_async16(to + S::ROWS, v + from);
                        }
                    }
                    const float *scale = lane < 16 ? p.ks + page * p.ks_stride : p.vs + page * p.vs_stride;
                    cp_async4(at + 2 * S::ROWS + 4 * lane, scale + row + (lane & 15));
                }
            } else {
                const int row = h * p.page + (t - page_of(t) * p.page);    // of this lane's token
                // places go round whole, not as page and row: 16 sequences of 16384, pages of 20, heads of
                // 128 102 -> 95 us, 256 200 -> 181
                const int64_t in_k = page * p.k_stride + (int64_t)row * p.D, in_v = page * p.v_stride + (int64_t)row * p.D;
#pragma unroll
                for (int i = 0; i < S::CH / 2; ++i) {
                    const int q = lane + 32 * i, r = q / S::CH, c = q % S::CH;
                    const int64_t k = __shfl_sync(0xffffffffu, in_k, r), v = __shfl_sync(0xffffffffu, in_v, r);
                    if (c < chunks && (mask >> r & 1)) {
                        cp_async16(at + chunk_at<DT>(r, c), p.k + k + c * 16);
                        cp_async16(at + S::ROWS + chunk_at<DT>(r, c), p.v + v + c * 16);
                    }
                }
                if (fine) {
                    const float *scale = lane < 16 ? p.ks + page * p.ks_stride : p.vs + page * p.vs_stride;
                    cp_async4(at + 2 * S::ROWS + 4 * lane, scale + row);
                }
            }
            if (lane == 0) asm volatile("st.shared.u32 [%0], %1;" ::"r"(at + 2 * S::ROWS + 128), "r"(mask) : "memory");
            if (--left > 0) {
                next.step(p);
                look_up();
            }
        }
        cp_commit();
    }

    // ---- one key head's running state -------------------------------------------------
    uint32_t qf[S::Q_SHARED ? 1 : NT][TERMS][S::STEPS][2];
    float qmul[NT][2];                  // turns a product into a score in base 2, without the key's scale
    float m[NT][2], sum[NT][2];         // of heads 2j and 2j + 1; sum: of this lane's tokens
    float vmul, vcap;                   // a power of two that the value scales carry; the largest scale it is for
    float acc[S::STEPS][NT][4];

    // The queries of the key head at `at`, as they lie: this lane's chunks of one head
    // of each eight.
    struct Queries {
        uint32_t w[NT][S::PIECES][4 * (int)sizeof(T)];
    };
    __device__ __forceinline__ void fetch(Queries &x, const Cursor &at) const {
        const int first = at.group * S::HEADS;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int head = first + nt * 8 + g;
            const T *q = static_cast<const T *>(p.q) + at.b * p.q_ld + (at.h * (int64_t)p.G + head) * p.q_hs;
#pragma unroll
            for (int i = 0; i < S::PIECES; ++i) {
                const int d = key_dim(i), n = S::words(i);       // 4 * n elements
                uint32_t(&w)[4 * (int)sizeof(T)] = x.w[nt][i];
                if (head >= p.G || d >= p.D) {
#pragma unroll
                    for (int e = 0; e < n * (int)sizeof(T); ++e) w[e] = 0;
                } else if (p.q_vec) {
#pragma unroll
                    for (int e = 0; e < n * (int)sizeof(T) / 4; ++e) {
                        const uint4 u = *reinterpret_cast<const uint4 *>(q + d + e * (16 / (int)sizeof(T)));
                        w[4 * e] = u.x; w[4 * e + 1] = u.y; w[4 * e + 2] = u.z; w[4 * e + 3] = u.w;
                    }
                } else if constexpr (SPLIT) {
#pragma unroll
                    for (int e = 0; e < 4 * n; ++e) w[e] = __float_as_uint(q[d + e]);
                } else {
                    const unsigned short *h = reinterpret_cast<const unsigned short *>(q + d);
#pragma unroll
                    for (int e = 0; e < 2 * n; ++e) w[e] = (uint32_t)h[2 * e] | (uint32_t)h[2 * e + 1] << 16;
                }
            }
        }
    }

    // The same as the MMA's B, scaled by a power of two into FP16's range (below 2^15: a
    // BF16 query is exact but for elements below 2^-31 of its largest).
    __device__ __forceinline__ void begin(const Cursor &at) {
        Queries x;
        fetch(x, at);
        auto value = [&](int nt, int i, int e) {
            if constexpr (SPLIT) return __uint_as_float(x.w[nt][i][e]);
            else return __uint_as_float((e & 1) ? x.w[nt][i][e >> 1] & 0xffff0000u : x.w[nt][i][e >> 1] << 16);
        };
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float most = 0.0f;
#pragma unroll
            for (int i = 0; i < S::PIECES; ++i)
#pragma unroll
                for (int e = 0; e < 4 * S::words(i); ++e) most = fmaxf(most, fabsf(value(nt, i, e)));
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
            const int k = min(14 - min(exponent(most), 127), 126);
            const float up = pow2(k), mul = p.scale_log2 * pow2(-k);
#pragma unroll
            for (int i = 0; i < S::PIECES; ++i)
#pragma unroll
                for (int w = 0; w < S::words(i); ++w) {
                    const float a = value(nt, i, 4 * w) * up, b = value(nt, i, 4 * w + 1) * up,
                                c = value(nt, i, 4 * w + 2) * up, d = value(nt, i, 4 * w + 3) * up;
                    const uint32_t lo = half_pair(a, b), hi = half_pair(c, d);
                    put_query(nt, 0, 4 * i + w, lo, hi);
                    if constexpr (SPLIT) put_query(nt, 1, 4 * i + w, half_pair_rest(a, b, lo), half_pair_rest(c, d, hi));
                }
            qmul[nt][0] = __shfl_sync(0xffffffffu, mul, 8 * j);
            qmul[nt][1] = __shfl_sync(0xffffffffu, mul, 8 * j + 4);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                m[nt][k] = -kLargest;
                sum[nt][k] = 0.0f;
            }
#pragma unroll
            for (int i = 0; i < S::STEPS; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[i][nt][k] = 0.0f;
        }
        vmul = 1.0f;
        vcap = -1.0f;
    }

    // A lane reads what it has written itself.
    __device__ __forceinline__ void put_query(int nt, int term, int step, uint32_t lo, uint32_t hi) {
        if constexpr (S::Q_SHARED) {
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

    // The first dim of this lane's i-th piece of a key row.
    __device__ __forceinline__ int key_dim(int i) const {
        if constexpr (DT <= 96) return i == 0 ? 16 * j : 64 + 8 * j;
        else if (DT == 192 && i == 2) return 128 + 16 * j;
        else return ((i >> 1) * 8 + 2 * j + (i & 1)) * 16;
    }

    __device__ __forceinline__ void consume(int s) {
        const uint32_t at = ring + s * S::STAGE;
        const uint32_t mask = lds4(at + 2 * S::ROWS + 128);
        // FP32: what an MMA cuts off goes by the largest of what it adds, so the queries' second
        // terms are summed apart, and every 64 dims (lse of 64 x 16 heads of 256, 73 tokens:
        // 0.6e-7 off instead of 3e-7).
        float sc[NT][4], rest[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 4; ++k) sc[nt][k] = rest[nt][k] = 0.0f;
#pragma unroll
        for (int i = 0; i < S::PIECES; ++i) {
            float dims[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int k = 0; k < 4; ++k) dims[nt][k] = 0.0f;
            const int c = key_dim(i) >> 4;
            uint4 lo, hi;
            if constexpr (DT == 96) {
                if (i == 1) {
                    const uint2 l = lds8(at + chunk_at<DT>(g, c) + 8 * (j & 1)), h = lds8(at + chunk_at<DT>(g + 8, c) + 8 * (j & 1));
                    lo = make_uint4(l.x, l.y, 0, 0);
                    hi = make_uint4(h.x, h.y, 0, 0);
                }
            }
            if (S::words(i) == 4) {
                lo = lds16(at + chunk_at<DT>(g, c));
                hi = lds16(at + chunk_at<DT>(g + 8, c));
            }
            const uint32_t wl[4] = {lo.x, lo.y, lo.z, lo.w}, wh[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
            for (int w = 0; w < S::words(i); ++w) {
                uint32_t a0, a1, a2, a3;
                q8_to_f16(wl[w], a0, a2);
                q8_to_f16(wh[w], a1, a3);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int t = 0; t < TERMS; ++t) {
                        const uint2 q = query(nt, t, 4 * i + w);
                        mma_f16(!SPLIT ? sc[nt] : t == 0 ? dims[nt] : rest[nt], a0, a1, a2, a3, q.x, q.y);
                    }
            }
            if constexpr (SPLIT) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int k = 0; k < 4; ++k) sc[nt][k] += dims[nt][k];
            }
        }
        const uint32_t scales = at + 2 * S::ROWS;
        const float k0 = __uint_as_float(lds4(scales + 4 * g)), k1 = __uint_as_float(lds4(scales + 4 * g + 32));
        float v0 = __uint_as_float(lds4(scales + 64 + 4 * g)), v1 = __uint_as_float(lds4(scales + 64 + 4 * g + 32));
        bool look = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            if constexpr (SPLIT) {
#pragma unroll
                for (int k = 0; k < 4; ++k) sc[nt][k] += rest[nt][k];
            }
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
        // FP16 takes the products p * (value scale) as x = p * u, u = scale * vmul.  vmul brings
        // the largest scale so far to [2^8, 2^10]; m is the head's, and such that its largest x
        // is between 2^8 and 2^15: both are kept until a scale passes vcap or an x 2^15.  FP16
        // rounds an x to 11 bits, or to 2^-24 where it is below 2^-14: by 2^-33 of the head's
        // largest product at most, whatever other tokens' scales are.  As u is at most 2^10,
        // scores up to m + 5 need no closer look (one at every strip: 2 to 4% of the time).
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            look |= fmaxf(sc[nt][0], sc[nt][2]) > m[nt][0] + 5.0f || fmaxf(sc[nt][1], sc[nt][3]) > m[nt][1] + 5.0f;
        look |= fmaxf(fabsf(v0), fabsf(v1)) > vcap;
        if (__any_sync(0xffffffffu, look) && (vcap < 0.0f || grown(sc, v0, v1))) rescale(sc, v0, v1);
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
        if constexpr (DT <= 96) {
            // 8 dims of 64 a lane: half a chunk of each of its four tokens; of 96, 4 more
            uint2 r[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) r[k] = lds8(vals + chunk_at<DT>(2 * j + (k & 1) + (k >> 1) * 8, g >> 1) + (g & 1) * 8);
            values(0, r[0].x, r[1].x, r[2].x, r[3].x, pf);
            values(1, r[0].y, r[1].y, r[2].y, r[3].y, pf);
            if constexpr (DT == 96) {
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    w[k] = lds4(vals + chunk_at<DT>(2 * j + (k & 1) + (k >> 1) * 8, 4 + (g >> 2)) + (g & 3) * 4);
                values(2, w[0], w[1], w[2], w[3], pf);
            }
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
            if constexpr (DT == 192) {
                uint2 r[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) r[k] = lds8(vals + chunk_at<DT>(2 * j + (k & 1) + (k >> 1) * 8, 8 + (g >> 1)) + (g & 1) * 8);
                values(4, r[0].x, r[1].x, r[2].x, r[3].x, pf);
                values(5, r[0].y, r[1].y, r[2].y, r[3].y, pf);
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
            for (int nt = 0; nt < NT; ++nt) {
                float(&sum_of)[4] = acc[2 * word + half][nt];
                if constexpr (SPLIT) {
                    // An MMA cuts off what its sum has no room for: over hundreds of strips that
                    // is several units in FP32's last place, so strips are added up outside (which
                    // took 64 x 16384 tokens from 3.9e-6 to 0.9e-6 off; a BF16 result is rounded
                    // by a thousand times that).
                    float strip[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int t = TERMS - 1; t >= 0; --t)
                        mma_f16(strip, lo[2 * half], lo[2 * half + 1], hi[2 * half], hi[2 * half + 1], pf[nt][t][0], pf[nt][t][1]);
#pragma unroll
                    for (int k = 0; k < 4; ++k) sum_of[k] += strip[k];
                } else {
                    mma_f16(sum_of, lo[2 * half], lo[2 * half + 1], hi[2 * half], hi[2 * half + 1], pf[nt][0][0], pf[nt][0][1]);
                }
            }
    }

    // log2 of u's size, as m goes by it: at most 10, which no finite u passes, and at least -45,
    // so that p stays below 2^60 where the values are (next to) nothing.
    static __device__ __forceinline__ float size_of(float u) { return fminf(fmaxf(log2_fast(fabsf(u)), -45.0f), 10.0f); }

    // Whether the scales that products carry have to change for this strip, by its largest ones.
    __device__ __forceinline__ bool grown(const float (&sc)[NT][4], float v0, float v1) const {
        const float l0 = size_of(v0 * vmul), l1 = size_of(v1 * vmul);
        bool more = fmaxf(fabsf(v0), fabsf(v1)) > vcap;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 2; ++k) more |= fmaxf(sc[nt][k] + l0, sc[nt][k + 2] + l1) > m[nt][k] + 15.0f;
        return __any_sync(0xffffffffu, more);
    }

    // A head's sums taken from m to another one, products' times f besides.
    __device__ __forceinline__ void move(int nt, int k, float to, float f) {
        const float d = exp2_fast(m[nt][k] - to);
        m[nt][k] = to;
        sum[nt][k] *= d;
#pragma unroll
        for (int i = 0; i < S::STEPS; ++i) {
            acc[i][nt][k] *= d * f;
            acc[i][nt][k + 2] *= d * f;
        }
    }

    // vmul for a larger scale than those so far.  What is there shrinks with it, and m goes
    // down by as much, or later tokens like those would be rounded by the new scale's size.  (By
    // less where sums of p would pass 2^60.)
    __device__ __forceinline__ void take_scale(float vm) {
        const int e = min(exponent(vm), 127);
        const int down = vcap < 0.0f ? 0 : (int)(__float_as_uint(vmul) >> 23) - 127 - (8 - e);
        vmul = pow2(8 - e);
        vcap = e < 126 ? pow2(e + 2) : INFINITY;
        if (down == 0) return;
        const float f = down <= 126 ? pow2(-down) : 0.0f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float s = sum[nt][k];
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) s = fmaxf(s, __shfl_xor_sync(0xffffffffu, s, o));
                move(nt, k, m[nt][k] - (float)min(down, max(60 - exponent(s), 0)), f);
            }
    }

    __device__ __forceinline__ void rescale(const float (&sc)[NT][4], float v0, float v1) {
        float vm = fmaxf(fabsf(v0), fabsf(v1));
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) vm = fmaxf(vm, __shfl_xor_sync(0xffffffffu, vm, o));
        if (vm > vcap) take_scale(vm);
        const float l0 = size_of(v0 * vmul) - 8.0f, l1 = size_of(v1 * vmul) - 8.0f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float x = fmaxf(sc[nt][k] + l0, sc[nt][k + 2] + l1);
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
                move(nt, k, fmaxf(floorf(x), m[nt][k]), 1.0f);      // a whole number, for lower()
            }
    }

    // The dim of acc[i][.][0 or 1]; [2 or 3] is the next one.
    __device__ __forceinline__ int dim_of(int i) const {
        const int word = i >> 1;
        if (DT <= 96) return (word < 2 ? 8 * g + 4 * word : 64 + 4 * g) + 2 * (i & 1);
        if (DT == 192 && word >= 4) return 128 + 8 * g + 4 * (word & 3) + 2 * (i & 1);
        return 16 * (g + 8 * (word >> 2)) + 4 * (word & 3) + 2 * (i & 1);
    }

    // The sums of p over the warp's lanes (each lane's heads 2j and 2j + 1).
    __device__ __forceinline__ void total() {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) sum[nt][k] += __shfl_xor_sync(0xffffffffu, sum[nt][k], o);
    }

    // For sums that are to be joined with others' and might pass FP32's range then (the values
    // beyond 2^40, or p far beyond 1): sums over 2^k, with m + k, exactly (both are whole
    // numbers).  The sum of p becomes 1/2 to 1, times 2^-12, as several thousand parts may be joined.
    __device__ __forceinline__ void lower() {
        bool far = vmul < pow2(-40);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) far |= fmaxf(sum[nt][0], sum[nt][1]) > pow2(30);
        if (!__any_sync(0xffffffffu, far)) return;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int over = min(exponent(sum[nt][k]) + 13, 126);
                const float down = pow2(-over);
                m[nt][k] += (float)over;
                sum[nt][k] *= down;
#pragma unroll
                for (int i = 0; i < S::STEPS; ++i) {
                    acc[i][nt][k] *= down;
                    acc[i][nt][k + 2] *= down;
                }
            }
    }

    // As a part: see part_at.
    __device__ __forceinline__ void store(float *part) {
        lower();
        const float w = inverse_pow2(vmul);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int head = nt * 8 + 2 * j + k;
#pragma unroll
                for (int i = 0; i < S::STEPS; i += 2)
                    *reinterpret_cast<float4 *>(part + part_at<DT>(head, dim_of(i))) =
                        make_float4(acc[i][nt][k] * w, acc[i][nt][k + 2] * w, acc[i + 1][nt][k] * w, acc[i + 1][nt][k + 2] * w);
                if (g == 0) *reinterpret_cast<float2 *>(part + S::HEADS * DT + 2 * head) = make_float2(m[nt][k], sum[nt][k]);
            }
    }
    __device__ __forceinline__ void finish(const Cursor &at) const {
        const float w = inverse_pow2(vmul);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int head = at.group * S::HEADS + nt * 8 + 2 * j + k;
                if (head >= p.G) continue;
                const float total = sum[nt][k], inv = total != 0.0f ? 1.0f / total : 0.0f;
                T *to = static_cast<T *>(p.out) + at.b * p.o_ld + (at.h * (int64_t)p.G + head) * p.o_hs;
#pragma unroll
                for (int i = 0; i < S::STEPS; i += 2) {
                    const int d = dim_of(i);
                    const float v[4] = {acc[i][nt][k] * inv * w, acc[i][nt][k + 2] * inv * w, acc[i + 1][nt][k] * inv * w,
                                        acc[i + 1][nt][k + 2] * inv * w};
                    if (d < p.D) store_out<T>(p, to + d, v);
                }
                if (g == 0 && p.lse) p.lse[(at.b * (int64_t)p.Hk + at.h) * p.G + head] = lse_of(m[nt][k], total);
            }
    }
};

// Adds n parts of other blocks (part i at where(i)); eight parts' loads are under way
// together.
template <int DT, int NT, typename Where>
__device__ __forceinline__ void sum_parts(Sum &sum, int n, Where where, int head, int d) {
    constexpr int BATCH = 8;
    for (int i0 = 0; i0 < n; i0 += BATCH) {
        float2 y[BATCH];
        float4 x[BATCH];
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const float *from = where(min(i0 + i, n - 1));
            y[i] = __ldcg(reinterpret_cast<const float2 *>(from + 8 * NT * DT + 2 * head));
            x[i] = __ldcg(reinterpret_cast<const float4 *>(from + part_at<DT>(head, d)));
        }
        float to = sum.top;
#pragma unroll
        for (int i = 0; i < BATCH; ++i) to = fmaxf(to, y[i].x);
        sum.rise(to);
#pragma unroll
        for (int i = 0; i < BATCH; ++i)
            if (i0 + i < n) sum.add(y[i], x[i]);
    }
}

template <int DT, int NT>
__device__ __forceinline__ void put_part(float *part, int head, int d, const Sum &sum) {
    *reinterpret_cast<float4 *>(part + part_at<DT>(head, d)) = sum.o;
    if (d == 0) *reinterpret_cast<float2 *>(part + 8 * NT * DT + 2 * head) = make_float2(sum.top, sum.total);
}

// What a warp leaves of the key heads that it did not have alone.  head: the one it
// ended but did not begin; tail: the one it did not end.
struct Leftover {
    int has_head, has_tail, through;    // through: the tail was not begun here either
    struct Item {
        int b, h, group;
        int n, at;                      // the key head's strips, and its place in the list
    } head, tail;
};

// A key head that another block has a part of too.
struct Shared {
    Leftover::Item item;
    int first, count;                   // blocks first .. first + count - 1; count 0: none
};
static_assert(sizeof(Leftover) <= 72 && 2 * sizeof(Shared) + 72 <= 128, "they fit the room that Shape::NOTES has");

// Counts this block in; true if it is the last of n.  One thread, behind a fence.
__device__ __forceinline__ bool last_of(unsigned *ticket, int n) {
    const bool last = atomicAdd(ticket, 1u) == (unsigned)(n - 1);
    if (last) *ticket = 0;          // as it was found
    return last;
}

// Joins what blocks share, once a block has nothing else to do: its first key head
// may have been begun by another block (kind 0), its last be ended by another
// (kind 1).  The last block of each kJoin neighbours to come here sums their parts
// into the first one's place, the last of those sums the sums.
template <int DT, int NT, typename T>
__device__ __forceinline__ void join(const AttendParams &p, const Shared *shared, int *note) {
    using S = typename Attend<DT, NT, T>::S;
    constexpr int TASKS = S::HEADS * DT / 4, MINE = (TASKS + S::THREADS - 1) / S::THREADS;
    if (threadIdx.x == 0) {
        __threadfence();        // the block's parts, which a barrier has put before this
#pragma unroll
        for (int kind = 0; kind < 2; ++kind) {
            const Shared j = shared[kind];
            bool last = false;
            if (j.count > 0) {
                const int g0 = ((int)blockIdx.x - j.first) / kJoin * kJoin;
                last = last_of(p.tickets + 2 * (j.first + g0) + (g0 == 0 ? 1 : 0), min(kJoin, j.count - g0));
            }
            note[kind] = last;
        }
        __threadfence();
    }
    __syncthreads();
#pragma unroll 1
    for (int kind = 0; kind < 2; ++kind) {
        if (note[kind] == 0) continue;
        const Shared j = shared[kind];
        const int head0 = j.item.group * S::HEADS;
        const int g0 = ((int)blockIdx.x - j.first) / kJoin * kJoin, gn = min(kJoin, j.count - g0);
        const int groups = (j.count + kJoin - 1) / kJoin;
        // block i's part: the first block's is its kind 1
        auto where = [&](int i) { return p.parts + ((int64_t)(j.first + i) * (S::WARPS + 2) + (i == 0 ? 1 : 0)) * S::PART; };
        Sum sum[MINE];
#pragma unroll
        for (int k = 0; k < MINE; ++k) {
            const int i = threadIdx.x + k * S::THREADS, head = i / (DT / 4), d = (i % (DT / 4)) * 4;
            if (i < TASKS) sum_parts<DT, NT>(sum[k], gn, [&](int q) { return where(g0 + q); }, head, d);
        }
        if (groups > 1) {
            __syncthreads();    // every part has been read before the first one is written over
#pragma unroll
            for (int k = 0; k < MINE; ++k) {
                const int i = threadIdx.x + k * S::THREADS, head = i / (DT / 4), d = (i % (DT / 4)) * 4;
                if (i >= TASKS) continue;
                put_part<DT, NT>(where(g0), head, d, sum[k]);
            }
            __syncthreads();
            if (threadIdx.x == 0) {
                __threadfence();
                note[2] = last_of(p.tickets + 2 * gridDim.x + j.first, groups);
                __threadfence();
            }
            __syncthreads();
            if (note[2] == 0) continue;
#pragma unroll
            for (int k = 0; k < MINE; ++k) {
                const int i = threadIdx.x + k * S::THREADS, head = i / (DT / 4), d = (i % (DT / 4)) * 4;
                sum[k] = Sum();
                if (i < TASKS) sum_parts<DT, NT>(sum[k], groups, [&](int q) { return where(q * kJoin); }, head, d);
            }
        }
#pragma unroll
        for (int k = 0; k < MINE; ++k) {
            const int i = threadIdx.x + k * S::THREADS, head = i / (DT / 4), d = (i % (DT / 4)) * 4;
            if (i < TASKS) finish_head<T>(p, j.item.b, j.item.h, head0 + head, d, sum[k].o, sum[k].top, sum[k].total);
        }
    }
}

// The results of sequences without tokens, and complaints about lengths.  A thread
// looks at one sequence of each gridDim.x; `found` has a word for each warp.
template <int THREADS, typename T>
__device__ __forceinline__ void nothing(const AttendParams &p, uint32_t *found) {
    for (int64_t first = blockIdx.x; first < p.B; first += (int64_t)gridDim.x * THREADS) {
        const int64_t own = first + (int64_t)gridDim.x * threadIdx.x;
        bool empty = false;
        if (own < p.B) {
            const int n = p.lens[own];
            if (n < 0 || n > p.width * p.page) record_error(p.err, kErrBadIndex);
            empty = n <= 0 || p.width == 0;
        }
        const uint32_t some = __ballot_sync(0xffffffffu, empty);
        if (!__syncthreads_or(some != 0)) continue;
        if (threadIdx.x % 32 == 0) found[threadIdx.x / 32] = some;
        __syncthreads();
        for (int w = 0; w < THREADS / 32; ++w) {
            for (uint32_t left = found[w]; left != 0; left &= left - 1) {
                const int64_t b = first + (int64_t)gridDim.x * (32 * w + __ffs(left) - 1);
                for (int i = threadIdx.x; i < p.Hk * p.G * p.D; i += THREADS)
                    static_cast<T *>(p.out)[b * p.o_ld + (i / p.D) * p.o_hs + i % p.D] = from_f32<T>(0.0f);
                if (p.lse)
                    for (int i = threadIdx.x; i < p.Hk * p.G; i += THREADS) p.lse[b * p.Hk * p.G + i] = -INFINITY;
            }
        }
        __syncthreads();
    }
}

template <int DT, int NT, typename T>
__global__ void __launch_bounds__((Attend<DT, NT, T>::S::THREADS), 1)
attend_kernel(const __grid_constant__ AttendParams p) {
    using S = typename Attend<DT, NT, T>::S;
    extern __shared__ uint8_t raw[];
    uint8_t *smem = raw + ((128 - (smem_u32(raw) & 127)) & 127);
    Leftover *left = reinterpret_cast<Leftover *>(smem + S::WARPS * (S::STAGES * S::STAGE + S::QUERIES));   // of each warp
    int *sums = reinterpret_cast<int *>(left + S::WARPS);       // strips of each warp's run of sequences
    Shared *shared = reinterpret_cast<Shared *>(sums + S::WARPS);
    int *note = reinterpret_cast<int *>(shared + 2);
    const int tid = threadIdx.x, warp = tid >> 5;
    auto parts = [&](int i) { return p.parts + ((int64_t)blockIdx.x * (S::WARPS + 2) + i) * S::PART; };

    // The list's length, and where this warp's strips begin and end.
    pdl_wait();
    pdl_trigger();
    Locator list;
    int total = 0;
    list.sums = sums;
    list.run = ((p.B + S::WARPS - 1) / S::WARPS + 31) & ~31;
    if (p.B > 32) {
        int count = 0;
        const int b1 = min(p.B, (warp + 1) * list.run);
        for (int b = warp * list.run + (tid & 31); b < b1; b += 32) count += span_of(p, tokens_of(p, b)).strips;
        count *= p.Hk * p.groups;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) count += __shfl_xor_sync(0xffffffffu, count, o);
        if ((tid & 31) == 0) sums[warp] = count;
        __syncthreads();
        for (int w = 0; w < S::WARPS; ++w) total += sums[w];
    }
    list.load(p, 0, 0);
    if (p.B <= 32) total = list.all();
    const Division div(total, S::WARPS * kLeast, Attend<DT, NT, T>::TERMS);
    nothing<S::THREADS, T>(p, reinterpret_cast<uint32_t *>(note));
    if ((int)blockIdx.x >= div.blocks || total == 0) return;
    int *bounds = note, *starts = note + 2;     // of the block, of its warps
    if (warp < 2) {
        const int x = div.start(p, list, blockIdx.x + warp);
        if ((tid & 31) == 0) bounds[warp] = x;
    }
    __syncthreads();
    const int begin = bounds[0], end = bounds[1];
    if (begin >= end) return;

    Attend<DT, NT, T> a(p, smem_u32(smem));
    // This warp's even share of the block's strips, but for a begin that would divide a
    // short key head.
    Cursor cur;
    int at = begin + Shares(end - begin, S::WARPS).begin(warp);
    if (at < end) {
        cur = list.find(p, at);
        const int n = cur.span.strips;
        if (n <= kWhole && cur.strip > 0) {
            const int to = Division::moved(at, cur.strip, n);
            if (to < at) {
                cur.strip = 0;
            } else if (to < end) {
                cur.strip = n - 1;
                cur.step(p);
            }
            at = to;
        }
    }
    if (a.lane == 0) starts[warp] = at;
    __syncthreads();
    int todo = (warp + 1 < S::WARPS ? starts[warp + 1] : end) - at;
    bool has_tail = false;
    if (a.lane == 0) left[warp].has_head = left[warp].has_tail = left[warp].through = 0;
    if (tid < 2) shared[tid].count = 0;
    a.next = cur;
    a.left = todo;
    if (todo > 0) a.look_up();
#pragma unroll 1
    for (int s = 0; s < S::STAGES - 1; ++s) a.load(s);

    int stage = 0, fill = S::STAGES - 1;
    while (todo > 0) {
        // the strips of one key head that are this warp's
        const int strips = cur.span.strips;
        const int n = min(todo, strips - cur.strip);
        a.begin(cur);
        for (int i = 0; i < n; ++i) {
            cp_wait<S::STAGES - 2>();
            __syncwarp();       // every lane's copies have landed, and the stage filled next has been read
            a.load(fill);
            a.consume(stage);
            stage = stage + 1 == S::STAGES ? 0 : stage + 1;
            fill = fill + 1 == S::STAGES ? 0 : fill + 1;
        }
        a.total();
        const bool begun = cur.strip == 0, ended = cur.strip + n == strips;
        if (begun && ended) {
            a.finish(cur);
        } else {
            if (ended) a.store(parts(2 + warp));
            if (a.lane == 0) {
                const Leftover::Item item{cur.b, cur.h, cur.group, strips, at - cur.strip};
                if (ended) {
                    left[warp].has_head = 1;
                    left[warp].head = item;
                } else {
                    left[warp].has_tail = 1;
                    left[warp].through = !begun;
                    left[warp].tail = item;
                }
            }
        }
        at += n;
        todo -= n;
        if (todo > 0) {
            cur.strip += n - 1;
            cur.step(p);
        } else if (!ended) {
            has_tail = true;
        }
    }
    cp_wait<0>();
    __syncwarp();
    auto ring_of = [&](int w) { return reinterpret_cast<float *>(smem + w * (S::STAGES * S::STAGE)); };
    if (has_tail) a.store(ring_of(warp));       // nothing is on its way into the ring any more
    __syncthreads();

    // What warps share.  A run is a key head's parts in consecutive warps: tails, and
    // at its end the head part of the warp that ended it.
    const bool mine = a.lane < S::WARPS;
    const uint32_t heads = __ballot_sync(0xffffffffu, mine && left[a.lane].has_head);
    const uint32_t tails = __ballot_sync(0xffffffffu, mine && left[a.lane].has_tail);
    const uint32_t through = __ballot_sync(0xffffffffu, mine && left[a.lane].through);
    const bool from_before = (heads | through) & 1;      // the block's first key head was begun by another
    const uint32_t begins = tails & ~through;
    const int runs = __popc(begins) + (from_before ? 1 : 0);
    constexpr int TASKS = S::HEADS * DT / 4;
    for (int i = tid; i < runs * TASKS; i += S::THREADS) {
        const int run = i / TASKS, head = i % TASKS / (DT / 4), d = (i % (DT / 4)) * 4;
        uint32_t open = begins;
        for (int k = from_before ? 1 : 0; k < run; ++k) open &= open - 1;
        const bool early = from_before && run == 0;
        const int w0 = early ? 0 : __ffs(open) - 1;
        const uint32_t ends = heads & (early ? ~0u : ~((2u << w0) - 1));     // behind the run's begin
        const int w1 = ends ? __ffs(ends) - 1 : 32 - __clz(tails);           // the tails are those of w0 to w1 - 1
        Sum sum;
        float4 x;
        float2 y;
        if (ends) {
            const float *from = parts(2 + w1);
            y = *reinterpret_cast<const float2 *>(from + S::HEADS * DT + 2 * head);
            x = *reinterpret_cast<const float4 *>(from + part_at<DT>(head, d));
        }
        const uint32_t rings = smem_u32(smem), at_m = 4 * (S::HEADS * DT + 2 * head), at_o = 4 * part_at<DT>(head, d);
#pragma unroll 8
        for (int w = w0; w < w1; ++w) sum.top = fmaxf(sum.top, __uint_as_float(lds4(rings + w * (S::STAGES * S::STAGE) + at_m)));
        if (ends) sum.top = fmaxf(sum.top, y.x);
#pragma unroll 4
        for (int w = w0; w < w1; ++w) {
            const uint32_t from = rings + w * (S::STAGES * S::STAGE);
            const uint2 m = lds8(from + at_m);
            const uint4 o = lds16(from + at_o);
            sum.add(make_float2(__uint_as_float(m.x), __uint_as_float(m.y)),
                    make_float4(__uint_as_float(o.x), __uint_as_float(o.y), __uint_as_float(o.z), __uint_as_float(o.w)));
        }
        if (ends) sum.add(y, x);
        // an early run that its first warp ends is that one head part
        const Leftover::Item &item = early && left[w0].has_head ? left[w0].head : left[w0].tail;
        if (!early && ends) {
            finish_head<T>(p, item.b, item.h, item.group * S::HEADS + head, d, sum.o, sum.top, sum.total);
        } else {
            put_part<DT, NT>(parts(early ? 0 : 1), head, d, sum);
            if (i % TASKS == 0) {
                Shared with{item, 0, 0};
                int last;
                div.blocks_of(item.at, item.n, with.first, last);
                with.count = last - with.first + 1;
                shared[early ? 0 : 1] = with;
            }
        }
    }
    __syncthreads();
    if (shared[0].count == 0 && shared[1].count == 0) return;
    join<DT, NT, T>(p, shared, note);
}

template <int DT, int NT, typename T>
cudaError_t attend_launch(const AttendParams &p, int sms, cudaStream_t stream) {
    using S = typename Attend<DT, NT, T>::S;
    static std::atomic<uint64_t> allowed{0};        // a bit for each device that has been told
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if ((allowed.load(std::memory_order_relaxed) & bit) == 0) {
        e = cudaFuncSetAttribute(attend_kernel<DT, NT, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
        if (e != cudaSuccess) return e;
        allowed.fetch_or(bit, std::memory_order_relaxed);
    }
    return launch_dependent(attend_kernel<DT, NT, T>, sms, S::THREADS, S::SMEM, stream, p);
}

template <int DT>
cudaError_t attend_of_dim(const AttendParams &p, int type, int nt, int sms, cudaStream_t stream) {
    using B = __nv_bfloat16;
    const bool b = type == kTypeBf16;
    if (nt == 1) return b ? attend_launch<DT, 1, B>(p, sms, stream) : attend_launch<DT, 1, float>(p, sms, stream);
    if (b && nt == 2) return attend_launch<DT, 2, B>(p, sms, stream);
    if constexpr (attend_sets(DT, false) >= 2)
        if (!b && nt == 2) return attend_launch<DT, 2, float>(p, sms, stream);
    if constexpr (attend_sets(DT, false) >= 3)
        if (!b && nt == 3) return attend_launch<DT, 3, float>(p, sms, stream);
    if constexpr (attend_sets(DT, true) >= 3)
        if (b && nt == 3) return attend_launch<DT, 3, B>(p, sms, stream);
    if constexpr (attend_sets(DT, true) >= 4)
        if (b && nt == 4) return attend_launch<DT, 4, B>(p, sms, stream);
    return cudaErrorInvalidConfiguration;       // more than attend_sets()
}

}  // namespace

#endif  // __CUDACC__

}  // namespace sgemm_gb300
