// q8.cuh -- shared parts of the 8-bit serving operators: argument structs,
// element types, the exact 8-bit to FP16 expansion, and the block-wide row
// quantisation.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace sgemm_gb300 {

// Element types of the floating operands (the SGEMM_TYPE_* values of the C ABI).
enum : int { kTypeFp32 = 0, kTypeBf16 = 1 };

struct Q8RowsArgs {
    int64_t M, K;
    int type;                          // of x, residual, h, y
    const void *x; int64_t ldx;
    const void *residual; int64_t ldr;  // or nullptr
    const float *weight;               // K floats: RMS norm; nullptr: plain quantisation
    float eps;
    void *h; int64_t ldh;              // or nullptr
    void *y; int64_t ldy;              // or nullptr
    int8_t *q; int64_t ldq;
    float *scale;
    cudaStream_t stream;
    int sm_count;
};

struct Q8LinearArgs {
    int64_t M, N, K;
    const int8_t *X; int64_t ldx;
    const float *xs;
    const int8_t *W; int64_t ldw;
    const float *ws;
    const float *bias; int act;
    void *C; int64_t ldc; int type;    // of C
    cudaStream_t stream;
    unsigned *err;
    uint64_t wait_ns;
    int sm_count;
    EncodeTiledFn encode;
};

struct Q8MoeArgs {
    int T, E, top_k, H, I;
    int type;                          // of x and out
    const void *x; int64_t ldx;
    const float *router; int64_t ldr;
    const int8_t *w_up; int64_t ldu; const float *s_up;
    const int8_t *w_down; int64_t ldd; const float *s_down;
    int renormalize;
    void *out; int64_t ldo;
    int *ids; float *gates;            // or nullptr
    cudaStream_t stream;
    unsigned *err;
    uint64_t wait_ns;
    int sm_count;
    EncodeTiledFn encode;
};

cudaError_t launch_q8_rows(const Q8RowsArgs &a);
cudaError_t launch_q8_stream(const Q8LinearArgs &a);
// The tensor-core form, for more tokens than the streaming kernel is for.
bool q8_mma_can_run(const Q8LinearArgs &a);
size_t q8_mma_workspace_bytes(const Q8LinearArgs &a);
cudaError_t launch_q8_mma(const Q8LinearArgs &a, void *workspace);
cudaError_t launch_q8_moe(const Q8MoeArgs &a, void *workspace);
size_t q8_moe_workspace_bytes(int T, int E, int top_k, int H, int I);

// Limits of the expert layer (its routing tables live in shared memory).
constexpr int kMoeMaxTokens = 64, kMoeMaxTopK = 16, kMoeMaxExperts = 512;
// Longest dot product whose 8-bit products cannot overflow a 32-bit sum.
constexpr int64_t kQ8MaxK = 131071;

// Groups of `per` among n > 0 rows (as (n - 1) / per + 1, the ring kernel for 16 tokens
// compiled to 18.0 us instead of 17.8), and whether the 32 rows from `first` are all below
// n, for every n an int holds.
constexpr int groups_of(int n, int per) { return (int)(((unsigned)n + (unsigned)per - 1u) / (unsigned)per); }
constexpr bool all_32_below(int first, int n) { return first <= n - 32; }
static_assert(groups_of(1, 64) == 1 && groups_of(64, 64) == 1 && groups_of(65, 64) == 2, "groups");
static_assert(groups_of(INT32_MAX, 16) == 1 << 27 && groups_of(INT32_MAX, 64) == 1 << 25, "groups of the most rows");
static_assert(all_32_below(0, 32) && !all_32_below(0, 31) && !all_32_below(INT32_MAX - 31, INT32_MAX) &&
              all_32_below(INT32_MAX - 63, INT32_MAX), "32 rows at the end of the most");

#ifdef __CUDACC__

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// V consecutive elements as floats, through 16-byte (or V-element) accesses.
template <typename T, int V>
__device__ __forceinline__ void load_vec(const T *p, float (&v)[V]) {
    if constexpr (V == 1) {
        v[0] = to_f32<T>(*p);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
            const float4 f = *reinterpret_cast<const float4 *>(p + 4 * i);
            v[4 * i] = f.x; v[4 * i + 1] = f.y; v[4 * i + 2] = f.z; v[4 * i + 3] = f.w;
        }
    } else {
        uint32_t w[V / 2];
        if constexpr (V == 8) {
            const uint4 u = *reinterpret_cast<const uint4 *>(p);
            w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
        } else {
            const uint2 u = *reinterpret_cast<const uint2 *>(p);
            w[0] = u.x; w[1] = u.y;
        }
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {   // a bf16 is the upper half of its float
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
}

template <typename T, int V>
__device__ __forceinline__ void store_vec(T *p, const float (&v)[V]) {
    if constexpr (V == 1) {
        *p = from_f32<T>(v[0]);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < V / 4; ++i)
            *reinterpret_cast<float4 *>(p + 4 * i) = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    } else {
        uint32_t w[V / 2];
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&b);
        }
        if constexpr (V == 8) *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        else *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    }
}

// How one row is quantised once its largest magnitude is known.  The maximum
// is taken on the bit patterns of |p| as unsigned numbers, which order like
// the values and put every NaN above infinity, so a row holding a NaN or an
// infinity is seen as such: it gets scale NaN and q = 0.  A row of zeros gets
// scale 0 and q = 0.  A row whose maximum is below 2^-100 is lifted by 2^100
// (exactly) first, so that 127/max stays finite.
struct RowQuant {
    float pre, inv;    // q = rint((p * pre) * inv)
    float step, unpre; // max/127 = step * unpre: p is about q times that
    __device__ __forceinline__ explicit RowQuant(uint32_t max_bits) {
        const float m = __uint_as_float(max_bits);
        if (max_bits >= 0x7f800000u) {
            pre = 0.0f; inv = 0.0f; step = __uint_as_float(0x7fc00000u); unpre = 1.0f;
        } else if (max_bits == 0u) {
            pre = 0.0f; inv = 0.0f; step = 0.0f; unpre = 1.0f;
        } else {
            const bool tiny = m < 7.8886090522101181e-31f;          // 2^-100
            pre = tiny ? 1.2676506002282294e30f : 1.0f;             // 2^100
            unpre = tiny ? 7.8886090522101181e-31f : 1.0f;
            inv = __fdiv_rn(127.0f, m * pre);
            step = __fdiv_rn(m * pre, 127.0f);
        }
    }
    // Whole numbers in [-127, 127]; NaN (only in rows marked so) becomes 0.
    __device__ __forceinline__ int operator()(float p) const {
        return __float2int_rn(__fmul_rn(__fmul_rn(p, pre), inv));
    }
};

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

__device__ __forceinline__ uint32_t pack4(int a, int b, int c, int d) {
    return (uint32_t)(a & 0xff) | ((uint32_t)(b & 0xff) << 8) | ((uint32_t)(c & 0xff) << 16) |
           ((uint32_t)d << 24);
}

// rint(x) in the low byte, for |x| < 2^22: adding 1.5 * 2^23 leaves the whole
// number, rounded to nearest even, in the last bits of the mantissa.  (Two
// instructions at full rate less than a conversion at a quarter of it.)
__device__ __forceinline__ uint32_t rint_byte(float x) { return __float_as_uint(__fadd_rn(x, 12582912.0f)); }

__device__ __forceinline__ uint32_t low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// V values (1, 4 or 8) as 8-bit whole numbers.
template <int V>
__device__ __forceinline__ void store_q(int8_t *p, const RowQuant &rq, const float (&v)[V]) {
    if constexpr (V == 1) {
        *p = (int8_t)rq(v[0]);
    } else {
        uint32_t w[V / 4];
        if (rq.pre == 1.0f) {          // the same for the whole row
#pragma unroll
            for (int i = 0; i < V / 4; ++i)
                w[i] = low_bytes(rint_byte(__fmul_rn(v[4 * i], rq.inv)), rint_byte(__fmul_rn(v[4 * i + 1], rq.inv)),
                                 rint_byte(__fmul_rn(v[4 * i + 2], rq.inv)), rint_byte(__fmul_rn(v[4 * i + 3], rq.inv)));
        } else {                       // zeros, NaN, or numbers to be lifted
#pragma unroll
            for (int i = 0; i < V / 4; ++i)
                w[i] = pack4(rq(v[4 * i]), rq(v[4 * i + 1]), rq(v[4 * i + 2]), rq(v[4 * i + 3]));
        }
        if constexpr (V == 4) *reinterpret_cast<uint32_t *>(p) = w[0];
        else *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    }
}

// Largest value and sum over the block (any number of whole warps); every
// thread gets both.  `red` holds 64 words.
__device__ __forceinline__ void block_max_sum(uint32_t &mx, float &sum, uint32_t *red) {
    mx = __reduce_max_sync(0xffffffffu, mx);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = (int)(blockDim.x >> 5);
    __syncthreads();   // earlier readers of `red` are done
    if (lane == 0) {
        red[warp] = mx;
        red[32 + warp] = __float_as_uint(sum);
    }
    __syncthreads();
    mx = __reduce_max_sync(0xffffffffu, lane < nw ? red[lane] : 0u);
    float s = lane < nw ? __uint_as_float(red[32 + lane]) : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    sum = s;
}

// Four 8-bit whole numbers as four FP16 values, exactly: 0x6400 | u is
// 1024 + u, and u = b + 128 after flipping the sign bit, so subtracting 1152
// gives b.  lo: bytes 0 and 1, hi: bytes 2 and 3.
__device__ __forceinline__ void q8_to_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t l = __byte_perm(u, 0x64646464u, 0x4140);
    const uint32_t h = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 bias = __half2half2(__ushort_as_half((unsigned short)0x6480));   // 1152
    const __half2 rl = __hsub2(*reinterpret_cast<const __half2 *>(&l), bias);
    const __half2 rh = __hsub2(*reinterpret_cast<const __half2 *>(&h), bias);
    lo = *reinterpret_cast<const uint32_t *>(&rl);
    hi = *reinterpret_cast<const uint32_t *>(&rh);
}

#endif  // __CUDACC__

}  // namespace sgemm_gb300
