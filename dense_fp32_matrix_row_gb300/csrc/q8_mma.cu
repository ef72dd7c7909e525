// q8_mma.cu -- 8-bit linear product on the tcgen05 tensor cores, exactly:
//
//     C[m][n] = act(xs[m] * ws[n] * sum_k X[m][k] * W[n][k] + bias[n])
//
// sm_103a has no fast 8-bit integer MMA (and no tcgen05 kind::i8).  But an
// 8-bit whole number is exact in FP16, a product of two is at most 2^14, and a
// sum of 1024 of them at most 2^24: the FP16 tensor cores with FP32
// accumulators give the integer sum exactly, as long as the accumulator is
// emptied every 1024 k.  The chunk sums are added in FP32 registers, exact
// while they stay within 2^24 and rounded once per chunk beyond.
//
// Roles are swapped against a usual product: the 128 lanes of the accumulator
// are rows of W (output channels), its columns are tokens, so a few tokens
// waste nothing and C's rows are stored 32 channels at a time.
//
//   W   travels and rests in 8 bits.  TMA brings 128 k of 128 rows into a
//       shared-memory ring; eight converter warps, four to a stage, read a row per thread, expand
//       it to FP16 in registers and store it to tensor memory, from where the
//       MMA takes its A operand.  The 16-bit form of W never touches shared
//       memory, whose bandwidth is what bounds such a kernel (16 KB written and
//       read per stage and SM for W, where 16-bit tiles would move 32 and 32).
//   X   is expanded to FP16 once, by q8_prepare_kernel (2 bytes of L2 traffic per
//       element), and comes in by TMA as the B operand, 128 k per stage.
//   MMA one thread issues eight tcgen05.mma kind::f16 per stage.
//   Eight more warps empty the accumulator, add the chunks and store.  The
//       warpgroups trade registers (setmaxnreg), so that each of these threads
//       can hold its 128 sums.
//
// PAIR: two SMs share a tile of 256 W rows x NT tokens (cta_group::2), each
// with its own 128 rows of W and half of the tokens' X.
//
// Emptying an accumulator must not stop the MMAs.  Up to 128 tokens there are
// two accumulators, used in turn.  At 256 tokens one fills tensor memory
// beside the A stages; it is used as two halves of 128 columns, and the MMAs
// of two stages at a time are issued for one half, then for the other, so
// that a half is emptied while the other is computed (8192 x 14336 x 4096:
// 600 us when each chunk stopped for the whole accumulator).
//
// When the tiles do not fill the GPU, K is divided into `ks` parts per tile;
// the parts' sums go to the workspace and the last warp to arrive adds them in
// part order.
//
// Every wait is bounded; on a time-out the roles record it and wind down.  Whichever
// role gave up, the block ends (and gives tensor memory back) only when its copies
// have landed and its MMAs are done.
//
// Measured: 8192 x 14336 x 4096 492 us in a burst (1950 TFLOP/s of FP16 MMAs, bound
// by the tensor cores), 534 sustained, with 2 us for X's expansion; 2048 x 4096 x
// 4096 48 us (1420); 512 x 4096 x 4096 20 us (860: tiles for half the GPU, K divided
// in two); 128 x 14336 x 4096 22.4 us (W alone is 9 us of memory time: one tile of
// 128 tokens for 112 of the 152 SMs, and the expansion is a launch of its own).
#include <cuda_fp16.h>

#include <algorithm>

#include "q8_stream.cuh"
#include "tcgen05.cuh"

namespace sgemm_gb300 {
namespace {

// Warpgroups: two that empty the accumulator, two of converters (stages of
// either parity), and one whose first three warps load W, issue the MMAs and
// load X.
constexpr int EPI_WARPS = 8, CONV_WARPS = 8;
constexpr int W_WARP = EPI_WARPS + CONV_WARPS, MMA_WARP = W_WARP + 1, X_WARP = W_WARP + 2;
constexpr int THREADS = (EPI_WARPS + CONV_WARPS + 4) * 32;
// Registers per thread: at launch, and what each warpgroup takes.  The shares
// have to add up to no more than the launch's, or setmaxnreg.inc would wait.
constexpr int REGS = 96, EPI_REGS = 152, CONV_REGS = 64, OTHER_REGS = 48;
static_assert(EPI_REGS * EPI_WARPS + CONV_REGS * CONV_WARPS + OTHER_REGS * 4 <= REGS * (THREADS / 32),
              "register shares");
constexpr int KT = 128;                       // k per stage
constexpr int CHUNK = 8;                      // stages per accumulation chunk: 1024 k
constexpr uint32_t W_STAGE = 128 * KT;        // bytes
constexpr uint64_t DRAIN_NS = 1000000000ull;

template <int NT_, bool PAIR_>
struct Cfg {
    static constexpr int NT = NT_;                         // tokens per tile
    static constexpr bool PAIR = PAIR_;
    static constexpr int NL = PAIR ? NT / 2 : NT;          // tokens staged by one SM
    static constexpr int ROWS = PAIR ? 256 : 128;          // W rows per tile
    static constexpr bool HALVES = NT == 256;              // one accumulator, emptied by halves
    static constexpr int DB = HALVES ? 1 : 2;              // accumulators
    static constexpr int NM = HALVES ? NT / 2 : NT;        // columns of an MMA
    static constexpr int R = PAIR ? 2 : 1;                 // SMs per tile
    static constexpr int ST = 4;                           // X and A stages
    static constexpr int WST = NT <= 64 ? 8 : 4;           // W stages
    static constexpr uint32_t X_HALF = NL * 128;           // bytes: 64 FP16 per token
    static constexpr uint32_t X_STAGE = 2 * X_HALF;
    static constexpr uint32_t A_COL = DB * NT;             // tensor-memory column of A stage 0
    static constexpr int COLS = NT / 2;                    // columns per epilogue thread
    static constexpr size_t SMEM = 1024 + (size_t)ST * X_STAGE + (size_t)WST * W_STAGE + 512;
    // kind::f16, FP16 operands (format 0), FP32 accumulator, both K-major
    static constexpr uint32_t IDESC = (1u << 4) | ((uint32_t)(NM >> 3) << 17) | ((uint32_t)(ROWS >> 4) << 24);
    static_assert(A_COL + ST * (KT / 2) <= 512, "tensor memory");
    static_assert(SMEM <= 227 * 1024, "shared memory per block");
    static_assert(X_HALF % 1024 == 0 && W_STAGE % 1024 == 0, "stages keep 1024-byte alignment");
    static_assert(COLS % 16 == 0, "the drain reads 16 columns at a time");
};

// The division of the product into units: tile (W rows, tokens) and part of K.
struct Plan {
    int nt, mt;      // tiles along W rows and along tokens
    int ks, per;     // parts of K per tile, stages per part
    int stages;
    __host__ __device__ int units() const { return nt * mt * ks; }
};

constexpr int RASTER = 8;   // W tiles walked together over the tokens (L2 reuse)

__device__ __forceinline__ void plan_unit(const Plan &p, int u, int &tn, int &tm, int &s0, int &s1) {
    const int tile = u / p.ks, part = u - tile * p.ks;
    const int per_group = RASTER * p.mt;
    const int first = (tile / per_group) * RASTER;
    const int gsz = min(RASTER, p.nt - first);
    tn = first + (tile % per_group) % gsz;
    tm = (tile % per_group) / gsz;
    s0 = part * p.per;
    s1 = min(s0 + p.per, p.stages);
}

template <bool PAIR>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    if constexpr (PAIR)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
            "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
            "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
}

__device__ __forceinline__ void tc_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
        "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
        "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tc_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Arrive on the barrier at offset `bar` of CTA `cta` of the cluster.  Relaxed:
// what it hands over is tensor memory alone, which the completed tcgen05
// operations and tcgen05.fence before it order.  (A release at cluster scope
// waits about 1500 cycles here, once per stage and warp: the 8192 x 14336 x
// 4096 product took 1209 us with it.)
__device__ __forceinline__ void arrive_relaxed(uint32_t bar, uint32_t cta) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr(bar, cta))
                 : "memory");
}

// Adds to a word in shared memory of CTA `cta` of the cluster.
__device__ __forceinline__ void add_cta(uint32_t addr, uint32_t cta, uint32_t v) {
    asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(cluster_addr(addr, cta)), "r"(v)
                 : "memory");
}

// Takes `bytes` off what the barrier's phase still waits for.
__device__ __forceinline__ void mbar_complete_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

// One stage of X: 128 k of NL tokens as two 64-wide halves, through a map whose
// dimensions are (k % 64, token, k / 64).
template <bool PAIR>
__device__ __forceinline__ void tma_load_x(uint32_t dst, const CUtensorMap *map, uint32_t bar, int token, int k64) {
    if constexpr (PAIR)
        asm volatile(
            "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(0), "r"(token), "r"(k64)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(0), "r"(token), "r"(k64)
            : "memory");
}

template <int N, bool UP>
__device__ __forceinline__ void set_registers() {
    if constexpr (UP) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// The epilogue's activation.  SiLU and GELU are v times a logistic function (GELU:
// of 2 sqrt(2/pi) (v + 0.044715 v^3), the same function as the tanh form) with the
// short quotient, good to 2 units in the last place (0 for results below 1e-36),
// and for a bf16 result the short exponential, good to about 1e-5 where the result
// keeps 4e-3.  tanhf, expf and the exact quotient cost some 40 instructions for each
// of a thread's 128 values, more than the MMAs give it time for: 2048 x 14336 x 4096
// took 188 us with SiLU and an FP32 result, 150 with GELU and bf16, and takes 125
// without an activation.
template <int ACT, typename OutT>
__device__ __forceinline__ float finish_value(float v) {
    if constexpr (ACT == kActSilu || ACT == kActGelu) {
        const float x = ACT == kActSilu ? -v : -1.5957691216057308f * fmaf(0.044715f * v, v * v, v);
        return __fdividef(v, 1.0f + (sizeof(OutT) == 2 ? __expf(x) : expf(x)));
    } else {
        return ACT == kActRelu && v < 0.0f ? 0.0f : v;     // ReLU keeps NaN
    }
}

template <typename C, typename OutT>
__global__ void __launch_bounds__(THREADS, 1)
q8_mma_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, int M, int N,
              Plan plan, const float *__restrict__ xs, const float *__restrict__ ws, Epilogue ep,
              OutT *__restrict__ out, int64_t ldc, float *part, uint32_t *counters, unsigned *err,
              uint64_t wait_ns, int w_copied) {
    constexpr bool PAIR = C::PAIR;
    constexpr int ST = C::ST, WST = C::WST, NT = C::NT, COLS = C::COLS;
    extern __shared__ unsigned char smem_raw[];
    const uintptr_t base = (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023);
    unsigned char *xring = reinterpret_cast<unsigned char *>(base);
    unsigned char *wring = xring + (size_t)ST * C::X_STAGE;
    uint64_t *wfull = reinterpret_cast<uint64_t *>(wring + (size_t)WST * W_STAGE);
    uint64_t *wempty = wfull + WST;
    uint64_t *xfull = wempty + WST;     // even SM of a pair: both SMs' bytes
    uint64_t *afull = xfull + ST;       // even SM of a pair: both SMs' converters
    uint64_t *empty = afull + ST;       // the MMAs that read X and A stage s are done
    uint64_t *dfull = empty + ST;       // [2] accumulator holds a finished chunk
    uint64_t *dempty = dfull + 2;       // [2] accumulator has been read
    uint64_t *drainbar = dempty + 2;
    uint64_t *xdone = drainbar + 1;     // even SM of a pair: the odd one has issued its last X
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(xdone + 1);
    // Even SM of a pair: stages of X the odd one issued.  (In the dynamic array, as the words
    // above, it made the 256-token kernel spill 70 registers instead of 2.)
    __shared__ uint32_t odd_stages;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t rank = 0;
    if constexpr (PAIR) asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    const bool lead = rank == 0;
    const int worker = PAIR ? (int)(blockIdx.x >> 1) : (int)blockIdx.x;
    const int workers = PAIR ? (int)(gridDim.x >> 1) : (int)gridDim.x;
    const int units = plan.units();

    if (threadIdx.x == 0) {
        for (int s = 0; s < WST; ++s) {
            mbar_init(smem_u32(&wfull[s]), 1);
            mbar_init(smem_u32(&wempty[s]), CONV_WARPS / 2);
        }
        for (int s = 0; s < ST; ++s) {
            mbar_init(smem_u32(&xfull[s]), 1);
            mbar_init(smem_u32(&afull[s]), C::R * CONV_WARPS / 2);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&dfull[b]), 1);
            mbar_init(smem_u32(&dempty[b]), C::R * EPI_WARPS / (C::HALVES ? 2 : 1));
        }
        mbar_init(smem_u32(drainbar), 1);
        mbar_init(smem_u32(xdone), 1);
        mbar_fence_init();
        odd_stages = 0u;
    }
    if (warp == 0) {
        __syncwarp();
        if constexpr (PAIR) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                             smem_u32(tmem_slot)), "r"(512u) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                             smem_u32(tmem_slot)), "r"(512u) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        }
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (PAIR) cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(tmem_slot);

    if (warp < EPI_WARPS) {
        // Epilogue warp w: tensor-memory lanes 32 * (w % 4) .. + 31 (a W row
        // each), accumulator columns (w / 4) * COLS .. + COLS (tokens).
        set_registers<EPI_REGS, true>();
        const int half = warp >> 2, lane_base = (warp & 3) * 32;
        const int row = lane_base + lane;
        const uint32_t lane_addr = tmem + ((uint32_t)lane_base << 16);
        bool ok = true;
        uint32_t gc = 0;
        for (int u = worker; u < units && ok; u += workers) {
            int tn, tm, s0, s1;
            plan_unit(plan, u, tn, tm, s0, s1);
            float acc[COLS];
#pragma unroll
            for (int j = 0; j < COLS; ++j) acc[j] = 0.0f;
            for (int c0 = s0; c0 < s1; c0 += CHUNK, ++gc) {
                const int b = C::HALVES ? half : (int)(gc % C::DB);
                if (!warp_wait(smem_u32(&dfull[b]), (gc / C::DB) & 1, wait_ns)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d = lane_addr + (uint32_t)((C::HALVES ? 0 : b * NT) + half * COLS);
#pragma unroll
                for (int piece = 0; piece < COLS / 16; ++piece) {
                    float v[16];
                    __syncwarp();
                    tc_ld16(d + (uint32_t)(piece * 16), v);
#pragma unroll
                    for (int i = 0; i < 16; ++i) acc[piece * 16 + i] += v[i];
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (PAIR) arrive_relaxed(smem_u32(&dempty[b]), 0);
                    else mbar_arrive(smem_u32(&dempty[b]));
                }
            }
            if (!ok) break;
            pdl_wait();   // returns at once: X's stages could not have come before
            if (NT <= 128 && plan.ks > 1) {
                // this unit's sums to the workspace; the last part's warp adds them all
                const int tile = u / plan.ks, own = u - tile * plan.ks;
                float *slot = part + (((int64_t)u * C::R + rank) * NT + half * COLS) * 128 + row;
#pragma unroll
                for (int j = 0; j < COLS; ++j) __stcg(slot + j * 128, acc[j]);
                __threadfence();
                __syncwarp();
                uint32_t arrived = 0;
                if (lane == 0) arrived = atomicAdd(counters + (tile * C::R + (int)rank) * EPI_WARPS + warp, 1u);
                arrived = __shfl_sync(0xffffffffu, arrived, 0);
                if (arrived != (uint32_t)(plan.ks - 1)) continue;
                __syncwarp();      // lane 0's count before the other lanes' fences
                __threadfence();
                float sum[COLS];
#pragma unroll
                for (int j = 0; j < COLS; ++j) sum[j] = 0.0f;
                for (int p = 0; p < plan.ks; ++p) {
                    const float *o = slot + (int64_t)(p - own) * C::R * NT * 128;
#pragma unroll
                    for (int j = 0; j < COLS; ++j) sum[j] += __ldcg(o + j * 128);
                }
#pragma unroll
                for (int j = 0; j < COLS; ++j) acc[j] = sum[j];
            }
            // Column j of this thread's sums is token m0 + at(j), the thread channel
            // n: a warp stores 32 channels of one token at a time.  (A half of the
            // accumulator holds 64 tokens of each SM's 128.)
            constexpr auto at = [](int j) { return C::HALVES ? j + (j >= 64 ? 64 : 0) : j; };
            const int n = tn * C::ROWS + 128 * (int)rank + row;
            const int m0 = tm * NT + half * (C::HALVES ? 64 : COLS);
            const float wsn = __ldg(ws + min(n, N - 1));
            const float bias = ep.bias != nullptr ? __ldg(ep.bias + min(n, N - 1)) : 0.0f;
            float xv[(COLS + 31) / 32];       // lane l holds the scale of column 32 i + l
#pragma unroll
            for (int i = 0; i < (COLS + 31) / 32; ++i) xv[i] = __ldg(xs + min(m0 + at(32 * i) + lane, M - 1));
            // In place first, then the stores: next to the sums there are few
            // registers, and one pass over both ran one dependent chain per column
            // (110 cycles each, longer than a chunk's MMAs).
            auto finish = [&](auto act) {
#pragma unroll
                for (int j = 0; j < COLS; ++j)
                    acc[j] = act(fmaf(acc[j] * __shfl_sync(0xffffffffu, xv[j / 32], j % 32), wsn, bias));
            };
            switch (ep.act) {
                case kActRelu: finish([](float v) { return finish_value<kActRelu, OutT>(v); }); break;
                case kActGelu: finish([](float v) { return finish_value<kActGelu, OutT>(v); }); break;
                case kActSilu: finish([](float v) { return finish_value<kActSilu, OutT>(v); }); break;
                default: finish([](float v) { return v; });
            }
            OutT *o = out + (int64_t)m0 * ldc + n;
            if (all_32_below(n - lane, N) && m0 + at(COLS - 1) < M) {
#pragma unroll
                for (int j = 0; j < COLS; ++j) {
                    *o = from_f32<OutT>(acc[j]);
                    if (j + 1 < COLS) o += ldc * (at(j + 1) - at(j));
                }
            } else {
#pragma unroll
                for (int j = 0; j < COLS; ++j)
                    if (n < N && m0 + at(j) < M) o[(int64_t)at(j) * ldc] = from_f32<OutT>(acc[j]);
            }
        }
        if (!ok && lane == 0) record_error(err, kErrWaitTimeout);
    } else if (warp < W_WARP) {
        // Converter warp w: W rows (tensor-memory lanes) 32 * (w % 4) .. + 31 of
        // the stages of parity (w / 4) % 2.
        set_registers<CONV_REGS, false>();
        const int lane_base = (warp & 3) * 32;
        const int row = lane_base + lane;
        const uint32_t a_addr = tmem + ((uint32_t)lane_base << 16) + C::A_COL;
        const uint32_t swz = (uint32_t)(row & 7);   // the 128-byte swizzle of this row
        uint32_t total = 0;
        for (int u = worker; u < units; u += workers) {
            int tn, tm, s0, s1;
            plan_unit(plan, u, tn, tm, s0, s1);
            total += (uint32_t)(s1 - s0);
        }
        bool ok = true;
        for (uint32_t g = (uint32_t)(warp >> 2) & 1; g < total; g += 2) {
            const int w = (int)(g % WST), s = (int)(g % ST);
            if (!warp_wait(smem_u32(&wfull[w]), (g / WST) & 1, wait_ns)) {
                ok = false;
                break;
            }
            const uint32_t src = smem_u32(wring + (size_t)w * W_STAGE) + (uint32_t)row * 128;
            uint4 q[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) q[c] = lds128(src + (((uint32_t)c ^ swz) << 4));
            if (g >= (uint32_t)ST) {
                if (!warp_wait(smem_u32(&empty[s]), (g / ST - 1) & 1, wait_ns)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {      // 64 k at a time
                uint32_t r[32];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    q8_to_f16(q[c].x, r[8 * c], r[8 * c + 1]);
                    q8_to_f16(q[c].y, r[8 * c + 2], r[8 * c + 3]);
                    q8_to_f16(q[c].z, r[8 * c + 4], r[8 * c + 5]);
                    q8_to_f16(q[c].w, r[8 * c + 6], r[8 * c + 7]);
                }
                if (h == 0) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) q[c] = lds128(src + (((uint32_t)(c + 4) ^ swz) << 4));
                }
                tc_st32(a_addr + (uint32_t)(s * (KT / 2) + 32 * h), r);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&wempty[w]));
            tc_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (PAIR) arrive_relaxed(smem_u32(&afull[s]), 0);
                else mbar_arrive(smem_u32(&afull[s]));
            }
        }
        if (!ok && lane == 0) record_error(err, kErrWaitTimeout);
    } else {
        set_registers<OTHER_REGS, false>();
        if (warp == W_WARP || warp == X_WARP) {
            // One warp fills each ring.  The caller's W may be read before the
            // preceding kernel (q8_prepare_kernel) has finished: that kernel
            // itself waited for all earlier work.
            const bool is_w = warp == W_WARP;
            const int depth = is_w ? WST : ST;
            uint64_t *freed = is_w ? wempty : empty;
            if (lane == 0) tma_prefetch_desc(is_w ? &tmW : &tmX);
            if (!is_w || w_copied) {
                pdl_wait();
                asm volatile("fence.proxy.async;" ::: "memory");
            }
            bool ok = true;
            uint32_t g = 0;
            for (int u = worker; u < units && ok; u += workers) {
                int tn, tm, s0, s1;
                plan_unit(plan, u, tn, tm, s0, s1);
                for (int k = s0; k < s1; ++k, ++g) {
                    const int s = (int)(g % (uint32_t)depth);
                    if (g >= (uint32_t)depth &&
                        !warp_wait(smem_u32(&freed[s]), (g / (uint32_t)depth - 1) & 1, wait_ns)) {
                        ok = false;
                        break;
                    }
                    if (elect_one()) {
                        if (is_w) {
                            const uint32_t bar = smem_u32(&wfull[s]);
                            mbar_arrive_expect_tx(bar, W_STAGE);
                            tma_load_2d(smem_u32(wring + (size_t)s * W_STAGE), &tmW, bar, k * KT,
                                        tn * C::ROWS + 128 * (int)rank);
                        } else {
                            const uint32_t bar = smem_u32(&xfull[s]);
                            if (lead) mbar_arrive_expect_tx(bar, (PAIR ? 2 : 1) * C::X_STAGE);
                            tma_load_x<PAIR>(smem_u32(xring + (size_t)s * C::X_STAGE), &tmX,
                                             PAIR ? cluster_addr(bar, 0) : bar, tm * NT + C::NL * (int)rank, 2 * k);
                        }
                    }
                    __syncwarp();
                }
            }
            // The copies have to land before the block ends, whichever role gave up; with no
            // time-out the MMAs have waited, or are about to wait, for all of them.
            if (lane == 0) {
                if (!ok) record_error(err, kErrWaitTimeout);
                uint32_t other = g;     // stages of X that the other SM of a pair issued
                bool told = true;
                if (PAIR && !is_w) {
                    if (lead) {
                        told = mbar_wait_cluster(smem_u32(xdone), 0, wait_ns + DRAIN_NS);
                        other = *const_cast<volatile uint32_t *>(&odd_stages);
                    } else {
                        add_cta(smem_u32(&odd_stages), 0, g);
                        mbar_arrive_cta(smem_u32(xdone), 0);
                    }
                }
                if (is_w || lead) {
                    // Both SMs' X completes on the even SM's barriers.  What one SM issued and
                    // the other did not is made up for.  (A stage is issued after the MMAs of
                    // the stage `depth` before it: only the last `depth` can be open.)
                    const uint32_t most = told && other > g ? other : g;
                    for (uint32_t q = most > (uint32_t)depth ? most - (uint32_t)depth : 0; q < most; ++q) {
                        const uint32_t bar = smem_u32(&(is_w ? wfull : xfull)[q % (uint32_t)depth]);
                        if (told && q >= g) mbar_arrive_expect_tx(bar, C::X_STAGE);
                        else if (told && q >= other) mbar_complete_tx(bar, C::X_STAGE);
                        mbar_wait(bar, (q / (uint32_t)depth) & 1, DRAIN_NS);
                    }
                }
            }
        } else if (warp == MMA_WARP && lead) {
            // The whole warp walks the stages and one elected lane issues: the
            // operands then stay in uniform registers (23 cycles per MMA of 32
            // tokens, against 54 from a loop that a single lane runs).
            auto wait = [&](uint64_t *bar, uint32_t parity) {
                const bool done = PAIR ? mbar_wait_cluster(smem_u32(bar), parity, wait_ns)
                                       : mbar_wait(smem_u32(bar), parity, wait_ns);
                return __all_sync(0xffffffffu, done) != 0;
            };
            auto commit = [&](uint64_t *bar) {
                if constexpr (PAIR) tc2_commit_both(smem_u32(bar));
                else tc_commit(smem_u32(bar));
            };
            const uint64_t xdesc = smem_desc<128>(smem_u32(xring));   // addresses count in 16 bytes
            bool ok = true, issued = false;
            uint32_t g = 0, gc = 0;
            for (int u = worker; u < units && ok; u += workers) {
                int tn, tm, s0, s1;
                plan_unit(plan, u, tn, tm, s0, s1);
                for (int c0 = s0; c0 < s1 && ok; c0 += CHUNK, ++gc) {
                    const int c1 = min(c0 + CHUNK, s1);
                    // the accumulator (or half) b is free for this chunk
                    auto acquire = [&](int b) {
                        if (gc >= (uint32_t)C::DB && !wait(&dempty[b], (gc / C::DB - 1) & 1)) ok = false;
                        tc_fence_after();
                        return ok;
                    };
                    auto staged = [&](uint32_t at) {   // X and A of stage `at` are there
                        const uint32_t par = (at / ST) & 1;
                        if (!wait(&xfull[at % ST], par) || !wait(&afull[at % ST], par)) ok = false;
                        tc_fence_after();
                        return ok;
                    };
                    // the eight MMAs of stage `at` into the accumulator columns at d
                    auto issue = [&](uint32_t d, uint32_t at, uint32_t rows, bool first) {
                        const uint32_t s = at % ST;
                        const uint32_t a = tmem + C::A_COL + s * (KT / 2);
                        const uint64_t x = xdesc + (uint64_t)(s * (C::X_STAGE >> 4) + rows * 8);
#pragma unroll
                        for (int kk = 0; kk < KT / 16; ++kk)
                            mma_ts<PAIR>(d, a + kk * 8, x + (kk >> 2) * (C::X_HALF >> 4) + (kk & 3) * 2, C::IDESC,
                                         (!first || kk != 0) ? 1u : 0u);
                    };
                    if constexpr (C::HALVES) {
                        for (int k = c0; k < c1; k += 2) {
                            const int two = min(2, c1 - k);
                            if (!staged(g) || (two > 1 && !staged(g + 1))) break;
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                if (k == c0 && !acquire(h)) break;
                                if (elect_one()) {
                                    issue(tmem + (uint32_t)(h * C::NM), g, (uint32_t)h * 64, k == c0);
                                    if (h == 1) commit(&empty[g % ST]);
                                    if (two > 1) {
                                        issue(tmem + (uint32_t)(h * C::NM), g + 1, (uint32_t)h * 64, false);
                                        if (h == 1) commit(&empty[(g + 1) % ST]);
                                    }
                                    if (k + 2 >= c1) commit(&dfull[h]);
                                }
                                __syncwarp();
                                issued = true;
                            }
                            if (!ok) break;
                            g += (uint32_t)two;
                        }
                    } else {
                        const int b = (int)(gc % C::DB);
                        if (!acquire(b)) break;
                        for (int k = c0; k < c1; ++k, ++g) {
                            if (!staged(g)) break;
                            if (elect_one()) {
                                issue(tmem + (uint32_t)(b * NT), g, 0u, k == c0);
                                commit(&empty[g % ST]);
                                if (k + 1 == c1) commit(&dfull[b]);
                            }
                            __syncwarp();
                            issued = true;
                        }
                    }
                }
            }
            if (!ok && lane == 0) record_error(err, kErrWaitTimeout);
            if (issued) {     // the epilogue may have given up on the last chunks
                if (elect_one()) {
                    if constexpr (PAIR)
                        asm volatile(
                            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                                smem_u32(drainbar)) : "memory");
                    else
                        tc_commit(smem_u32(drainbar));
                }
                __syncwarp();
                mbar_wait(smem_u32(drainbar), 0, DRAIN_NS);
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if constexpr (PAIR) cluster_sync_all();
    if (warp == 0) {
        __syncwarp();
        tc_fence_after();
        if constexpr (PAIR)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
        else
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
    }
}

// What has to be laid out before the product: X (any alignment and stride) as
// FP16 [M][ldh], ldh a multiple of 64, zeros past K; rows of W that TMA cannot
// address (O not NULL) as [N][ldo], ldo a multiple of 16, zeros past K; and
// `nzero` counters cleared.
// Blocks of 256 threads, `wide` of them (a power of two, 1 << shift) to a row.
__global__ void __launch_bounds__(256)
q8_prepare_kernel(int M, int N, int K, const int8_t *__restrict__ X, int64_t ldx, int vec, uint16_t *__restrict__ H,
                  int64_t ldh, const int8_t *__restrict__ W, int64_t ldw, int8_t *__restrict__ O, int64_t ldo,
                  int shift, uint32_t *zero, int nzero) {
    pdl_wait();
    pdl_trigger();
    const int64_t row0 = ((int64_t)blockIdx.x << (8 - shift)) + (threadIdx.x >> shift);
    const int64_t rows = (int64_t)gridDim.x << (8 - shift);
    const int c0 = 16 * (int)(threadIdx.x & ((1u << shift) - 1)), step = 16 << shift;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < nzero; i += (int64_t)gridDim.x * 256) zero[i] = 0u;
    for (int64_t m = row0; m < M; m += rows)
        for (int k = c0; k < ldh; k += step) {
            const int8_t *p = X + m * ldx + k;
            uint4 v;
            if (k + 16 > K) v = load16_bytes(p, max(0, K - k));
            else if (vec) v = *reinterpret_cast<const uint4 *>(p);
            else v = load16_unaligned(p, X, X + (int64_t)(M - 1) * ldx + K);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            uint32_t r[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) q8_to_f16(w[j], r[2 * j], r[2 * j + 1]);
            uint4 *o = reinterpret_cast<uint4 *>(H + m * ldh + k);
            o[0] = make_uint4(r[0], r[1], r[2], r[3]);
            o[1] = make_uint4(r[4], r[5], r[6], r[7]);
        }
    if (O == nullptr) return;
    for (int64_t n = row0; n < N; n += rows)
        for (int k = c0; k < ldo; k += step) {
            const int8_t *p = W + n * ldw + k;
            *reinterpret_cast<uint4 *>(O + n * ldo + k) =
                k + 16 > K ? load16_bytes(p, K - k) : load16_unaligned(p, W, W + (int64_t)(N - 1) * ldw + K);
        }
}

bool encode_bytes(EncodeTiledFn enc, CUtensorMap *map, const int8_t *base, int64_t inner, int64_t rows, int64_t ld,
                  uint32_t box_inner, uint32_t box_rows) {
    if (enc == nullptr) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)ld};
    const cuuint32_t box[2] = {box_inner, box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// X expanded, FP16 [rows][ld] (ld a multiple of 64), in boxes of 128 k of
// `box_rows` tokens.
bool encode_x(EncodeTiledFn enc, CUtensorMap *map, void *base, int64_t ld, int64_t rows, uint32_t box_rows) {
    if (enc == nullptr) return false;
    const cuuint64_t dims[3] = {64, (cuuint64_t)rows, (cuuint64_t)(ld / 64)};
    const cuuint64_t strides[2] = {(cuuint64_t)ld * 2, 128};
    const cuuint32_t box[3] = {64, box_rows, 2};
    const cuuint32_t estr[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, base, dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename... P, typename... A>
cudaError_t launch_with(void (*kern)(P...), unsigned grid, int threads, size_t smem, int cluster, cudaStream_t s,
                        A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

constexpr int64_t round16(int64_t v) { return (v + 15) / 16 * 16; }
constexpr size_t round256(size_t v) { return (v + 255) / 256 * 256; }

// Which tile a product runs on, and its division.
struct Choice {
    int nt;          // tokens per tile: 32 (one SM), 64, 128 or 256 (a pair of SMs)
    Plan plan;
    int workers;     // CTAs, or pairs of them
};

Choice choose(int64_t M, int64_t N, int64_t K, int sms) {
    Choice c{};
    const int stages = (int)((K + KT - 1) / KT);
    const int64_t pair_tiles = ((N + 255) / 256) * ((M + 255) / 256);
    c.nt = M <= 32 ? 32 : M <= 64 ? 64 : M <= 128 || pair_tiles < sms / 4 ? 128 : 256;
    const int rows = c.nt == 32 ? 128 : 256;
    const int workers = c.nt == 32 ? sms : sms / 2;
    Plan &p = c.plan;
    p.nt = (int)((N + rows - 1) / rows);
    p.mt = (int)((M + c.nt - 1) / c.nt);
    p.stages = stages;
    p.ks = 1;
    if (c.nt != 256) {
        // the number of parts that ends soonest: rounds of units, each its
        // stages and a fixed cost (set-up and the exchange of sums)
        const int64_t tiles = (int64_t)p.nt * p.mt;
        int64_t best = INT64_MAX;
        for (int ks = 1; ks <= 16 && ks <= stages; ++ks) {
            const int64_t per = (stages + ks - 1) / ks;
            const int64_t rounds = (tiles * ks + workers - 1) / workers;
            const int64_t cost = rounds * (per + (ks > 1 ? 10 : 2));
            if (cost < best) {
                best = cost;
                p.ks = ks;
            }
        }
    }
    p.per = (stages + p.ks - 1) / p.ks;
    p.ks = (stages + p.per - 1) / p.per;
    c.workers = p.units() < workers ? p.units() : workers;
    return c;
}

struct Layout {
    int64_t ldh, ldw;
    size_t x, w, part, counters, total;
    int ncounters;
};

Layout layout(const Q8LinearArgs &a, const Choice &c, bool copy_w) {
    Layout l{};
    l.ldh = (a.K + 63) / 64 * 64;
    l.ldw = copy_w ? round16(a.K) : a.ldw;
    size_t at = 0;
    l.x = at; at += round256((size_t)a.M * l.ldh * 2);
    l.w = at; at += copy_w ? round256((size_t)a.N * l.ldw) : 0;
    l.part = at; at += c.plan.ks > 1 ? round256((size_t)c.plan.units() * (c.nt == 32 ? 1 : 2) * c.nt * 128 * 4) : 0;
    l.ncounters = c.plan.ks > 1 ? c.plan.nt * c.plan.mt * (c.nt == 32 ? 1 : 2) * EPI_WARPS : 0;
    l.counters = at; at += round256((size_t)l.ncounters * 4);
    l.total = at;
    return l;
}

template <typename C, typename OutT>
cudaError_t launch_c(const Q8LinearArgs &a, const Choice &c, const Layout &l, unsigned char *ws, const int8_t *W) {
    alignas(64) CUtensorMap tW, tX;
    if (!encode_bytes(a.encode, &tW, W, a.K, a.N, l.ldw, KT, 128) ||
        !encode_x(a.encode, &tX, ws + l.x, l.ldh, a.M, C::NL))
        return cudaErrorInvalidValue;
    auto kern = q8_mma_kernel<C, OutT>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
    if (e != cudaSuccess) return e;
    // the warpgroups' register shares need the launch to bring REGS per thread
    static const bool regs_ok = [kern] {
        cudaFuncAttributes at;
        return cudaFuncGetAttributes(&at, kern) == cudaSuccess && at.numRegs >= REGS;
    }();
    if (!regs_ok) return cudaErrorInvalidConfiguration;
    const unsigned grid = (unsigned)(C::PAIR ? 2 * c.workers : c.workers);
    return launch_with(kern, grid, THREADS, C::SMEM, C::PAIR ? 2 : 1, a.stream, tW, tX, (int)a.M, (int)a.N, c.plan,
                       a.xs, a.ws, Epilogue{1.0f, 0.0f, a.bias, a.act}, (OutT *)a.C, a.ldc,
                       reinterpret_cast<float *>(ws + l.part), reinterpret_cast<uint32_t *>(ws + l.counters), a.err,
                       a.wait_ns, W != a.W);
}

template <typename OutT>
cudaError_t launch_o(const Q8LinearArgs &a, const Choice &c, const Layout &l, unsigned char *ws, const int8_t *W) {
    switch (c.nt) {
        case 32: return launch_c<Cfg<32, false>, OutT>(a, c, l, ws, W);
        case 64: return launch_c<Cfg<64, true>, OutT>(a, c, l, ws, W);
        case 128: return launch_c<Cfg<128, true>, OutT>(a, c, l, ws, W);
        default: return launch_c<Cfg<256, true>, OutT>(a, c, l, ws, W);
    }
}

bool w_aligned(const Q8LinearArgs &a) {
    return reinterpret_cast<uintptr_t>(a.W) % 16 == 0 && a.ldw % 16 == 0;
}

}  // namespace

bool q8_mma_can_run(const Q8LinearArgs &a) {
    if (a.K < 1) return false;
    const int64_t tiles = ((a.N + 127) / 128) * ((a.M + 31) / 32);
    return tiles <= (INT32_MAX >> 6);
}

size_t q8_mma_workspace_bytes(const Q8LinearArgs &a) {
    return layout(a, choose(a.M, a.N, a.K, a.sm_count), !w_aligned(a)).total;
}

cudaError_t launch_q8_mma(const Q8LinearArgs &a, void *workspace) {
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    const bool copy_w = !w_aligned(a);
    const Choice c = choose(a.M, a.N, a.K, a.sm_count);
    const Layout l = layout(a, c, copy_w);
    int8_t *copy = copy_w ? reinterpret_cast<int8_t *>(ws + l.w) : nullptr;
    const int8_t *W = copy_w ? copy : a.W;
    const int vec = reinterpret_cast<uintptr_t>(a.X) % 16 == 0 && a.ldx % 16 == 0;
    // threads to a row: a 16-byte piece each, up to a whole block
    int shift = 2;
    while (shift < 8 && (16 << shift) < a.K) ++shift;
    const int64_t rows = std::max(a.M, copy_w ? a.N : 0), blocks = (rows + (256 >> shift) - 1) >> (8 - shift);
    const int64_t most = (int64_t)(a.sm_count > 0 ? a.sm_count : 1) * 8;
    const cudaError_t e = launch_with(q8_prepare_kernel, (unsigned)(blocks < most ? blocks : most), 256, 0, 1, a.stream,
                                      (int)a.M, (int)a.N, (int)a.K, a.X, a.ldx, vec,
                                      reinterpret_cast<uint16_t *>(ws + l.x), l.ldh, a.W, a.ldw, copy, l.ldw, shift,
                                      reinterpret_cast<uint32_t *>(ws + l.counters), l.ncounters);
    if (e != cudaSuccess) return e;
    return a.type == kTypeBf16 ? launch_o<__nv_bfloat16>(a, c, l, ws, W) : launch_o<float>(a, c, l, ws, W);
}

}  // namespace sgemm_gb300
