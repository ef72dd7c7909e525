// q8_api.cu -- the 8-bit serving operators of include/sgemm_gb300.h: argument
// checks, quick returns and kernel choice.
#include <cstdint>

#include "q8.cuh"
#include "sgemm_gb300.h"
#include "workspace.cuh"

using namespace sgemm_gb300;

namespace {

constexpr int64_t kMaxElems = int64_t(1) << 40;
// Which products stream W past 16 tokens at a time instead of running on the
// tensor cores' tiles: up to 16 tokens (16 x 8192 x 4096: 10.8 against 13.3 us),
// and as long as blocks of 16 tokens x 32 channels give every SM at most two,
// where the tiles' set-up counts for more than reading W again (128 x 512 x 512
// 3.3 against 8.4 us, 64 x 2048 x 4096 11.5 either way; at four to an SM, 64 x
// 4096 x 1024, 11.8 against 8.4).  The latter needs the fast streaming kernel,
// for which W is 16-byte aligned.
constexpr int64_t kStreamTokens = 16;
bool streams(const Q8LinearArgs &a) {
    if (a.M <= kStreamTokens) return true;
    const bool aligned = reinterpret_cast<uintptr_t>(a.W) % 16 == 0 && a.ldw % 16 == 0 && a.K >= 64;
    return aligned && ((a.M + 15) / 16) * ((a.N + 31) / 32) <= 2 * (int64_t)a.sm_count;
}

size_t type_size(int type) { return type == SGEMM_TYPE_BF16 ? 2 : 4; }
bool known_type(int type) { return type == SGEMM_TYPE_FP32 || type == SGEMM_TYPE_BF16; }

// The bytes a rows x cols array with row stride ld touches; empty for NULL.
struct Range {
    uintptr_t lo = 0, hi = 0;
    const void *p = nullptr;
    int64_t ld = 0;
    Range(const void *ptr, int64_t rows, int64_t cols, int64_t stride, size_t elem) : p(ptr), ld(stride) {
        if (ptr == nullptr || rows <= 0 || cols <= 0) return;
        lo = reinterpret_cast<uintptr_t>(ptr);
        hi = lo + (uintptr_t)((rows - 1) * stride + cols) * elem;
    }
    bool overlaps(const Range &o) const { return lo < o.hi && o.lo < hi; }
    bool same(const Range &o) const { return p == o.p && ld == o.ld; }
};

int check_matrix(const void *p, int64_t rows, int64_t cols, int64_t ld) {
    if (p == nullptr) return SGEMM_ERR_NULL_PTR;
    if (ld < cols) return SGEMM_ERR_BAD_LD;
    if (ld > 0 && rows > kMaxElems / ld) return SGEMM_ERR_BAD_DIM;
    return SGEMM_OK;
}

// Pointers to FP32 and BF16 elements are element-aligned.
bool misaligned(const void *p, size_t elem) { return reinterpret_cast<uintptr_t>(p) % elem != 0; }

int device_args(unsigned **err, uint64_t *wait_ns, int *sm_count, EncodeTiledFn *encode) {
    GemmArgs g{};
    const int rc = fill_device_args(g);
    if (rc != SGEMM_OK) return rc;
    if (err) *err = g.err;
    if (wait_ns) *wait_ns = g.wait_ns;
    if (sm_count) *sm_count = g.sm_count;
    if (encode) *encode = g.encode;
    return SGEMM_OK;
}

int launch_status(cudaError_t e) {
    if (e == cudaSuccess) return SGEMM_OK;
    (void)cudaGetLastError();
    return SGEMM_ERR_CUDA;
}

int rows_call(Q8RowsArgs a) {
    if (a.M < 0 || a.K < 0) return SGEMM_ERR_BAD_DIM;
    if (!known_type(a.type)) return SGEMM_ERR_BAD_ARG;
    if (a.M == 0) return SGEMM_OK;
    if (a.M > INT32_MAX) return SGEMM_ERR_BAD_DIM;
    if (a.scale == nullptr) return SGEMM_ERR_NULL_PTR;
    const size_t es = type_size(a.type);
    if (a.K > 0) {
        int rc = check_matrix(a.x, a.M, a.K, a.ldx);
        if (rc == SGEMM_OK) rc = check_matrix(a.q, a.M, a.K, a.ldq);
        if (rc == SGEMM_OK && a.residual) rc = check_matrix(a.residual, a.M, a.K, a.ldr);
        if (rc == SGEMM_OK && a.h) rc = check_matrix(a.h, a.M, a.K, a.ldh);
        if (rc == SGEMM_OK && a.y) rc = check_matrix(a.y, a.M, a.K, a.ldy);
        if (rc != SGEMM_OK) return rc;
    }
    if (misaligned(a.x, es) || misaligned(a.residual, es) || misaligned(a.h, es) || misaligned(a.y, es) ||
        misaligned(a.weight, 4) || misaligned(a.scale, 4))
        return SGEMM_ERR_BAD_ARG;
    const Range x(a.x, a.M, a.K, a.ldx, es), r(a.residual, a.M, a.K, a.ldr, es), w(a.weight, 1, a.K, a.K, 4);
    const Range h(a.h, a.M, a.K, a.ldh, es), y(a.y, a.M, a.K, a.ldy, es), q(a.q, a.M, a.K, a.ldq, 1);
    const Range s(a.scale, 1, a.M, a.M, 4);
    // every output apart from every input and every other output, except that
    // h may take the place of x or of the residual
    for (const Range *o : {&h, &y, &q, &s})
        for (const Range *i : {&x, &r, &w})
            if (o->overlaps(*i) && !(o == &h && (i == &x || i == &r) && o->same(*i))) return SGEMM_ERR_ALIAS;
    if (h.overlaps(y) || h.overlaps(q) || h.overlaps(s) || y.overlaps(q) || y.overlaps(s) || q.overlaps(s))
        return SGEMM_ERR_ALIAS;
    const int rc = device_args(nullptr, nullptr, &a.sm_count, nullptr);
    if (rc != SGEMM_OK) return rc;
    return launch_status(launch_q8_rows(a));
}

}  // namespace

extern "C" {

int sgemm_q8_quantize(int64_t M, int64_t K, const void *x, int64_t ldx, int type, int8_t *q, int64_t ldq,
                      float *scale, void *stream) {
    Q8RowsArgs a{};
    a.M = M; a.K = K; a.type = type;
    a.x = x; a.ldx = ldx;
    a.q = q; a.ldq = ldq; a.scale = scale;
    a.stream = static_cast<cudaStream_t>(stream);
    return rows_call(a);
}

int sgemm_q8_rmsnorm(int64_t M, int64_t K, const void *x, int64_t ldx, const void *residual, int64_t ldr,
                     int type, const float *weight, float eps, void *h, int64_t ldh, void *y, int64_t ldy,
                     int8_t *q, int64_t ldq, float *scale, void *stream) {
    if (M > 0 && K > 0 && weight == nullptr) return SGEMM_ERR_NULL_PTR;
    if (!(eps >= 0.0f)) return SGEMM_ERR_BAD_ARG;
    Q8RowsArgs a{};
    a.M = M; a.K = K; a.type = type;
    a.x = x; a.ldx = ldx; a.residual = residual; a.ldr = ldr;
    a.weight = weight; a.eps = eps;
    a.h = h; a.ldh = ldh; a.y = y; a.ldy = ldy;
    a.q = q; a.ldq = ldq; a.scale = scale;
    a.stream = static_cast<cudaStream_t>(stream);
    return rows_call(a);
}

int sgemm_q8_linear(int64_t M, int64_t N, int64_t K, const int8_t *X, int64_t ldx, const float *xs,
                    const int8_t *W, int64_t ldw, const float *ws, const float *bias, int activation, void *C,
                    int64_t ldc, int type, void *stream) {
    if (M < 0 || N < 0 || K < 0 || K > kQ8MaxK || M > INT32_MAX || N > INT32_MAX) return SGEMM_ERR_BAD_DIM;
    if (!known_type(type) || activation < SGEMM_ACT_NONE || activation > SGEMM_ACT_SILU) return SGEMM_ERR_BAD_ARG;
    if (M == 0 || N == 0) return SGEMM_OK;
    int rc = check_matrix(C, M, N, ldc);
    if (rc != SGEMM_OK) return rc;
    if (xs == nullptr || ws == nullptr) return SGEMM_ERR_NULL_PTR;
    if (K > 0) {
        rc = check_matrix(X, M, K, ldx);
        if (rc == SGEMM_OK) rc = check_matrix(W, N, K, ldw);
        if (rc != SGEMM_OK) return rc;
    }
    if (misaligned(C, type_size(type)) || misaligned(xs, 4) || misaligned(ws, 4) || misaligned(bias, 4))
        return SGEMM_ERR_BAD_ARG;
    const Range c(C, M, N, ldc, type_size(type));
    const Range ins[] = {Range(X, M, K, ldx, 1), Range(W, N, K, ldw, 1), Range(xs, 1, M, M, 4),
                         Range(ws, 1, N, N, 4), Range(bias, 1, N, N, 4)};
    for (const Range &i : ins)
        if (c.overlaps(i)) return SGEMM_ERR_ALIAS;
    Q8LinearArgs a{};
    a.M = M; a.N = N; a.K = K;
    a.X = X; a.ldx = ldx; a.xs = xs; a.W = W; a.ldw = ldw; a.ws = ws;
    a.bias = bias; a.act = activation;
    a.C = C; a.ldc = ldc; a.type = type;
    a.stream = static_cast<cudaStream_t>(stream);
    rc = device_args(&a.err, &a.wait_ns, &a.sm_count, &a.encode);
    if (rc != SGEMM_OK) return rc;
    if (streams(a) || !q8_mma_can_run(a)) return launch_status(launch_q8_stream(a));
    WorkspaceLease work;
    rc = stream_workspace(q8_mma_workspace_bytes(a), a.stream, work);
    if (rc != SGEMM_OK) return rc;
    return launch_status(launch_q8_mma(a, work.p));
}

int sgemm_q8_moe(int64_t T, int64_t E, int64_t top_k, int64_t H, int64_t I, const void *x, int64_t ldx, int type,
                 const float *router, int64_t ldr, const int8_t *w_up, int64_t ldu, const float *s_up,
                 const int8_t *w_down, int64_t ldd, const float *s_down, int renormalize, void *out, int64_t ldo,
                 int32_t *ids, float *gates, void *stream) {
    if (T < 0 || E < 1 || top_k < 1 || top_k > E || H < 1 || I < 1 || H > kQ8MaxK || I > kQ8MaxK)
        return SGEMM_ERR_BAD_DIM;
    if (T > kMoeMaxTokens || E > kMoeMaxExperts || top_k > kMoeMaxTopK) return SGEMM_ERR_TOO_LARGE;
    if (!known_type(type)) return SGEMM_ERR_BAD_ARG;
    if (T == 0) return SGEMM_OK;
    int rc = check_matrix(x, T, H, ldx);
    if (rc == SGEMM_OK) rc = check_matrix(out, T, H, ldo);
    if (rc == SGEMM_OK) rc = check_matrix(router, E, H, ldr);
    if (rc == SGEMM_OK) rc = check_matrix(w_up, E * 2 * I, H, ldu);
    if (rc == SGEMM_OK) rc = check_matrix(w_down, E * H, I, ldd);
    if (rc != SGEMM_OK) return rc;
    if (s_up == nullptr || s_down == nullptr) return SGEMM_ERR_NULL_PTR;
    const size_t es = type_size(type);
    if (misaligned(x, es) || misaligned(out, es) || misaligned(router, 4) || misaligned(s_up, 4) ||
        misaligned(s_down, 4) || misaligned(ids, 4) || misaligned(gates, 4))
        return SGEMM_ERR_BAD_ARG;
    const Range outs[] = {Range(out, T, H, ldo, es), Range(ids, 1, T * top_k, T * top_k, 4),
                          Range(gates, 1, T * top_k, T * top_k, 4)};
    const Range ins[] = {Range(x, T, H, ldx, es), Range(router, E, H, ldr, 4),
                         Range(w_up, E * 2 * I, H, ldu, 1), Range(s_up, 1, E * 2 * I, E * 2 * I, 4),
                         Range(w_down, E * H, I, ldd, 1), Range(s_down, 1, E * H, E * H, 4)};
    for (const Range &o : outs)
        for (const Range &i : ins)
            if (o.overlaps(i)) return SGEMM_ERR_ALIAS;
    if (outs[0].overlaps(outs[1]) || outs[0].overlaps(outs[2]) || outs[1].overlaps(outs[2])) return SGEMM_ERR_ALIAS;
    Q8MoeArgs a{};
    a.T = (int)T; a.E = (int)E; a.top_k = (int)top_k; a.H = (int)H; a.I = (int)I;
    a.type = type; a.x = x; a.ldx = ldx; a.router = router; a.ldr = ldr;
    a.w_up = w_up; a.ldu = ldu; a.s_up = s_up; a.w_down = w_down; a.ldd = ldd; a.s_down = s_down;
    a.renormalize = renormalize != 0;
    a.out = out; a.ldo = ldo; a.ids = ids; a.gates = gates;
    a.stream = static_cast<cudaStream_t>(stream);
    rc = device_args(&a.err, &a.wait_ns, &a.sm_count, &a.encode);
    if (rc != SGEMM_OK) return rc;
    WorkspaceLease work;
    rc = stream_workspace(q8_moe_workspace_bytes(a.T, a.E, a.top_k, a.H, a.I), a.stream, work);
    if (rc != SGEMM_OK) return rc;
    return launch_status(launch_q8_moe(a, work.p));
}

}  // extern "C"
