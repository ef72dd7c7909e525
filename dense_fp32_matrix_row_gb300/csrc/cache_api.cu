// cache_api.cu -- the attention operators of include/sgemm_gb300.h: argument checks,
// quick returns, and the counters that a stream's attention calls share.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <map>
#include <mutex>

#include "cache.cuh"
#include "workspace.cuh"

using namespace sgemm_gb300;

namespace {

constexpr int64_t kMaxElems = int64_t(1) << 40;   // keeps every offset far from int64 overflow
constexpr int64_t kMaxHeads = 65535;

size_t type_size(int type) { return type == SGEMM_TYPE_BF16 ? 2 : 4; }
bool known_type(int type) { return type == SGEMM_TYPE_FP32 || type == SGEMM_TYPE_BF16; }
bool misaligned(const void *p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to != 0; }

// The bytes an array touches: `span` of them from each multiple of `step` on (step 0:
// any bytes between lo and hi).
struct Range {
    uintptr_t lo = 0, hi = 0, step = 0, span = 0;
    const sgemm_heads *heads = nullptr;
    Range() = default;
    Range(const void *p, int64_t bytes) {
        if (p == nullptr || bytes <= 0) return;
        lo = reinterpret_cast<uintptr_t>(p);
        hi = lo + (uintptr_t)bytes;
    }
    Range(const void *p, int64_t n, int64_t stride, int64_t each) : Range(p, n > 0 ? (n - 1) * stride + each : 0) {
        if (n > 1 && stride >= each) {
            step = (uintptr_t)stride;
            span = (uintptr_t)each;
        }
    }
    bool overlaps(const Range &o) const {
        if (!(lo < o.hi && o.lo < hi)) return false;
        if (step == 0 || step != o.step) return true;
        const uintptr_t off = o.lo >= lo ? (o.lo - lo) % step : (step - (lo - o.lo) % step) % step;
        return off < span || off + o.span > step;
    }
};

bool there(const sgemm_heads *h) { return h != nullptr && h->heads != 0; }

Range range_of(const sgemm_heads *h, int64_t T, int64_t D, size_t es) {
    if (!there(h)) return Range();
    const int64_t each = (h->heads - 1) * h->hs + D, n = (int64_t)es;
    Range r = T > 1 && h->ld >= each ? Range(h->p, T, h->ld * n, each * n) : Range(h->p, ((T - 1) * h->ld + each) * n);
    r.heads = h;
    return r;
}

// In place: the same elements in the same places.
bool same(const Range &a, const Range &b) {
    return a.heads && b.heads && a.heads->p == b.heads->p && a.heads->heads == b.heads->heads &&
           a.heads->ld == b.heads->ld && (a.heads->heads == 1 || a.heads->hs == b.heads->hs);
}

// Heads of T > 0 tokens.
int check_heads(const sgemm_heads *h, int64_t T, int64_t D, int type, bool output) {
    if (!there(h)) return SGEMM_OK;
    if (h->heads < 0 || h->heads > kMaxHeads) return SGEMM_ERR_BAD_DIM;
    if (h->p == nullptr) return SGEMM_ERR_NULL_PTR;
    if (h->ld < 0 || h->hs < 0) return SGEMM_ERR_BAD_LD;
    // hs leads from head to head: of a single one it is not used
    if (h->ld > kMaxElems || (h->heads > 1 && h->hs > kMaxElems / h->heads) || (h->ld > 0 && T > kMaxElems / h->ld))
        return SGEMM_ERR_BAD_DIM;
    if (output) {
        const bool by_token = (h->heads == 1 || h->hs >= D) && (T == 1 || h->ld >= (h->heads - 1) * h->hs + D);
        const bool by_head = (T == 1 || h->ld >= D) && (h->heads == 1 || h->hs >= (T - 1) * h->ld + D);
        if (!by_token && !by_head) return SGEMM_ERR_BAD_LD;
    }
    return misaligned(h->p, type_size(type)) ? SGEMM_ERR_BAD_ARG : SGEMM_OK;
}

int check_dim(int64_t D) { return D < 16 || D > kCacheMaxDim || D % 16 != 0 ? SGEMM_ERR_BAD_DIM : SGEMM_OK; }

int check_cache(const sgemm_q8_cache *c) {
    if (c == nullptr) return SGEMM_ERR_NULL_PTR;
    const int rc = check_dim(c->dim);
    if (rc != SGEMM_OK) return rc;
    if (c->blocks < 0 || c->heads < 1 || c->heads > kMaxHeads || c->page < 1 || c->page > (1 << 30) ||
        c->heads * c->page > INT_MAX)
        return SGEMM_ERR_BAD_DIM;
    if (c->blocks > kMaxElems / c->page) return SGEMM_ERR_BAD_DIM;
    if (c->blocks == 0) return SGEMM_OK;
    if (!c->k || !c->v || !c->k_scale || !c->v_scale) return SGEMM_ERR_NULL_PTR;
    const int64_t rows = c->heads * c->page;
    for (int64_t s : {c->k_stride, c->v_stride}) {
        if (s < rows * c->dim) return SGEMM_ERR_BAD_LD;
        if (c->blocks > kMaxElems / s) return SGEMM_ERR_BAD_DIM;
        if (s % 16 != 0) return SGEMM_ERR_BAD_ARG;
    }
    for (int64_t s : {c->k_scale_stride, c->v_scale_stride}) {
        if (s < rows) return SGEMM_ERR_BAD_LD;
        if (c->blocks > kMaxElems / s) return SGEMM_ERR_BAD_DIM;
    }
    if (misaligned(c->k, 16) || misaligned(c->v, 16) || misaligned(c->k_scale, 4) || misaligned(c->v_scale, 4))
        return SGEMM_ERR_BAD_ARG;
    return SGEMM_OK;
}

struct CacheRanges {
    Range r[4];
    explicit CacheRanges(const sgemm_q8_cache &c) {
        const int64_t rows = c.heads * c.page;
        r[0] = Range(c.k, c.blocks, c.k_stride, rows * c.dim);
        r[1] = Range(c.v, c.blocks, c.v_stride, rows * c.dim);
        r[2] = Range(c.k_scale, c.blocks, c.k_scale_stride * 4, rows * 4);
        r[3] = Range(c.v_scale, c.blocks, c.v_scale_stride * 4, rows * 4);
    }
    bool overlaps(const Range &o) const {
        for (const Range &x : r)
            if (x.overlaps(o)) return true;
        return false;
    }
    bool overlap_each_other() const {
        for (int i = 0; i < 4; ++i)
            for (int j = 0; j < i; ++j)
                if (r[i].overlaps(r[j])) return true;
        return false;
    }
};

int check_rotary(const sgemm_rotary *r, int64_t T, int64_t D) {
    if (r == nullptr || r->dims == 0) return SGEMM_OK;
    if (r->dims < 0 || r->dims > D || r->dims % 2 != 0 || r->rows < 0) return SGEMM_ERR_BAD_DIM;
    if (r->positions == nullptr && r->rows < T) return SGEMM_ERR_BAD_DIM;
    if (r->rows > 0 && (r->cos == nullptr || r->sin == nullptr)) return SGEMM_ERR_NULL_PTR;
    if (r->ld < r->dims / 2) return SGEMM_ERR_BAD_LD;
    if (r->rows > kMaxElems / r->ld) return SGEMM_ERR_BAD_DIM;
    if (misaligned(r->cos, 4) || misaligned(r->sin, 4) || misaligned(r->positions, 8)) return SGEMM_ERR_BAD_ARG;
    return SGEMM_OK;
}

int device_args(unsigned **err, int *sm_count) {
    GemmArgs g{};
    const int rc = fill_device_args(g);
    if (rc != SGEMM_OK) return rc;
    *err = g.err;
    *sm_count = g.sm_count;
    return SGEMM_OK;
}

int launch_status(cudaError_t e) {
    if (e == cudaSuccess) return SGEMM_OK;
    (void)cudaGetLastError();
    return SGEMM_ERR_CUDA;
}

sgemm_heads value(const sgemm_heads *h) {
    if (!there(h)) return sgemm_heads{nullptr, 0, 0, 0};
    return sgemm_heads{h->p, h->heads, h->ld, h->heads > 1 ? h->hs : 0};
}

// The three calls on new tokens' heads; `cache` nullptr: float results alone.
int head_rows(int64_t T, int64_t D, int type, const sgemm_heads *q, const sgemm_heads *q_out, const float *q_weight,
              const sgemm_heads *k, const sgemm_heads *k_out, const float *k_weight, const sgemm_heads *v, float eps,
              const sgemm_rotary *rotary, const int64_t *slots, const sgemm_q8_cache *cache, void *stream) {
    if (T < 0 || T > INT32_MAX) return SGEMM_ERR_BAD_DIM;
    int rc = check_dim(D);
    if (rc != SGEMM_OK) return rc;
    if (!known_type(type) || !(eps >= 0.0f)) return SGEMM_ERR_BAD_ARG;
    if (T == 0) return SGEMM_OK;
    rc = check_heads(q, T, D, type, false);
    if (rc == SGEMM_OK) rc = check_heads(q_out, T, D, type, true);
    if (rc == SGEMM_OK) rc = check_heads(k, T, D, type, false);
    if (rc == SGEMM_OK) rc = check_heads(k_out, T, D, type, true);
    if (rc == SGEMM_OK) rc = check_heads(v, T, D, type, false);
    if (rc == SGEMM_OK) rc = check_rotary(rotary, T, D);
    if (rc != SGEMM_OK) return rc;
    // every kind of head with its result
    if (there(q) && !there(q_out)) return SGEMM_ERR_NULL_PTR;
    if (there(q) && q->heads != q_out->heads) return SGEMM_ERR_BAD_DIM;
    if (cache != nullptr) {
        if (!there(k) || !there(v) || slots == nullptr) return SGEMM_ERR_NULL_PTR;
        if (k->heads != cache->heads || v->heads != cache->heads) return SGEMM_ERR_BAD_DIM;
        if (misaligned(slots, 8)) return SGEMM_ERR_BAD_ARG;
    } else {
        if (there(k) && !there(k_out)) return SGEMM_ERR_NULL_PTR;
        if (there(k) && k->heads != k_out->heads) return SGEMM_ERR_BAD_DIM;
        if (!there(q) && !there(k)) return SGEMM_OK;
    }
    if (misaligned(q_weight, 4) || misaligned(k_weight, 4)) return SGEMM_ERR_BAD_ARG;

    const bool turned = rotary != nullptr && rotary->dims != 0;
    const size_t es = type_size(type);
    const Range rq = range_of(q, T, D, es), rk = range_of(k, T, D, es), rv = range_of(v, T, D, es);
    const Range oq = there(q) ? range_of(q_out, T, D, es) : Range(), ok = cache || !there(k) ? Range() : range_of(k_out, T, D, es);
    Range more[6] = {Range(q_weight, 4 * D), Range(k_weight, 4 * D), Range(slots, 8 * T)};
    if (turned) {
        const int64_t bytes = rotary->rows > 0 ? 4 * ((rotary->rows - 1) * rotary->ld + rotary->dims / 2) : 0;
        more[3] = Range(rotary->cos, bytes);
        more[4] = Range(rotary->sin, bytes);
        more[5] = Range(rotary->positions, 8 * T);
    }
    for (const Range *o : {&oq, &ok}) {
        for (const Range *i : {&rq, &rk, &rv})
            if (o->overlaps(*i) && !(same(*o, *i) && i == (o == &oq ? &rq : &rk))) return SGEMM_ERR_ALIAS;
        for (const Range &i : more)
            if (o->overlaps(i)) return SGEMM_ERR_ALIAS;
    }
    if (oq.overlaps(ok)) return SGEMM_ERR_ALIAS;
    if (cache != nullptr && cache->blocks > 0) {
        const CacheRanges c(*cache);
        if (c.overlap_each_other() || c.overlaps(rq) || c.overlaps(rk) || c.overlaps(rv) || c.overlaps(oq)) return SGEMM_ERR_ALIAS;
        for (const Range &i : more)
            if (c.overlaps(i)) return SGEMM_ERR_ALIAS;
    }

    HeadRowsArgs a{};
    a.T = T; a.D = (int)D; a.type = type;
    a.q = value(q); a.k = value(k); a.v = cache ? value(v) : value(nullptr);
    a.q_out = there(q) ? value(q_out) : value(nullptr);
    a.k_out = there(k) && !cache ? value(k_out) : value(nullptr);
    a.q_weight = q_weight; a.k_weight = k_weight; a.eps = eps;
    if (turned) a.rotary = *rotary;
    if (cache != nullptr) {
        a.slots = slots;
        a.cache = *cache;
    }
    a.stream = static_cast<cudaStream_t>(stream);
    rc = device_args(&a.err, &a.sm_count);
    if (rc != SGEMM_OK) return rc;
    return launch_status(launch_head_rows(a));
}

// ---- counters -------------------------------------------------------------------------

// kAttendTickets words for each (device, stream), zero between calls: every call
// leaves them as it found them, so they are cleared when they are made and never again.
std::mutex g_tickets_mu;
std::map<StreamKey, unsigned *> g_tickets;

bool release_tickets() {
    std::lock_guard<std::mutex> lock(g_tickets_mu);
    int cur = 0;
    bool ok = cudaGetDevice(&cur) == cudaSuccess;
    for (auto &kv : g_tickets) {
        if (cudaSetDevice(kv.first.dev) != cudaSuccess || kv.first.synchronize() != cudaSuccess ||
            cudaFree(kv.second) != cudaSuccess)
            ok = false;
    }
    g_tickets.clear();
    return cudaSetDevice(cur) == cudaSuccess && ok;
}

int stream_tickets(cudaStream_t s, unsigned **out) try {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return SGEMM_ERR_CUDA;
    std::lock_guard<std::mutex> lock(g_tickets_mu);
    const StreamKey key(dev, s);
    auto it = g_tickets.find(key);
    if (it == g_tickets.end()) {
        if (s != nullptr && s != cudaStreamLegacy) {     // the legacy stream cannot be captured
            cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
            if (cudaStreamIsCapturing(s, &cs) != cudaSuccess) {
                (void)cudaGetLastError();
                return SGEMM_ERR_CUDA;
            }
            if (cs != cudaStreamCaptureStatusNone) return SGEMM_ERR_CAPTURE;
        }
        it = g_tickets.emplace(key, nullptr).first;
        void *p = nullptr;
        const size_t bytes = kAttendTickets * sizeof(unsigned);
        if (cudaMallocAsync(&p, bytes, s) != cudaSuccess || cudaMemsetAsync(p, 0, bytes, s) != cudaSuccess) {
            (void)cudaGetLastError();
            if (p != nullptr) (void)cudaFreeAsync(p, s);
            g_tickets.erase(it);
            return SGEMM_ERR_CUDA;
        }
        it->second = static_cast<unsigned *>(p);
        on_release(release_tickets);
    }
    *out = it->second;
    return SGEMM_OK;
} catch (...) {      // no memory for the map
    return SGEMM_ERR_CUDA;
}

}  // namespace

extern "C" {

int sgemm_norm_rope(int64_t T, int64_t D, int type, const sgemm_heads *q, const sgemm_heads *q_out,
                    const float *q_weight, const sgemm_heads *k, const sgemm_heads *k_out, const float *k_weight,
                    float eps, const sgemm_rotary *rotary, void *stream) {
    return head_rows(T, D, type, q, q_out, q_weight, k, k_out, k_weight, nullptr, eps, rotary, nullptr, nullptr, stream);
}

int sgemm_q8_cache_write(int64_t T, int type, const sgemm_heads *k, const sgemm_heads *v, const int64_t *slots,
                         const sgemm_q8_cache *cache, void *stream) {
    const int rc = check_cache(cache);
    if (rc != SGEMM_OK) return rc;
    return head_rows(T, cache->dim, type, nullptr, nullptr, nullptr, k, nullptr, nullptr, v, 0.0f, nullptr, slots, cache,
                     stream);
}

int sgemm_q8_norm_rope_write(int64_t T, int type, const sgemm_heads *q, const sgemm_heads *q_out,
                             const float *q_weight, const sgemm_heads *k, const float *k_weight, const sgemm_heads *v,
                             float eps, const sgemm_rotary *rotary, const int64_t *slots, const sgemm_q8_cache *cache,
                             void *stream) {
    const int rc = check_cache(cache);
    if (rc != SGEMM_OK) return rc;
    return head_rows(T, cache->dim, type, q, q_out, q_weight, k, nullptr, k_weight, v, eps, rotary, slots, cache, stream);
}

int sgemm_q8_cache_read(int64_t N, int type, const sgemm_q8_cache *cache, const int64_t *slots,
                        const sgemm_heads *k_out, const sgemm_heads *v_out, void *stream) {
    int rc = check_cache(cache);
    if (rc != SGEMM_OK) return rc;
    if (N < 0 || N > INT32_MAX) return SGEMM_ERR_BAD_DIM;
    if (!known_type(type)) return SGEMM_ERR_BAD_ARG;
    if (N == 0 || (!there(k_out) && !there(v_out))) return SGEMM_OK;
    rc = check_heads(k_out, N, cache->dim, type, true);
    if (rc == SGEMM_OK) rc = check_heads(v_out, N, cache->dim, type, true);
    if (rc != SGEMM_OK) return rc;
    if (slots == nullptr) return SGEMM_ERR_NULL_PTR;
    if (misaligned(slots, 8)) return SGEMM_ERR_BAD_ARG;
    for (const sgemm_heads *h : {k_out, v_out})
        if (there(h) && h->heads != cache->heads) return SGEMM_ERR_BAD_DIM;
    const size_t es = type_size(type);
    const Range ok = range_of(k_out, N, cache->dim, es), ov = range_of(v_out, N, cache->dim, es), at(slots, 8 * N);
    const CacheRanges c(*cache);
    if (ok.overlaps(ov) || ok.overlaps(at) || ov.overlaps(at) || c.overlaps(ok) || c.overlaps(ov)) return SGEMM_ERR_ALIAS;
    CacheReadArgs a{};
    a.N = N; a.type = type;
    a.cache = *cache; a.slots = slots;
    a.k_out = value(k_out); a.v_out = value(v_out);
    a.stream = static_cast<cudaStream_t>(stream);
    rc = device_args(&a.err, &a.sm_count);
    if (rc != SGEMM_OK) return rc;
    return launch_status(launch_cache_read(a));
}

int sgemm_q8_attend(int64_t B, int type, const sgemm_heads *q, const sgemm_q8_cache *cache, const int32_t *table,
                    int64_t ld_table, int64_t pages, const int32_t *lens, float scale, int64_t window,
                    const sgemm_heads *out, float *lse, void *stream) {
    int rc = check_cache(cache);
    if (rc != SGEMM_OK) return rc;
    if (B < 0 || B > (1 << 30) || pages < 0 || pages > INT32_MAX / cache->page) return SGEMM_ERR_BAD_DIM;
    if (!known_type(type) || !std::isfinite(scale * kLog2e) || window < 0) return SGEMM_ERR_BAD_ARG;
    if (B == 0) return SGEMM_OK;
    if (!there(q) || !there(out) || lens == nullptr || (table == nullptr && pages > 0)) return SGEMM_ERR_NULL_PTR;
    rc = check_heads(q, B, cache->dim, type, false);
    if (rc == SGEMM_OK) rc = check_heads(out, B, cache->dim, type, true);
    if (rc != SGEMM_OK) return rc;
    if (q->heads != out->heads || q->heads % cache->heads != 0) return SGEMM_ERR_BAD_DIM;
    // The kernel counts the strips of 16 tokens of all sequences, key heads and groups of query
    // heads in 32 bits.  A group takes 8 heads at least.
    const int64_t G = q->heads / cache->heads;
    if (cache->heads * std::min(G, 2 * ((G + 7) / 8)) * (pages * cache->page / 16 + 2) > INT32_MAX / B) return SGEMM_ERR_TOO_LARGE;
    if (ld_table < pages) return SGEMM_ERR_BAD_LD;
    if (ld_table > 0 && B > kMaxElems / ld_table) return SGEMM_ERR_BAD_DIM;
    if (misaligned(table, 4) || misaligned(lens, 4) || misaligned(lse, 4)) return SGEMM_ERR_BAD_ARG;
    const size_t es = type_size(type);
    const Range ins[] = {range_of(q, B, cache->dim, es), Range(table, pages > 0 ? 4 * ((B - 1) * ld_table + pages) : 0),
                         Range(lens, 4 * B)};
    const Range o = range_of(out, B, cache->dim, es), l(lse, 4 * B * q->heads);
    for (const Range &i : ins)
        if (o.overlaps(i) || l.overlaps(i)) return SGEMM_ERR_ALIAS;
    const CacheRanges c(*cache);
    if (o.overlaps(l) || c.overlaps(o) || c.overlaps(l)) return SGEMM_ERR_ALIAS;
    AttendArgs a{};
    a.B = (int)B; a.Hk = (int)cache->heads; a.G = (int)G; a.D = (int)cache->dim; a.type = type;
    a.q = value(q); a.out = value(out);
    a.cache = *cache;
    a.table = table; a.ld_table = ld_table; a.width = (int)pages; a.lens = lens;
    a.scale = scale;
    a.window = (int)(window < INT32_MAX ? window : 0);
    a.lse = lse;
    a.stream = static_cast<cudaStream_t>(stream);
    rc = device_args(&a.err, &a.sm_count);
    if (rc != SGEMM_OK) return rc;
    unsigned *tickets = nullptr;
    rc = stream_tickets(a.stream, &tickets);
    if (rc != SGEMM_OK) return rc;
    WorkspaceLease work;
    rc = stream_workspace(attend_workspace_bytes(a), a.stream, work);
    if (rc != SGEMM_OK) return rc;
    return launch_status(launch_attend(a, work.p, tickets));
}

}  // extern "C"
