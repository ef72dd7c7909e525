// attend.cu -- attention over the paged cache: the choice of a form (attend.cuh)
// and its parameters.
#include "attend.cuh"

namespace sgemm_gb300 {
namespace {

// The form that heads of D run in (8 key heads of 8, 16 sequences of 16384: heads of 96 in 128 86
// us, in 96 75; of 80 95 and 82; of 192 in 256 154, in 192 139; of 144 154 and 121; FP32 96 108 and 91,
// 192 187 and 147).
int padded(int D) { return D <= 64 ? 64 : D <= 96 ? 96 : D <= 128 ? 128 : D <= 192 ? 192 : 256; }

// Sets of 8 MMA columns.  More than 8 query heads to a key head take up to four sets,
// which read a strip once for all (8 key heads, 16 sequences of 16384: 16 heads of 64 73 us against
// 113 for two sets of 8 one after the other, 128: 107 and 172; 24 heads of 64 91 against 139 for two
// times two sets, 128: 141 and 214; 32 heads 106 and 139, 168 and 214; FP32, three sets against two
// times two, 64: 120 and 199, 128: 200 and 306).  Heads of 192 take two (16 heads
// 155 us, 8 139; FP32 217 and 147), of 256 two, in FP32 one: more leave too few registers or warps (24
// heads of 256 in three sets 398 us, in two times two 362; FP32, two sets 213, two times one 200).
// As few times as that allows, alike.
int tiles(const AttendArgs &a) {
    const int sets = (a.G + 7) / 8, times = (sets - 1) / attend_sets(padded(a.D), a.type == kTypeBf16) + 1;
    return (sets + times - 1) / times;
}

bool aligned16(const sgemm_heads &h, int es) {
    return reinterpret_cast<uintptr_t>(h.p) % 16 == 0 && h.ld * es % 16 == 0 && h.hs * es % 16 == 0;
}

// t / d = (t * mul) >> shift for 0 <= t < 2^31: mul = ceil(2^shift / d), which is off
// by less than 2^(shift-31) / t of it.
void divider(uint32_t d, uint32_t *mul, uint32_t *shift) {
    uint32_t l = 0;
    while (((uint64_t)1 << l) < d) ++l;
    *shift = 31 + l;
    *mul = (uint32_t)((((uint64_t)1 << *shift) + d - 1) / d);
}

}  // namespace

size_t attend_workspace_bytes(const AttendArgs &a) {
    const int dt = padded(a.D), nt = tiles(a);
    const int terms = a.type == kTypeBf16 ? 1 : 2;
    return (size_t)a.sm_count * attend_parts(dt, nt, terms) * attend_part(dt, nt) * sizeof(float);
}

cudaError_t launch_attend(const AttendArgs &a, void *workspace, unsigned *tickets) {
    const int es = a.type == kTypeBf16 ? 2 : 4, dt = padded(a.D), nt = tiles(a);
    if (3 * a.sm_count > kAttendTickets) return cudaErrorInvalidConfiguration;
    AttendParams p{};
    p.B = a.B; p.Hk = a.Hk; p.G = a.G; p.D = a.D;
    p.groups = (a.G + 8 * nt - 1) / (8 * nt);
    p.page = (int)a.cache.page;
    p.width = a.width;
    divider((uint32_t)p.page, &p.page_mul, &p.page_shift);
    p.chunk_mul = 65536 / (a.D / 16) + 1;      // above 2^16 / chunks by at most 1
    p.whole = p.page % kStrip == 0;
    p.window = a.window;
    p.scale_log2 = a.scale * kLog2e;
    p.q = a.q.p; p.q_ld = a.q.ld; p.q_hs = a.q.hs; p.q_vec = aligned16(a.q, es);
    p.out = a.out.p; p.o_ld = a.out.ld; p.o_hs = a.out.hs; p.o_vec = aligned16(a.out, es);
    p.k = a.cache.k; p.v = a.cache.v; p.ks = a.cache.k_scale; p.vs = a.cache.v_scale;
    p.k_stride = a.cache.k_stride; p.v_stride = a.cache.v_stride;
    p.ks_stride = a.cache.k_scale_stride; p.vs_stride = a.cache.v_scale_stride;
    p.blocks = a.cache.blocks;
    p.table = a.table; p.ld_table = a.ld_table; p.lens = a.lens;
    p.lse = a.lse;
    p.parts = static_cast<float *>(workspace);
    p.tickets = tickets;
    p.err = a.err;
    switch (dt) {
        case 64: return launch_attend_64(p, a.type, nt, a.sm_count, a.stream);
        case 96: return launch_attend_96(p, a.type, nt, a.sm_count, a.stream);
        case 128: return launch_attend_128(p, a.type, nt, a.sm_count, a.stream);
        case 192: return launch_attend_192(p, a.type, nt, a.sm_count, a.stream);
        default: return launch_attend_256(p, a.type, nt, a.sm_count, a.stream);
    }
}

}  // namespace sgemm_gb300
