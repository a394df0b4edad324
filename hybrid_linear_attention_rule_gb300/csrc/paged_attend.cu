// paged_attend.cu -- picks the paged attention's kernel (paged_attend.cuh) and lays out its workspace.
#include "paged_rows.cuh"

namespace k3kda {

#ifndef XR
#define XR 16
#endif
static constexpr int kRowsFrom = XR;

// whether blocks of 128 rows fit tensor memory
static bool wide_ok(int dqk, int dv) { return dqk <= 192 && dv <= 128; }

// Status word and counters, then two records a CTA: its first and its last (sequence, head, row block).  One size for all
// shapes, that of the largest records, so that any call may follow any other in one workspace.
size_t paged_attend_workspace(int, int) {
    static_assert(128 * (128 + 2) >= attend::kMaxRows * (256 + 2), "the largest record");
    return attend::kHeadBytes + (size_t)attend::kMaxCtas * 2 * 128 * (128 + 2) * sizeof(float);
}

cudaError_t launch_paged_attend(const k3mla_paged_cache *c, const k3mla_view *q, int bf16, int Hq, const int32_t *cu, int T,
                                int max_new, const k3mla_rope_args *rope, float scale, const k3mla_view *gate, void *out,
                                int out_bf16, void *ws, cudaStream_t s) {
    attend::Args A;
    A.P = make_paged(c);
    A.q = make_view(q);
    A.gate = make_view(gate);
    A.in_bf16 = bf16; A.out_bf16 = out_bf16; A.Hq = Hq; A.G = Hq / c->heads; A.T = T;
    A.cu = cu;
    A.r = make_rope(rope);
    A.qmul = scale * 1.4426950408889634f;
    A.per_page = c->page_size / kStrip;
    A.per_page_inv = A.per_page > 1 ? (unsigned)(((1ull << 32) + A.per_page - 1) / A.per_page) : 0;
    A.out = out;
    A.status = static_cast<unsigned *>(ws);
    A.counters = A.status + 64;
    A.partial = reinterpret_cast<float *>(static_cast<char *>(ws) + attend::kHeadBytes);
    if (!cu) max_new = 1;
    // Four rows at a time where no sequence has more (half the products and registers), else eight; from kRowsFrom rows on blocks
    // of 128 on tcgen05, whose rows beyond the sequence's cost nothing more.
    const long long rows = (long long)max_new * A.G;
    const bool i4 = c->format == K3MLA_CACHE_I4;
    if (rows > kRowsFrom && wide_ok(c->dqk, c->dv)) return i4 ? attend::run_i4_rows(c->dqk, c->dv, A, s) : attend::run_bf16_rows(c->dqk, c->dv, A, s);
    if (i4) return rows <= 4 ? attend::run_i4_r4(c->dqk, c->dv, A, max_new, s) : attend::run_i4_r8(c->dqk, c->dv, A, max_new, s);
    return rows <= 4 ? attend::run_bf16_r4(c->dqk, c->dv, A, max_new, s) : attend::run_bf16_r8(c->dqk, c->dv, A, max_new, s);
}

}  // namespace k3kda
