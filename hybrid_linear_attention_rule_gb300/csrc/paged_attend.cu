// paged_attend.cu -- picks the paged attention's kernel (paged_attend.cuh) and lays out its workspace.
#include "paged_attend.cuh"

namespace k3kda {

// status word and counters, then two records a CTA: its first and its last (sequence, head, row block)
size_t paged_attend_workspace(int dv) {
    return attend::kHeadBytes + (size_t)attend::kMaxCtas * 2 * attend::kMaxRows * (dv + 2) * sizeof(float);
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
    // four rows at a time where no sequence has more (half the products and registers), else eight
    const bool four = (long long)max_new * A.G <= 4;
    if (c->format == K3MLA_CACHE_I4) return four ? attend::run_i4_r4(c->dqk, c->dv, A, max_new, s) : attend::run_i4_r8(c->dqk, c->dv, A, max_new, s);
    return four ? attend::run_bf16_r4(c->dqk, c->dv, A, max_new, s) : attend::run_bf16_r8(c->dqk, c->dv, A, max_new, s);
}

}  // namespace k3kda
