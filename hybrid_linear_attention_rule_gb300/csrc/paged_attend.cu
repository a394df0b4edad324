// paged_attend.cu -- picks the paged attention's kernel (paged_attend.cuh) and lays out its workspace.
#include "paged_rows.cuh"

namespace k3kda {

// From how many query rows of a key head on blocks of 128 rows take over from blocks of 8.  The latter's time grows with every
// 8 rows, the former's hardly up to 128, and the wider keys are the more its products gain.  Measured in us, 8-row blocks against
// 128-row blocks: 4-bit pages of 128 + 128 channels, 32 sequences of 4000 keys, 4 heads: 90 / 106 at 32 rows, 109 / 108 at 40,
// 126 / 108 at 48; one sequence of 60,000, 8 heads: 83 / 95 at 32, 97 / 99 at 40, 115 / 100 at 48; 16 sequences of 4000 with 64 + 64
// channels 41 / 47 at 40, 48 / 47 at 48, with 192 + 128 78 / 91 at 24, 96 / 92 at 32.  bf16 pages, 32 sequences of 4000: 57 / 85 at 8 rows,
// 95 / 86 at 12; one of 60,000: 69 / 78 at 8, 86 / 80 at 12; 64 of 300: 46 / 52 at 12, 61 / 55 at 24.
static int rows_from(bool i4, int dqk) { return i4 ? 52 - dqk / 8 : 8; }

// whether blocks of 128 rows fit tensor memory
static bool wide_ok(int dqk, int dv) { return dqk <= 192 && dv <= 128; }

// Which kernel takes a call: four rows at a time where no sequence has more (half the products and registers), else eight, else
// blocks of 128 on tcgen05.
static int rows_at_once(bool i4, int dqk, int dv, long long rows) {
    return rows > rows_from(i4, dqk) && wide_ok(dqk, dv) ? 128 : rows <= 4 ? 4 : 8;
}

// What the call's units (paged_attend.cuh) cannot exceed, whatever the lengths are: every row block of every sequence with the tiles of
// the whole table, one block begun for each sequence that has a token.  The kernels count them in 31 bits.
double paged_attend_units(const k3mla_paged_cache *c, int G, int T, int max_new, bool packed) {
    const bool i4 = c->format == K3MLA_CACHE_I4;
    const int rows = rows_at_once(i4, c->dqk, c->dv, (long long)(packed ? max_new : 1) * G);
    const int tile = rows == 128 ? attend::kRowsTile : attend::few_strips(i4, (c->dqk + c->dv) / 64) * kStrip;
    const int extra = rows == 128 ? attend::kRowsExtra : attend::kExtra;
    const long long width = (long long)c->max_pages * c->page_size, tiles = width > tile ? (width + tile - 1) / tile : 1;
    const double blocks = (double)((long long)T * G / rows) + (T < c->N ? T : c->N);
    return blocks * c->heads * (double)(tiles + extra);
}

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
    const bool i4 = c->format == K3MLA_CACHE_I4;
    const int rows = rows_at_once(i4, c->dqk, c->dv, (long long)max_new * A.G);
    A.test_limit = rows == 128 ? take_paged_test_timeout() : 0;
    if (rows == 128) return i4 ? attend::run_i4_rows(c->dqk, c->dv, A, s) : attend::run_bf16_rows(c->dqk, c->dv, A, s);
    if (i4) return rows == 4 ? attend::run_i4_r4(c->dqk, c->dv, A, max_new, s) : attend::run_i4_r8(c->dqk, c->dv, A, max_new, s);
    return rows == 4 ? attend::run_bf16_r4(c->dqk, c->dv, A, max_new, s) : attend::run_bf16_r8(c->dqk, c->dv, A, max_new, s);
}

}  // namespace k3kda
