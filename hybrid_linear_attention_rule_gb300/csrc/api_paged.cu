// api_paged.cu -- the C ABI of the rotary positions and the paged cache (declared in include/k3kda.h):
// argument checks on the host, then one launch on the caller's stream.  Nothing here allocates,
// synchronises, throws or prints.
#include <math.h>

#include "common.cuh"

using namespace k3kda;

namespace {

std::atomic<unsigned> g_paged_test_timeout{0};

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool type_ok(int t) { return t == K3KDA_F32 || t == K3KDA_BF16; }
int size_of(int t) { return t == K3KDA_BF16 ? 2 : 4; }

// A [T, H, *] view to read, or to write (then no two of its rows may be the same).
int check_view(const k3mla_view *v, int dtype, int T, int H, bool write) {
    if (!v || !v->data || v->token_stride < 0 || v->head_stride < 0) return K3KDA_ERR_INVALID_ARG;
    if (write && ((T > 1 && v->token_stride == 0) || (H > 1 && v->head_stride == 0))) return K3KDA_ERR_INVALID_ARG;
    return aligned(v->data, (uintptr_t)size_of(dtype)) ? K3KDA_OK : K3KDA_ERR_ALIGNMENT;
}

// rope: the table of a head of d channels; NULL or dim 0: nothing is turned.
int check_rope(const k3mla_rope_args *r, int d) {
    if (!r || r->dim == 0) return K3KDA_OK;
    if (r->dim < 0 || (r->dim & 1) || r->dim > 512 || r->offset < 0 || r->offset > d - r->dim) return K3KDA_ERR_INVALID_ARG;
    if (r->layout != K3MLA_ROPE_HALF && r->layout != K3MLA_ROPE_INTERLEAVED) return K3KDA_ERR_INVALID_ARG;
    if (!r->phase || !isfinite(r->mscale)) return K3KDA_ERR_INVALID_ARG;
    return aligned(r->phase, 8) ? K3KDA_OK : K3KDA_ERR_ALIGNMENT;
}

int rope_impl(const k3mla_view *q, const k3mla_view *q_out, int Hq, const k3mla_view *k, const k3mla_view *k_out, int Hk,
              int shared, int dtype, const int32_t *pos, int T, int d, const k3mla_rope_args *rope, float sgn, void *stream) {
    if (T < 0 || Hq < 0 || Hk < 0 || Hq + (long long)Hk < 1 || !type_ok(dtype) || !rope) return K3KDA_ERR_INVALID_ARG;
    if (shared && Hk < 1) return K3KDA_ERR_INVALID_ARG;
    if (d < 1 || d > 1024) return K3KDA_ERR_UNSUPPORTED;
    if (int e = check_rope(rope, d)) return e;
    if ((Hq == 0) != (!q && !q_out) || (Hk == 0) != (!k && !k_out)) return K3KDA_ERR_INVALID_ARG;
    if (((long long)Hq + Hk) * d > (1 << 24)) return K3KDA_ERR_UNSUPPORTED;
    if (T == 0) return K3KDA_OK;
    if (!pos) return K3KDA_ERR_INVALID_ARG;
    if (Hq) {
        if (int e = check_view(q, dtype, T, Hq, false)) return e;
        if (int e = check_view(q_out, dtype, T, Hq, true)) return e;
    }
    if (Hk) {
        if (int e = check_view(k, dtype, T, Hk, false)) return e;
        if (int e = check_view(k_out, dtype, T, shared ? 1 : Hk, true)) return e;
        if (shared && k->data == k_out->data) return K3KDA_ERR_INVALID_ARG;
    }
    if (!aligned(pos, 4)) return K3KDA_ERR_ALIGNMENT;
    return status_of(launch_rope(q, q_out, Hq, k, k_out, Hk, shared, dtype == K3KDA_BF16, pos, T, d, rope, sgn,
                                 static_cast<cudaStream_t>(stream)));
}

bool dims_ok(int dqk, int dv) {
    return (dqk == 64 || dqk == 128 || dqk == 192 || dqk == 256) && (dv == 64 || dv == 128 || dv == 256);
}
bool page_ok(int page_size) { return page_size >= 16 && page_size <= 256 && page_size % 16 == 0; }

// The cache and the packing of T new tokens.
int check_cache(const k3mla_paged_cache *c, const int32_t *cu, const int32_t *cu_host, int T) {
    if (!c || c->N < 0 || c->heads < 1 || c->num_pages < 0 || c->max_pages < 0 || T < 0) return K3KDA_ERR_INVALID_ARG;
    if (c->format != K3MLA_CACHE_BF16 && c->format != K3MLA_CACHE_I4) return K3KDA_ERR_INVALID_ARG;
    if (!dims_ok(c->dqk, c->dv) || !page_ok(c->page_size) || c->heads > 65536) return K3KDA_ERR_UNSUPPORTED;
    // (positions and the ends of their tiles are counted in 31 bits)
    if ((long long)c->max_pages * c->page_size > (1LL << 31) - 256) return K3KDA_ERR_UNSUPPORTED;
    if (T > 0 && c->N == 0) return K3KDA_ERR_INVALID_ARG;
    if (!cu && T != c->N) return K3KDA_ERR_INVALID_ARG;
    if (cu_host) {
        if (cu_host[0] != 0 || cu_host[c->N] != T) return K3KDA_ERR_INVALID_ARG;
        for (int n = 0; n < c->N; ++n)
            if (cu_host[n + 1] < cu_host[n] || (!cu && cu_host[n + 1] != n + 1)) return K3KDA_ERR_INVALID_ARG;
    }
    if (c->kv_len_host)
        for (int n = 0; n < c->N; ++n) {
            const int len = c->kv_len_host[n];
            if (len < 0 || len > (long long)c->max_pages * c->page_size) return K3KDA_ERR_INVALID_ARG;
            if (cu_host && len < cu_host[n + 1] - cu_host[n]) return K3KDA_ERR_INVALID_ARG;
            if (!c->block_table_host) continue;
            for (int j = 0; j < (len + c->page_size - 1) / c->page_size; ++j) {
                const int page = c->block_table_host[(long long)n * c->max_pages + j];
                if (page < 0 || page >= c->num_pages) return K3KDA_ERR_INVALID_ARG;
            }
        }
    if (T == 0) return K3KDA_OK;
    if (!c->kv_len || (!c->pool && c->num_pages > 0) || (!c->block_table && c->max_pages > 0)) return K3KDA_ERR_INVALID_ARG;
    if (!aligned(c->pool, 16) || !aligned(c->block_table, 4) || !aligned(c->kv_len, 4) || !aligned(cu, 4)) return K3KDA_ERR_ALIGNMENT;
    return K3KDA_OK;
}

}  // namespace

unsigned k3kda::take_paged_test_timeout() { return g_paged_test_timeout.exchange(0u); }

extern "C" {

// Test hook, beside k3kda_test_arm_wait_timeout: the next attention in blocks of 128 rows asks for none of its first tile's
// copies in CTA 0, which gives up the wait for them after `tries` polls (0 disarms; a small call's CTA 0 may have no tile).  Only for tests on a working GPU: the armed call's outputs are
// invalid by design.
void k3kda_test_arm_paged_wait_timeout(unsigned tries) { g_paged_test_timeout.store(tries); }

int k3mla_rope_table(int dim, double theta, int scale_kind, double factor, double original_length, double beta_fast,
                     double beta_slow, uint64_t *phase_host, float *mscale) {
    if (dim < 2 || dim > 512 || (dim & 1) || !(theta > 0.0) || !isfinite(theta) || !phase_host || !mscale)
        return K3KDA_ERR_INVALID_ARG;
    if (scale_kind < K3MLA_SCALE_NONE || scale_kind > K3MLA_SCALE_BY_PARTS) return K3KDA_ERR_INVALID_ARG;
    if (scale_kind != K3MLA_SCALE_NONE && (!(factor > 0.0) || !isfinite(factor))) return K3KDA_ERR_INVALID_ARG;
    if (scale_kind == K3MLA_SCALE_NTK && dim == 2) return K3KDA_ERR_INVALID_ARG;
    if (scale_kind == K3MLA_SCALE_BY_PARTS &&
        (!(original_length > 0.0) || !isfinite(original_length) || !(beta_fast > beta_slow) || !isfinite(beta_fast - beta_slow)))
        return K3KDA_ERR_INVALID_ARG;
    constexpr double kTwoPi = 6.283185307179586476925286766559;
    const double base = scale_kind == K3MLA_SCALE_NTK ? theta * pow(factor, dim / (dim - 2.0)) : theta;
    for (int i = 0; i < dim / 2; ++i) {
        double f = pow(base, -2.0 * i / dim);
        if (scale_kind == K3MLA_SCALE_LINEAR) f /= factor;
        if (scale_kind == K3MLA_SCALE_BY_PARTS) {
            double g = (original_length * f / kTwoPi - beta_slow) / (beta_fast - beta_slow);
            g = g < 0.0 ? 0.0 : g > 1.0 ? 1.0 : g;
            f = f * g + f / factor * (1.0 - g);
        }
        // whole turns a position do not show; the rest is at most 2^64 - 2^11 after the product (53 bits)
        double turns = f / kTwoPi;
        if (!isfinite(turns)) return K3KDA_ERR_INVALID_ARG;
        turns -= floor(turns);
        phase_host[i] = (uint64_t)(turns * 18446744073709551616.0);
    }
    *mscale = scale_kind == K3MLA_SCALE_BY_PARTS ? (float)(0.1 * log(factor) + 1.0) : 1.f;
    return K3KDA_OK;
}

int k3mla_rope(const k3mla_view *q, const k3mla_view *q_out, int Hq, const k3mla_view *k, const k3mla_view *k_out, int Hk,
               int dtype, const int32_t *positions, int T, int d, const k3mla_rope_args *rope, void *stream) {
    return rope_impl(q, q_out, Hq, k, k_out, Hk, 0, dtype, positions, T, d, rope, 1.f, stream);
}

int k3mla_rope_backward(const k3mla_view *dq_out, const k3mla_view *dq, int Hq, const k3mla_view *dk_out, const k3mla_view *dk,
                        int Hk, int k_shared, int dtype, const int32_t *positions, int T, int d, const k3mla_rope_args *rope,
                        void *stream) {
    return rope_impl(dq_out, dq, Hq, dk_out, dk, Hk, k_shared != 0, dtype, positions, T, d, rope, -1.f, stream);
}

size_t k3mla_paged_block_bytes(int format, int page_size, int dqk, int dv) {
    if ((format != K3MLA_CACHE_BF16 && format != K3MLA_CACHE_I4) || !dims_ok(dqk, dv) || !page_ok(page_size)) return 0;
    return (size_t)(page_size / 16) * ((dqk + dv) / 64) * (format == K3MLA_CACHE_I4 ? 576 : 2048);
}

int k3mla_paged_append(const k3mla_paged_cache *cache, const k3mla_view *k_new, const k3mla_view *v_new, int in_dtype,
                       const int32_t *cu_seqlens, const int32_t *cu_seqlens_host, int T, const k3mla_rope_args *rope,
                       void *stream) {
    if (!type_ok(in_dtype)) return K3KDA_ERR_INVALID_ARG;
    if (int e = check_cache(cache, cu_seqlens, cu_seqlens_host, T)) return e;
    if (int e = check_rope(rope, cache->dqk)) return e;
    if (T == 0) return K3KDA_OK;
    if (int e = check_view(k_new, in_dtype, T, cache->heads, false)) return e;
    if (int e = check_view(v_new, in_dtype, T, cache->heads, false)) return e;
    return status_of(launch_paged_append(cache, k_new, v_new, in_dtype == K3KDA_BF16, cu_seqlens, T, rope,
                                         static_cast<cudaStream_t>(stream)));
}

int k3mla_paged_read(const k3mla_paged_cache *cache, const k3mla_view *k_out, const k3mla_view *v_out, int out_dtype,
                     const int32_t *cu_seqlens, const int32_t *cu_seqlens_host, int T, void *stream) {
    if (!type_ok(out_dtype)) return K3KDA_ERR_INVALID_ARG;
    if (int e = check_cache(cache, cu_seqlens, cu_seqlens_host, T)) return e;
    if (!k_out && !v_out) return K3KDA_ERR_INVALID_ARG;
    if (T == 0) return K3KDA_OK;
    if (k_out)
        if (int e = check_view(k_out, out_dtype, T, cache->heads, true)) return e;
    if (v_out)
        if (int e = check_view(v_out, out_dtype, T, cache->heads, true)) return e;
    return status_of(launch_paged_read(cache, k_out, v_out, out_dtype == K3KDA_BF16, cu_seqlens, T, static_cast<cudaStream_t>(stream)));
}

size_t k3mla_paged_attend_workspace_size(int Hq, int heads, int dqk, int dv) {
    if (heads < 1 || Hq < heads || Hq % heads != 0 || !dims_ok(dqk, dv)) return 0;
    return paged_attend_workspace(dqk, dv);
}

int k3mla_paged_attend(const k3mla_paged_cache *cache, const k3mla_view *q, int in_dtype, int Hq, const int32_t *cu_seqlens,
                       const int32_t *cu_seqlens_host, int T, int max_new, const k3mla_rope_args *rope, float scale,
                       const k3mla_view *gate, void *out, int out_dtype, void *workspace, size_t workspace_bytes, void *stream) {
    if (!type_ok(in_dtype) || !type_ok(out_dtype)) return K3KDA_ERR_INVALID_ARG;
    if (int e = check_cache(cache, cu_seqlens, cu_seqlens_host, T)) return e;
    if (Hq < 1 || Hq % cache->heads != 0 || max_new < 1 || !isfinite(scale)) return K3KDA_ERR_INVALID_ARG;
    if (Hq > 65536 || max_new > (1 << 24) || (long long)T * (Hq / cache->heads) > (1 << 28)) return K3KDA_ERR_UNSUPPORTED;
    if (cu_seqlens_host)
        for (int n = 0; n < cache->N; ++n)
            if (cu_seqlens_host[n + 1] - cu_seqlens_host[n] > max_new) return K3KDA_ERR_INVALID_ARG;
    if (paged_attend_units(cache, Hq / cache->heads, T, max_new, cu_seqlens != nullptr) > 2147483647.0) return K3KDA_ERR_UNSUPPORTED;
    if (int e = check_rope(rope, cache->dqk)) return e;
    if (T == 0) return K3KDA_OK;
    if (int e = check_view(q, in_dtype, T, Hq, false)) return e;
    if (gate)
        if (int e = check_view(gate, in_dtype, T, Hq, false)) return e;
    if (!out) return K3KDA_ERR_INVALID_ARG;
    if (!aligned(out, 16)) return K3KDA_ERR_ALIGNMENT;
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < paged_attend_workspace(cache->dqk, cache->dv)) return K3KDA_ERR_WORKSPACE;
    return status_of(launch_paged_attend(cache, q, in_dtype == K3KDA_BF16, Hq, cu_seqlens, T, max_new, rope, scale, gate, out,
                                         out_dtype == K3KDA_BF16, workspace, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
