// api_lin.cu -- the C ABI of linear attention with a decay a head and of the norms around a block (declared in
// include/k3kda.h): argument checks on the host, then launches on the caller's stream.  Nothing here allocates on the
// device, synchronises, throws or prints.
#include <math.h>

#include <initializer_list>
#include <new>

#include "block_norm.cuh"
#include "lin.cuh"

using namespace k3kda;

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool type_ok(int t) { return t == K3KDA_F32 || t == K3KDA_BF16; }
bool dim_ok(int d) { return d >= 16 && d <= 128 && d % 16 == 0; }

// Sizes that every call of linear attention shares.  Rows and states are counted in 31 bits where a grid or a tensor map needs it.
int check_sizes(int N, int T, int Hk, int H, int dk, int dv) {
    if (N < 1 || T < 0 || Hk < 1 || H < 1 || H % Hk != 0) return K3KDA_ERR_INVALID_ARG;
    if (!dim_ok(dk) || !dim_ok(dv) || H > 65535 || T > 0x7fffffff - 128 || (long long)N * H > (1LL << 28)) return K3KDA_ERR_UNSUPPORTED;
    return K3KDA_OK;
}

int check_cu(const int32_t *cu, const int32_t *host, int N, int T) {
    if (host) {
        if (host[0] != 0 || host[N] != T) return K3KDA_ERR_INVALID_ARG;
        for (int n = 0; n < N; ++n)
            if (host[n + 1] < host[n]) return K3KDA_ERR_INVALID_ARG;
    }
    if (!cu && N != 1) return K3KDA_ERR_INVALID_ARG;
    return aligned(cu, 4) ? K3KDA_OK : K3KDA_ERR_ALIGNMENT;
}

int check_slots(const int32_t *idx, const int32_t *host, int N, int num_slots, int H) {
    if (!idx) return host ? K3KDA_ERR_INVALID_ARG : K3KDA_OK;
    if (num_slots < 1) return K3KDA_ERR_INVALID_ARG;
    if ((long long)num_slots * H > 0x7fffffffLL) return K3KDA_ERR_UNSUPPORTED;
    if (!aligned(idx, 4)) return K3KDA_ERR_ALIGNMENT;
    if (!host) return K3KDA_OK;
    unsigned char *seen = new (std::nothrow) unsigned char[(size_t)num_slots]();
    if (!seen) return K3KDA_ERR_INVALID_ARG;
    bool ok = true;
    for (int n = 0; n < N && ok; ++n) {
        ok = host[n] >= 0 && host[n] < num_slots && !seen[host[n]];
        if (ok) seen[host[n]] = 1;
    }
    delete[] seen;
    return ok ? K3KDA_OK : K3KDA_ERR_INVALID_ARG;
}

// An array of a call as memory, and whether two have a byte in common.
struct Span {
    const void *p;
    size_t bytes;
};
bool overlap(const Span &a, const Span &b) {
    if (!a.p || !b.p || !a.bytes || !b.bytes) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x <= y ? y - x < a.bytes : x - y < b.bytes;
}
// Whether what is written lies clear of the inputs, which other CTAs and later launches still read meanwhile, and of one another.
// `in_place`: an output may be an input of its size.
bool clear(std::initializer_list<Span> outputs, std::initializer_list<Span> inputs, bool in_place = false) {
    for (const Span *o = outputs.begin(); o != outputs.end(); ++o) {
        for (const Span &i : inputs)
            if (!(in_place && o->p == i.p && o->bytes == i.bytes) && overlap(*o, i)) return false;
        for (const Span *u = outputs.begin(); u != o; ++u)
            if (overlap(*o, *u)) return false;
    }
    return true;
}

// Whether an output is one of some arrays.
template <class... P> bool is_one_of(const void *out, const P *...p) { return out && ((out == (const void *)p) || ...); }

// Bytes of linear attention's arrays for T rows.
struct LinBytes {
    size_t key, state, rows, heads, T;
    LinBytes(int T_, int Hk, int H, int dk, int dv, int dtype)
        : key((size_t)T_ * Hk * dk * size(dtype)), state((size_t)H * dk * dv * 4), rows((size_t)T_ * H * dv), heads((size_t)H), T((size_t)T_) {}
    static size_t size(int dtype) { return dtype == K3KDA_BF16 ? 2 : 4; }
    size_t wide(int dtype) const { return rows * size(dtype); }
    size_t decays(int per_head) const { return (per_head ? 1 : T) * heads * 4; }
};

template <class... P> bool all16(const P *...p) { return (aligned(p, 16) && ...); }

}  // namespace

extern "C" {

size_t k3lin_prefill_workspace_size(int N, int T, int Hk, int H, int dk, int dv, int in_dtype) {
    if (check_sizes(N, T, Hk, H, dk, dv) != K3KDA_OK || !type_ok(in_dtype)) return 0;
    return lin_workspace(N, T, Hk, H, dk, dv, in_dtype == K3KDA_BF16, 0);
}

int k3lin_prefill(const void *q, const void *k, const void *v, int in_dtype, const float *g, int g_per_head,
                  const float *initial_state, const int32_t *state_idx, const int32_t *state_idx_host, int num_slots,
                  const int32_t *cu_seqlens, const int32_t *cu_seqlens_host, int N, int T, int Hk, int H, int dk, int dv,
                  float scale, void *out, int out_dtype, float *final_state, void *workspace, size_t workspace_bytes,
                  void *stream) {
    if (!type_ok(in_dtype) || !type_ok(out_dtype) || !isfinite(scale)) return K3KDA_ERR_INVALID_ARG;
    if (int e = check_sizes(N, T, Hk, H, dk, dv)) return e;
    if (int e = check_cu(cu_seqlens, cu_seqlens_host, N, T)) return e;
    if (int e = check_slots(state_idx, state_idx_host, N, num_slots, H)) return e;
    if (T > 0 && (!q || !k || !v || !out || !g)) return K3KDA_ERR_INVALID_ARG;
    if (!all16(q, k, v, out, initial_state, final_state) || !aligned(g, 4)) return K3KDA_ERR_ALIGNMENT;
    const size_t need = lin_workspace(N, T, Hk, H, dk, dv, in_dtype == K3KDA_BF16, 0);
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < need) return K3KDA_ERR_WORKSPACE;
    const LinBytes b(T, Hk, H, dk, dv, in_dtype);
    const size_t states = (state_idx ? (size_t)num_slots : (size_t)N) * b.state;
    if (!clear({{out, b.wide(out_dtype)}, {final_state, states}, {workspace, need}},
               {{q, b.key}, {k, b.key}, {v, b.wide(in_dtype)}, {g, b.decays(g_per_head)},
                {initial_state, initial_state == final_state ? 0 : states}, {cu_seqlens, ((size_t)N + 1) * 4}, {state_idx, (size_t)N * 4}}))
        return K3KDA_ERR_INVALID_ARG;
    const LinArgs a{q, k, v, in_dtype == K3KDA_BF16, g, g_per_head != 0, initial_state, state_idx, num_slots, cu_seqlens,
                    N, T, Hk, H, dk, dv, scale, workspace};
    return status_of(launch_lin_prefill(a, out, out_dtype == K3KDA_BF16, final_state, static_cast<cudaStream_t>(stream)));
}

int k3lin_decode_step(const void *q, const void *k, const void *v, int in_dtype, const float *g, int g_per_head, float *state,
                      const int32_t *state_idx, const int32_t *state_idx_host, int num_slots, int N, int Hk, int H, int dk,
                      int dv, float scale, void *out, int out_dtype, void *stream) {
    if (!type_ok(in_dtype) || !type_ok(out_dtype) || !isfinite(scale) || N < 0) return K3KDA_ERR_INVALID_ARG;
    if (int e = check_sizes(N > 0 ? N : 1, N, Hk, H, dk, dv)) return e;
    if (int e = check_slots(state_idx, state_idx_host, N, num_slots, H)) return e;
    if (N == 0) return K3KDA_OK;
    if (!q || !k || !v || !g || !state || !out) return K3KDA_ERR_INVALID_ARG;
    if (!all16(q, k, v, out, state) || !aligned(g, 4)) return K3KDA_ERR_ALIGNMENT;
    const LinBytes b(N, Hk, H, dk, dv, in_dtype);
    const Span held{state, (state_idx ? (size_t)num_slots : (size_t)N) * b.state};
    if (!clear({{out, b.wide(out_dtype)}, held},
               {{q, b.key}, {k, b.key}, {v, b.wide(in_dtype)}, {g, b.decays(g_per_head)}, {state_idx, (size_t)N * 4}}))
        return K3KDA_ERR_INVALID_ARG;
    return status_of(launch_lin_decode(q, k, v, in_dtype == K3KDA_BF16, g, g_per_head != 0, state, state_idx, num_slots, N, Hk, H,
                                       dk, dv, scale, out, out_dtype == K3KDA_BF16, static_cast<cudaStream_t>(stream)));
}

size_t k3lin_backward_workspace_size(int N, int T, int Hk, int H, int dk, int dv, int in_dtype) {
    if (check_sizes(N, T, Hk, H, dk, dv) != K3KDA_OK || !type_ok(in_dtype)) return 0;
    return lin_workspace(N, T, Hk, H, dk, dv, in_dtype == K3KDA_BF16, 1);
}

int k3lin_backward(const void *q, const void *k, const void *v, int in_dtype, const float *g, int g_per_head,
                   const float *initial_state, const int32_t *cu_seqlens, const int32_t *cu_seqlens_host, int N, int T, int Hk,
                   int H, int dk, int dv, float scale, const void *dO, const float *dS_final, void *dq, void *dk_out,
                   void *dv_out, float *dg, float *dS0, void *workspace, size_t workspace_bytes, void *stream) {
    if (!type_ok(in_dtype) || !isfinite(scale)) return K3KDA_ERR_INVALID_ARG;
    if (int e = check_sizes(N, T, Hk, H, dk, dv)) return e;
    if (int e = check_cu(cu_seqlens, cu_seqlens_host, N, T)) return e;
    if (T > 0 && (!q || !k || !v || !g || !dO || !dq || !dk_out || !dv_out)) return K3KDA_ERR_INVALID_ARG;
    if (!all16(q, k, v, dO, dq, dk_out, dv_out, initial_state, dS_final, dS0) || !aligned(g, 4) || !aligned(dg, 4))
        return K3KDA_ERR_ALIGNMENT;
    const size_t need = lin_workspace(N, T, Hk, H, dk, dv, in_dtype == K3KDA_BF16, 1);
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < need) return K3KDA_ERR_WORKSPACE;
    const LinBytes b(T, Hk, H, dk, dv, in_dtype);
    if (!clear({{dq, b.key}, {dk_out, b.key}, {dv_out, b.wide(in_dtype)}, {dg, b.decays(g_per_head)}, {dS0, (size_t)N * b.state}, {workspace, need}},
               {{q, b.key}, {k, b.key}, {v, b.wide(in_dtype)}, {dO, b.wide(in_dtype)}, {g, b.decays(g_per_head)},
                {initial_state, (size_t)N * b.state}, {dS_final, (size_t)N * b.state}, {cu_seqlens, ((size_t)N + 1) * 4}}))
        return K3KDA_ERR_INVALID_ARG;
    const LinArgs a{q, k, v, in_dtype == K3KDA_BF16, g, g_per_head != 0, initial_state, nullptr, 0, cu_seqlens,
                    N, T, Hk, H, dk, dv, scale, workspace};
    return status_of(launch_lin_backward(a, dO, dS_final, dq, dk_out, dv_out, dg, dS0, static_cast<cudaStream_t>(stream)));
}

int k3blk_norm(const void *x, int dtype, const void *residual, const void *gate, int gate_act, const float *post_weight,
               const float *pre_weight, long long rows, int D, float alpha, float eps, void *sum_out, void *out, void *stream) {
    if (!type_ok(dtype) || rows < 0 || D < 1 || !isfinite(alpha) || !(eps >= 0.f) || !isfinite(eps)) return K3KDA_ERR_INVALID_ARG;
    if (gate_act != K3BLK_GATE_SIGMOID && gate_act != K3BLK_GATE_SILU) return K3KDA_ERR_INVALID_ARG;
    if (D > blk::MOST_D || rows > 0x7fffffffLL) return K3KDA_ERR_UNSUPPORTED;
    if (rows == 0) return K3KDA_OK;
    if (!x || (pre_weight == nullptr) != (out == nullptr) || (!out && !sum_out)) return K3KDA_ERR_INVALID_ARG;
    const uintptr_t unit = dtype == K3KDA_BF16 ? 2 : 4;
    for (const void *p : {x, residual, gate, (const void *)sum_out, (const void *)out})
        if (!aligned(p, unit)) return K3KDA_ERR_ALIGNMENT;
    if (!aligned(post_weight, 4) || !aligned(pre_weight, 4)) return K3KDA_ERR_ALIGNMENT;
    const size_t size = (size_t)rows * D * unit, weight = (size_t)D * 4;
    if (!clear({{sum_out, size}, {out, size}}, {{x, size}, {residual, size}, {gate, size}}, true) ||
        !clear({{sum_out, size}, {out, size}}, {{post_weight, weight}, {pre_weight, weight}}))
        return K3KDA_ERR_INVALID_ARG;
    blk::Args a{};
    a.x = x;
    a.gate = gate;
    a.residual = residual;
    a.post = post_weight;
    a.pre = pre_weight;
    a.s = sum_out;
    a.y = out;
    a.rows = rows;
    a.D = D;
    a.silu = gate_act == K3BLK_GATE_SILU;
    a.alpha = alpha;
    a.eps = eps;
    return status_of(launch_blk_norm(a, dtype == K3KDA_BF16, false, static_cast<cudaStream_t>(stream)));
}

size_t k3blk_norm_backward_workspace_size(long long rows, int D) {
    if (rows < 0 || rows > 0x7fffffffLL || D < 1 || D > blk::MOST_D) return 0;
    const size_t n = blk_norm_workspace(rows, D);
    return n < 256 ? 256 : n;
}

int k3blk_norm_backward(const void *x, int dtype, const void *ds, const void *dy, const void *sum, const void *gate, int gate_act,
                        const float *post_weight, const float *pre_weight, long long rows, int D, float alpha, float eps, void *dx,
                        void *dresidual, void *dgate, float *dpost_weight, float *dpre_weight, void *workspace,
                        size_t workspace_bytes, void *stream) {
    if (!type_ok(dtype) || rows < 0 || D < 1 || !isfinite(alpha) || !(eps >= 0.f) || !isfinite(eps)) return K3KDA_ERR_INVALID_ARG;
    if (gate_act != K3BLK_GATE_SIGMOID && gate_act != K3BLK_GATE_SILU) return K3KDA_ERR_INVALID_ARG;
    if (D > blk::MOST_D || rows > 0x7fffffffLL) return K3KDA_ERR_UNSUPPORTED;
    if ((post_weight == nullptr) != (dpost_weight == nullptr) || (pre_weight == nullptr) != (dpre_weight == nullptr)) return K3KDA_ERR_INVALID_ARG;
    if (!aligned(post_weight, 4) || !aligned(pre_weight, 4) || !aligned(dpost_weight, 4) || !aligned(dpre_weight, 4)) return K3KDA_ERR_ALIGNMENT;
    if (rows > 0) {
        if (!ds || !dx || (pre_weight && (!sum || !dy)) || (gate == nullptr) != (dgate == nullptr)) return K3KDA_ERR_INVALID_ARG;
        if ((post_weight || gate) && !x) return K3KDA_ERR_INVALID_ARG;
    }
    const uintptr_t unit = dtype == K3KDA_BF16 ? 2 : 4;
    for (const void *p : {x, ds, dy, sum, gate, (const void *)dx, (const void *)dresidual, (const void *)dgate})
        if (!aligned(p, unit)) return K3KDA_ERR_ALIGNMENT;
    if ((dpost_weight || dpre_weight) && (!workspace || !aligned(workspace, 256) || workspace_bytes < blk_norm_workspace(rows, D)))
        return K3KDA_ERR_WORKSPACE;
    if (rows > 0 && is_one_of(dresidual, post_weight || gate ? x : nullptr, gate)) return K3KDA_ERR_INVALID_ARG;
    const size_t size = (size_t)rows * D * unit, weight = (size_t)D * 4, parts = dpost_weight || dpre_weight ? blk_norm_workspace(rows, D) : 0;
    const Span from_x{post_weight || gate ? x : nullptr, size}, from_sum{pre_weight ? sum : nullptr, size}, from_dy{pre_weight ? dy : nullptr, size};
    if (!clear({{dx, size}, {dresidual, size}, {dgate, size}}, {from_x, {ds, size}, from_dy, from_sum, {gate, size}}, true) ||
        !clear({{dpost_weight, weight}, {dpre_weight, weight}}, {{post_weight, weight}, {pre_weight, weight}}, true) ||
        !clear({{dx, size}, {dresidual, size}, {dgate, size}, {workspace, parts}, {dpost_weight, weight}, {dpre_weight, weight}}, {}) ||
        !clear({{dx, size}, {dresidual, size}, {dgate, size}, {workspace, parts}}, {{post_weight, weight}, {pre_weight, weight}}) ||
        !clear({{workspace, parts}, {dpost_weight, weight}, {dpre_weight, weight}}, {from_x, {ds, size}, from_dy, from_sum, {gate, size}}))
        return K3KDA_ERR_INVALID_ARG;
    blk::Args a{};
    a.x = post_weight || gate ? x : nullptr;
    a.gate = gate;
    a.s_in = sum;
    a.ds = ds;
    a.dy = dy;
    a.post = post_weight;
    a.pre = pre_weight;
    a.dx = dx;
    a.dgate = dgate;
    a.dresidual = dresidual;
    a.dpost = dpost_weight;
    a.dpre = dpre_weight;
    a.parts = static_cast<float *>(workspace);
    a.rows = rows;
    a.D = D;
    a.silu = gate_act == K3BLK_GATE_SILU;
    a.alpha = alpha;
    a.eps = eps;
    return status_of(launch_blk_norm(a, dtype == K3KDA_BF16, true, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
