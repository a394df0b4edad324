// rope.cuh -- the rotary rotation's device helpers and host-side argument forms, shared by the
// rotation kernels (rope.cu) and the paged cache's (paged_append.cu, paged_attend.cu).
#pragma once

#include "common.cuh"

namespace k3kda {

// A pair table as the kernels take it; dim = 0: nothing is turned.
struct Rope {
    const uint64_t *phase;
    int dim, off, half, inter;
    float mscale;
};

inline Rope make_rope(const k3mla_rope_args *r) {
    Rope o{nullptr, 0, 0, 0, 0, 1.f};
    if (r && r->dim > 0) {
        o.phase = r->phase; o.dim = r->dim; o.off = r->offset; o.half = r->dim / 2;
        o.inter = r->layout == K3MLA_ROPE_INTERLEAVED; o.mscale = r->mscale;
    }
    return o;
}

struct View {
    char *p;
    int64_t ts, hs;          // strides in elements
};

inline View make_view(const k3mla_view *v) {
    return v ? View{static_cast<char *>(v->data), v->token_stride, v->head_stride} : View{nullptr, 0, 0};
}

// Every row of the view starts on a 16-byte boundary.
inline bool view_vec(const k3mla_view *v, int size, int T, int H) {
    if ((reinterpret_cast<uintptr_t>(v->data) & 15u) != 0) return false;
    if (T > 1 && (v->token_stride * size) % 16 != 0) return false;
    return !(H > 1 && (v->head_stride * size) % 16 != 0);
}

// The turn of `pos` positions in units of 2^-64: the product modulo 2^64 is the fraction of a turn,
// exact but for the phase's own rounding (2^-53 of it), whatever the position.
__device__ __forceinline__ uint64_t rope_turn(uint64_t phase, int pos) { return phase * (uint64_t)(int64_t)pos; }

// (cos, sin) in FP32: the nearest quarter turn is taken out exactly, the rest (at most 1/8 turn) has
// 2^-24 relative accuracy from its top 32 bits.
__device__ __forceinline__ float2 rope_cs(uint64_t phase, int pos) {
    const uint64_t t = rope_turn(phase, pos);
    const unsigned quarter = (unsigned)((t + (1ull << 61)) >> 62);
    const int rest = (int)(int64_t)((t - ((uint64_t)quarter << 62)) >> 32);
    float s, c;
    sincospif((float)rest * 4.656612873077393e-10f, &s, &c);     // half turns = rest * 2^-31
    const float cq = (quarter & 1) ? s : c, sq = (quarter & 1) ? c : s;
    return make_float2((quarter == 1 || quarter == 2) ? -cq : cq, (quarter & 2) ? -sq : sq);
}

__device__ __forceinline__ void rope_cs_f64(uint64_t phase, int pos, double &c, double &s) {
    sincospi((double)(int64_t)rope_turn(phase, pos) * 1.0842021724855044e-19, &s, &c);     // 2^-63
}

}  // namespace k3kda
