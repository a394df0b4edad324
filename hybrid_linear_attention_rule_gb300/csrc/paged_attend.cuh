// paged_attend.cuh -- attention of new tokens over the paged cache on sm_103a, bf16 and 4-bit pages.
//
//   out_r = sum_j p_rj v_j / sum_j p_rj,   p_rj = exp2(s_rj - m_r),   s_rj = scale log2(e) q_r . k_j
//
// over the keys j that row r = (new token, query head of the key head's group) sees.  Decode is bound by the
// cache's bytes, so everything serves one pass over them:
//
// Work.  The unit is a tile of NS strips of 16 tokens of one (sequence, key head, row block); all units of the call
// stand in one row (sequence, head, row block, tile) that is cut into equal runs, one a warp, whatever
// the lengths are.  A warp streams its run through a ring of its own in shared memory (bulk copies of
// whole strips, page numbers fetched one tile ahead), with no barrier to the other warps.  A (sequence, head, row
// block) that several warps share is joined from their (max, sum, weighted values): in shared memory within
// a CTA, then by the CTA that finishes last, always in the row's order, so results do not depend on timing.
//
// Arithmetic.  With 4 to 8 query rows the products are matrix-vector shaped; a tcgen05 tile would hold 128 keys by
// 8 rows but needs its 16-bit operand in shared memory, four times the 4-bit bytes written and read
// again, more than shared memory's bandwidth next to 6.8 TB/s of codes.  So the codes go from shared memory to registers and to
// mma.m16n8k16 there: keys (then value channels) are its 16 rows, and its 8 columns are 4 query rows, each as
// a high and a low 16-bit part (22 bits together for fp16, 16 for bf16): S^T = K Q^T, O^T = V^T P^T.
//   4-bit codes become fp16 by one AND: code * 2^-24 is the denormal with those low bits, code * 2^-20 the one four
//   bits up; the powers of two go into Q (16 on the first) and into O.  So a group's scale and minimum are taken out
//   of the product: s = sum_g scale_g (q_g . code_g) + min_g sum(q_g), and likewise scale_g goes into P before its
//   split and sum_j p_j min_gj is kept in FP32.  S comes out with tokens on rows; movmatrix turns P to the operand.
//   The running maximum is that of s + log2(scale), which bounds p scale by 2^14: nothing overflows fp16
//   and what is far below it keeps 2^-38 of the largest weight.
// A tile's products start at 0 and are added to O in FP32 by fma (which also rescales O): tensor-core sums of
// few terms, ordinary rounding over the long axis.
#pragma once

#include "paged.cuh"
#include "tc_ptx.cuh"

namespace k3kda {
namespace attend {

constexpr int kMaxCtas = 608;                          // partials and counters of a workspace
constexpr size_t kHeadBytes = 256 + 4096;              // status word, counters (4 B a CTA)
constexpr int kMaxRows = 8;
constexpr unsigned kWaitTries = 1u << 22;              // each try suspends for a while: seconds in all
static_assert(kMaxCtas * 4 <= 4096, "counters");

struct Args {
    Paged P;
    View q, gate;
    int in_bf16, out_bf16, Hq, G, T;
    const int32_t *cu;
    Rope r;
    float qmul;                                        // scale * log2(e)
    void *out;
    unsigned *status, *counters;
    float *partial;                                    // [kMaxCtas][2] records
};

template <int DQK_, int DV_, int RT_, bool I4_> struct Shape {
    static constexpr int DQK = DQK_, DV = DV_, RT = RT_;
    static constexpr bool I4 = I4_;
    static constexpr int PK = DQK / 64, PV = DV / 64, PL = PK + PV;
    static constexpr int ROWS = 4 * RT;
    static constexpr int PLANE = I4 ? kPlaneI4 : kPlaneBf16, STRIP = PL * PLANE;
    static constexpr int NS = I4 ? (PL <= 2 ? 4 : 2) : (PL <= 2 ? 2 : 1);       // strips of a tile
    static constexpr int TILE = NS * kStrip, STAGE = NS * STRIP;
    static constexpr int WARPS = I4 ? (PL <= 4 ? (RT == 1 ? 12 : 8) : RT == 1 ? 8 : 4) : (PL <= 4 ? 6 : 4);
    static constexpr int QS = DQK + 8;                                          // floats between staged rows
    static constexpr int RECORD = ROWS * (DV + 2);                              // floats: m, l, O
    static constexpr int STAGED = ROWS * (QS + PK + 1);                         // floats: rows, their sums and exponents
    static constexpr int SLOT1 = RECORD > STAGED ? RECORD : STAGED;
    static constexpr int FIXED = ((RECORD + SLOT1) * 4 + 127) / 128 * 128;      // bytes of a warp beside its ring
    static constexpr int COMMON = 1024 + 2 * WARPS * 48 + (WARPS * 32 + 2) * 8; // barriers, segments, prefix sums
    static constexpr int ROOM = (232448 - 256 - COMMON) / WARPS / 128 * 128;
    static constexpr int FIT = (ROOM - FIXED) / STAGE;
    static constexpr int STAGES = FIT > 6 ? 6 : FIT;
    static_assert(STAGES >= 2 && STAGES * WARPS * 8 <= 1024 && STAGES * NS <= 32, "ring");
    static constexpr int WARP_BYTES = STAGES * STAGE + FIXED;
    static constexpr int SMEM = COMMON + WARPS * WARP_BYTES;
    static_assert(STAGE % 128 == 0 || (STAGES * STAGE) % 64 == 0, "alignment");
};

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1, bool f16) {
    if (f16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&a)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4t(uint32_t (&a)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// x as a pair of 16-bit parts, the high one in the low half
template <bool F16> __device__ __forceinline__ uint32_t split_pair(float x) {
    if constexpr (F16) {
        const __half hi = __float2half_rn(x);
        const __half2 p = __halves2half2(hi, __float2half_rn(x - __half2float(hi)));
        return *reinterpret_cast<const uint32_t *>(&p);
    } else {
        const __nv_bfloat16 hi = __float2bfloat16_rn(x);
        const __nv_bfloat162 p = __halves2bfloat162(hi, __float2bfloat16_rn(x - __bfloat162float(hi)));
        return *reinterpret_cast<const uint32_t *>(&p);
    }
}
// the high (part 0) or low parts of two values
template <bool F16> __device__ __forceinline__ uint32_t pack_part(float x, float y, int part) {
    const uint32_t a = split_pair<F16>(x), b = split_pair<F16>(y);
    return __byte_perm(a, b, part ? 0x7632 : 0x5410);
}

// one sequence's share of the work
struct Seq {
    int len, q0, cnt, tiles, rbs;
    __device__ __forceinline__ int64_t units(int heads) const { return (int64_t)tiles * rbs * heads; }
};
template <class S> __device__ __forceinline__ Seq load_seq(const Args &A, int n) {
    Seq s;
    int b = n, e = n + 1;
    if (A.cu) seq_bounds(A.cu, n, A.T, b, e);
    s.len = paged_len(A.P, n);
    s.q0 = b;
    s.cnt = e - b;
    s.tiles = s.len > 0 ? (s.len + S::TILE - 1) / S::TILE : 1;   // an empty or bad sequence still writes its rows
    s.rbs = (int)(((int64_t)s.cnt * A.G + S::ROWS - 1) / S::ROWS);
    return s;
}

// a place in the row of units
struct Cursor {
    int n, h, rb, t;
    Seq s;
    // one past the last key that any row of the block sees, and that its first row sees
    template <class S> __device__ __forceinline__ int seen_most(const Args &A) const {
        const int last = min(s.cnt - 1, (int)(((int64_t)(rb + 1) * S::ROWS - 1) / A.G));
        return s.len - s.cnt + last + 1;
    }
    template <class S> __device__ __forceinline__ int seen_least(const Args &A) const {
        return s.len - s.cnt + (int)((int64_t)rb * S::ROWS / A.G) + 1;
    }
    template <class S> __device__ __forceinline__ void advance(const Args &A) {
        if (++t < s.tiles) return;
        t = 0;
        if (++rb < s.rbs) return;
        rb = 0;
        if (++h < A.P.heads) return;
        h = 0;
        while (++n < A.P.N) {
            s = load_seq<S>(A, n);
            if (s.rbs > 0) return;
        }
    }
};

// out = O / l (* sigmoid(gate)) for 4 channels of row r of a block; l = 0: a row that saw nothing
template <class S> __device__ __forceinline__ void store4(const Args &A, const Cursor &c, int r, int ch, float4 o, float l) {
    const int64_t R = (int64_t)c.rb * S::ROWS + r;
    if (R >= (int64_t)c.s.cnt * A.G) return;
    const int i = (int)(R / A.G), hq = c.h * A.G + (int)(R - (int64_t)i * A.G);
    const float inv = l == 0.f ? 0.f : 1.f / l;
    float x[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
    if (A.gate.p) {
        const char *g = A.gate.p + ((int64_t)(c.s.q0 + i) * A.gate.ts + (int64_t)hq * A.gate.hs + ch) * (A.in_bf16 ? 2 : 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] *= sigmoidf_(load_elt(g, e, A.in_bf16));
    }
    const int64_t at = ((int64_t)(c.s.q0 + i) * A.Hq + hq) * S::DV + ch;
    if (A.out_bf16) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
        *reinterpret_cast<uint2 *>(reinterpret_cast<__nv_bfloat16 *>(A.out) + at) =
            make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    } else {
        *reinterpret_cast<float4 *>(reinterpret_cast<float *>(A.out) + at) = make_float4(x[0], x[1], x[2], x[3]);
    }
}

// The warp's registers for one row block.  Lane (g, t) = (lane / 4, lane % 4) holds row 4 rt + t.
template <class S> struct State {
    uint32_t qf[S::RT][S::PK][4][2];      // Q^T operand of each plane's four k-steps
    float qsum[S::RT][S::PK];             // 4-bit: sum of the row's q over each group
    float fac[S::RT];                     // 4-bit: undoes the powers of two in q and the codes
    int vis[S::RT];                       // keys the row sees
    float m[S::RT], l[S::RT];             // running maximum; this lane's share of the sum
    float mn[S::RT][S::PV];               // 4-bit: this lane's share of sum_j p_j minimum_j
    float o[S::RT][S::PV][4][2];
};

// Rows of a block: loaded, rotated, scaled, split and laid out as the operand.
template <class S> __device__ __forceinline__ void load_rows(const Args &A, const Cursor &c, float *qs, State<S> &st) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int64_t rows = (int64_t)c.s.cnt * A.G, R0 = (int64_t)c.rb * S::ROWS;
    const int size = A.in_bf16 ? 2 : 4;
    __syncwarp();
#pragma unroll
    for (int r = 0; r < S::ROWS; ++r) {
        const bool ok = R0 + r < rows;
        const int i = ok ? (int)((R0 + r) / A.G) : 0, hq = c.h * A.G + (ok ? (int)((R0 + r) - (int64_t)i * A.G) : 0);
        const char *src = A.q.p + ((int64_t)(c.s.q0 + i) * A.q.ts + (int64_t)hq * A.q.hs) * size;
#pragma unroll
        for (int k = 0; k < S::DQK / 32; ++k)
            qs[r * S::QS + lane + 32 * k] = ok ? load_elt(src, lane + 32 * k, A.in_bf16) * A.qmul : 0.f;
    }
    __syncwarp();
    if (A.r.dim > 0) {
        for (int x = lane; x < S::ROWS * A.r.half; x += 32) {
            const int r = x / A.r.half, p = x - r * A.r.half;
            if (R0 + r >= rows) continue;
            const int pos = c.s.len - c.s.cnt + (int)((R0 + r) / A.G);
            const float2 cs = rope_cs(A.r.phase[p], pos);
            float *a = qs + r * S::QS + A.r.off + (A.r.inter ? 2 * p : p), *b = a + (A.r.inter ? 1 : A.r.half);
            const float u = *a * A.r.mscale, v = *b * A.r.mscale;
            *a = u * cs.x - v * cs.y;
            *b = v * cs.x + u * cs.y;
        }
        __syncwarp();
    }
    float *info = qs + S::ROWS * S::QS;                  // [ROWS][PK sums, largest magnitude]
    if constexpr (S::I4) {
#pragma unroll
        for (int rt = 0; rt < S::RT; ++rt) {
            const int r = 4 * rt + (lane >> 3);
            float big = 0.f;
#pragma unroll
            for (int p = 0; p < S::PK; ++p) {
                float sum = 0.f;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float x = qs[r * S::QS + 64 * p + 8 * k + (lane & 7)];
                    sum += x;
                    big = fmaxf(big, fabsf(x));
                }
#pragma unroll
                for (int o = 1; o < 8; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                if ((lane & 7) == 0) info[r * (S::PK + 1) + p] = sum;
            }
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
            if ((lane & 7) == 0) info[r * (S::PK + 1) + S::PK] = big;
        }
        __syncwarp();
    }
#pragma unroll
    for (int rt = 0; rt < S::RT; ++rt) {
        const int64_t R = R0 + 4 * rt + t;
        st.vis[rt] = R < rows ? c.s.len - c.s.cnt + (int)(R / A.G) + 1 : 0;
        st.m[rt] = -INFINITY;
        st.l[rt] = 0.f;
#pragma unroll
        for (int p = 0; p < S::PV; ++p) {
            st.mn[rt][p] = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) st.o[rt][p][j][0] = st.o[rt][p][j][1] = 0.f;
        }
        const float *row = qs + (4 * rt + (g >> 1)) * S::QS;
        float mul = 1.f;
        if constexpr (S::I4) {
            // 2^e brings the row's largest magnitude to [2^9, 2^10)
            auto exponent = [&](int r) {
                const int x = (int)(__float_as_uint(info[r * (S::PK + 1) + S::PK]) >> 23) - 127;
                return min(max(9 - x, -100), 120);
            };
            mul = __int_as_float((exponent(4 * rt + (g >> 1)) + 127) << 23);
            st.fac[rt] = __int_as_float((20 - exponent(4 * rt + t) + 127) << 23);
#pragma unroll
            for (int p = 0; p < S::PK; ++p) st.qsum[rt][p] = info[(4 * rt + t) * (S::PK + 1) + p];
        }
#pragma unroll
        for (int p = 0; p < S::PK; ++p)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (S::I4) {
                    const float *x = row + 64 * p + 16 * t + (i >> 1) * 8 + (i & 1) * 2;
                    st.qf[rt][p][i][0] = pack_part<true>(x[0] * mul * 16.f, x[4] * mul * 16.f, g & 1);
                    st.qf[rt][p][i][1] = pack_part<true>(x[1] * mul, x[5] * mul, g & 1);
                } else {
                    const float *x = row + 64 * p + 16 * i + 2 * t;
                    st.qf[rt][p][i][0] = pack_part<false>(x[0], x[1], g & 1);
                    st.qf[rt][p][i][1] = pack_part<false>(x[8], x[9], g & 1);
                }
            }
    }
    __syncwarp();
}

// Token of row r of an 8-row block of the 4-bit products: an order in which both the key rows that four lanes
// read together and the value rows do lie in different banks.
__device__ __forceinline__ int order8(int r) { return r ^ (r >> 2); }

// One tile.  j0: its first token; bad: strips on pages outside the pool.  MASK: some row does not see all of it.
template <class S, bool MASK> __device__ __forceinline__ void tile(const Args &A, const char *stage, int j0, int len, unsigned bad, State<S> &st) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int ta = S::I4 ? order8(g) : g;                // this lane's tokens of a strip: ta and ta + 8
    float p[S::NS][S::RT][2];
    [[maybe_unused]] __half2 vp[S::NS][S::PV][2];        // 4-bit: (scale, minimum) of the value groups
    float top[S::RT];
#pragma unroll
    for (int rt = 0; rt < S::RT; ++rt) top[rt] = -INFINITY;
#pragma unroll
    for (int s = 0; s < S::NS; ++s) {
        const char *sp = stage + s * S::STRIP;
        const int ja = j0 + 16 * s + ta;
        float e0 = 0.f, e1 = 0.f;
        if constexpr (S::I4) {
            float ps[S::RT][2], pm[S::RT][2];
#pragma unroll
            for (int rt = 0; rt < S::RT; ++rt) ps[rt][0] = ps[rt][1] = pm[rt][0] = pm[rt][1] = 0.f;
#pragma unroll
            for (int k = 0; k < S::PK; ++k) {
                const char *pl = sp + k * kPlaneI4;
                const uint2 wa = *reinterpret_cast<const uint2 *>(pl + ta * 32 + 8 * t);
                const uint2 wb = *reinterpret_cast<const uint2 *>(pl + ta * 32 + 256 + 8 * t);
                const float2 ka = __half22float2(*reinterpret_cast<const __half2 *>(pl + 512 + ta * 4));
                const float2 kb = __half22float2(*reinterpret_cast<const __half2 *>(pl + 544 + ta * 4));
                float c[S::RT][4];
#pragma unroll
                for (int rt = 0; rt < S::RT; ++rt) c[rt][0] = c[rt][1] = c[rt][2] = c[rt][3] = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t ua = (i < 2 ? wa.x : wa.y) >> (8 * (i & 1)), ub = (i < 2 ? wb.x : wb.y) >> (8 * (i & 1));
#pragma unroll
                    for (int rt = 0; rt < S::RT; ++rt)
                        mma(c[rt], ua & 0x000F000Fu, ub & 0x000F000Fu, ua & 0x00F000F0u, ub & 0x00F000F0u, st.qf[rt][k][i][0],
                            st.qf[rt][k][i][1], true);
                }
#pragma unroll
                for (int rt = 0; rt < S::RT; ++rt) {
                    ps[rt][0] = fmaf(ka.x, c[rt][0] + c[rt][1], ps[rt][0]);
                    ps[rt][1] = fmaf(kb.x, c[rt][2] + c[rt][3], ps[rt][1]);
                    pm[rt][0] = fmaf(ka.y, st.qsum[rt][k], pm[rt][0]);
                    pm[rt][1] = fmaf(kb.y, st.qsum[rt][k], pm[rt][1]);
                }
            }
            __half2 big0 = __float2half2_rn(0.f), big1 = big0;
#pragma unroll
            for (int v = 0; v < S::PV; ++v) {
                const char *pl = sp + (S::PK + v) * kPlaneI4;
                vp[s][v][0] = *reinterpret_cast<const __half2 *>(pl + 512 + ta * 4);
                vp[s][v][1] = *reinterpret_cast<const __half2 *>(pl + 544 + ta * 4);
                if (MASK) {                              // rows past the length hold anything, a NaN too
                    if (ja >= len) vp[s][v][0] = __float2half2_rn(0.f);
                    if (ja + 8 >= len) vp[s][v][1] = __float2half2_rn(0.f);
                }
                big0 = __hmax2(big0, vp[s][v][0]);
                big1 = __hmax2(big1, vp[s][v][1]);
            }
            // exponents of the largest scales (2^-24 at least): scale < 2^e
            e0 = (float)((int)(__float_as_uint(fmaxf(__low2float(big0), 5.9604645e-8f)) >> 23) - 126);
            e1 = (float)((int)(__float_as_uint(fmaxf(__low2float(big1), 5.9604645e-8f)) >> 23) - 126);
#pragma unroll
            for (int rt = 0; rt < S::RT; ++rt) {
                p[s][rt][0] = fmaf(ps[rt][0], st.fac[rt], pm[rt][0]);
                p[s][rt][1] = fmaf(ps[rt][1], st.fac[rt], pm[rt][1]);
            }
        } else {
            float c[S::RT][4];
#pragma unroll
            for (int rt = 0; rt < S::RT; ++rt) c[rt][0] = c[rt][1] = c[rt][2] = c[rt][3] = 0.f;
            const int tok = lane & 15, odd = lane >> 4;
#pragma unroll
            for (int k = 0; k < S::PK; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t a[4];
                    ldmatrix4(a, tc::smem_u32(sp + k * kPlaneBf16 + tok * 128 + (((2 * i + odd) ^ (tok & 7)) << 4)));
#pragma unroll
                    for (int rt = 0; rt < S::RT; ++rt)
                        mma(c[rt], a[0], a[1], a[2], a[3], st.qf[rt][k][i][0], st.qf[rt][k][i][1], false);
                }
#pragma unroll
            for (int rt = 0; rt < S::RT; ++rt) {
                // an infinite key: the low part's product may be the opposite infinity
                p[s][rt][0] = fabsf(c[rt][0]) < INFINITY ? c[rt][0] + c[rt][1] : c[rt][0];
                p[s][rt][1] = fabsf(c[rt][2]) < INFINITY ? c[rt][2] + c[rt][3] : c[rt][2];
            }
        }
#pragma unroll
        for (int rt = 0; rt < S::RT; ++rt) {
            if (MASK) {
                if ((bad >> s) & 1) p[s][rt][0] = p[s][rt][1] = __int_as_float(0x7fc00000);
                if (ja >= st.vis[rt]) p[s][rt][0] = -INFINITY;
                if (ja + 8 >= st.vis[rt]) p[s][rt][1] = -INFINITY;
            }
            top[rt] = fmaxf(top[rt], fmaxf(p[s][rt][0] + e0, p[s][rt][1] + e1));
        }
    }
    float corr[S::RT];
#pragma unroll
    for (int rt = 0; rt < S::RT; ++rt) {
        top[rt] = fmaxf(top[rt], __shfl_xor_sync(0xffffffffu, top[rt], 4));
        top[rt] = fmaxf(top[rt], __shfl_xor_sync(0xffffffffu, top[rt], 8));
        top[rt] = fmaxf(top[rt], __shfl_xor_sync(0xffffffffu, top[rt], 16));
        const float m = fmaxf(st.m[rt], S::I4 ? top[rt] - 14.f : top[rt]);
        const float base = m == -INFINITY ? 0.f : m;
        corr[rt] = ex2(st.m[rt] - base);
        st.m[rt] = m;
        float l = st.l[rt] * corr[rt];
#pragma unroll
        for (int s = 0; s < S::NS; ++s) {
            p[s][rt][0] = ex2(p[s][rt][0] - base);
            p[s][rt][1] = ex2(p[s][rt][1] - base);
            l += p[s][rt][0] + p[s][rt][1];
        }
        st.l[rt] = l;
    }
#pragma unroll
    for (int v = 0; v < S::PV; ++v) {
        if constexpr (S::I4) {
            uint32_t b[S::NS][S::RT][2];
#pragma unroll
            for (int rt = 0; rt < S::RT; ++rt) {
                float mn = st.mn[rt][v] * corr[rt];
#pragma unroll
                for (int s = 0; s < S::NS; ++s)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        float2 q = __half22float2(vp[s][v][x]);
                        // a key the row does not see weighs 0 even against a NaN
                        if (MASK && j0 + 16 * s + ta + 8 * x >= st.vis[rt]) q = make_float2(0.f, 0.f);
                        mn = fmaf(p[s][rt][x], q.y, mn);
                        b[s][rt][x] = transpose8x8(split_pair<true>(p[s][rt][x] * q.x));
                    }
                st.mn[rt][v] = mn;
            }
            uint32_t lo0[S::NS], hi0[S::NS], lo1[S::NS], hi1[S::NS];     // nibbles 0-3 and 4-7 of a token pair, a half each
#pragma unroll
            for (int s = 0; s < S::NS; ++s) {
                const char *pl = stage + s * S::STRIP + (S::PK + v) * kPlaneI4 + 4 * g;
                const int a = order8(2 * t) * 32, c = order8(2 * t + 1) * 32;
                const uint32_t wa = *reinterpret_cast<const uint32_t *>(pl + a), wb = *reinterpret_cast<const uint32_t *>(pl + c);
                const uint32_t wc = *reinterpret_cast<const uint32_t *>(pl + 256 + a), wd = *reinterpret_cast<const uint32_t *>(pl + 256 + c);
                lo0[s] = __byte_perm(wa, wb, 0x5410);
                hi0[s] = __byte_perm(wa, wb, 0x7632);
                lo1[s] = __byte_perm(wc, wd, 0x5410);
                hi1[s] = __byte_perm(wc, wd, 0x7632);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float c[S::RT][4];
#pragma unroll
                for (int rt = 0; rt < S::RT; ++rt) c[rt][0] = c[rt][1] = c[rt][2] = c[rt][3] = 0.f;
#pragma unroll
                for (int s = 0; s < S::NS; ++s) {
                    const uint32_t u0 = (j < 2 ? lo0[s] : hi0[s]) >> (8 * (j & 1)), u1 = (j < 2 ? lo1[s] : hi1[s]) >> (8 * (j & 1));
#pragma unroll
                    for (int rt = 0; rt < S::RT; ++rt)
                        mma(c[rt], u0 & 0x000F000Fu, u0 & 0x00F000F0u, u1 & 0x000F000Fu, u1 & 0x00F000F0u, b[s][rt][0], b[s][rt][1], true);
                }
#pragma unroll
                for (int rt = 0; rt < S::RT; ++rt) {
                    st.o[rt][v][j][0] = fmaf(st.o[rt][v][j][0], corr[rt], c[rt][0] + c[rt][1]);
                    st.o[rt][v][j][1] = fmaf(st.o[rt][v][j][1], corr[rt], c[rt][2] + c[rt][3]);
                }
            }
        } else {
            uint32_t b[S::NS][S::RT][2];
#pragma unroll
            for (int s = 0; s < S::NS; ++s)
#pragma unroll
                for (int rt = 0; rt < S::RT; ++rt) {
                    b[s][rt][0] = transpose8x8(split_pair<false>(p[s][rt][0]));
                    b[s][rt][1] = transpose8x8(split_pair<false>(p[s][rt][1]));
                }
            const int tok = (lane & 7) + ((lane >> 4) << 3), odd = (lane >> 3) & 1;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float c[S::RT][4];
#pragma unroll
                for (int rt = 0; rt < S::RT; ++rt) c[rt][0] = c[rt][1] = c[rt][2] = c[rt][3] = 0.f;
#pragma unroll
                for (int s = 0; s < S::NS; ++s) {
                    uint32_t a[4];
                    ldmatrix4t(a, tc::smem_u32(stage + s * S::STRIP + (S::PK + v) * kPlaneBf16 + tok * 128 +
                                               (((2 * j + odd) ^ (tok & 7)) << 4)));
                    if (MASK) {
                        // rows past the length hold anything; a value that is not finite goes to 0 here and makes
                        // NaN of the rows that see it, found by a product of indicators
                        uint32_t odd_ones = 0, flag[4];
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const int ja = j0 + 16 * s + 2 * t + 8 * (x >> 1);
                            a[x] &= (ja < len ? 0xffffu : 0u) | (ja + 1 < len ? 0xffff0000u : 0u);
                            flag[x] = __vcmpeq2(a[x] & 0x7f807f80u, 0x7f807f80u);
                            a[x] &= ~flag[x];
                            odd_ones |= flag[x];
                        }
                        if (__any_sync(0xffffffffu, odd_ones != 0)) {
#pragma unroll
                            for (int rt = 0; rt < S::RT; ++rt) {
                                const int ja = j0 + 16 * s + ta;
                                const uint32_t s0 = transpose8x8(ja < st.vis[rt] ? 0x3f80u : 0u), s1 = transpose8x8(ja + 8 < st.vis[rt] ? 0x3f80u : 0u);
                                float d[4] = {0.f, 0.f, 0.f, 0.f};
                                mma(d, flag[0] & 0x3f803f80u, flag[1] & 0x3f803f80u, flag[2] & 0x3f803f80u, flag[3] & 0x3f803f80u, s0, s1, false);
                                if (d[0] > 0.f) st.o[rt][v][j][0] = __int_as_float(0x7fc00000);
                                if (d[2] > 0.f) st.o[rt][v][j][1] = __int_as_float(0x7fc00000);
                            }
                        }
                    }
#pragma unroll
                    for (int rt = 0; rt < S::RT; ++rt) mma(c[rt], a[0], a[1], a[2], a[3], b[s][rt][0], b[s][rt][1], false);
                }
#pragma unroll
                for (int rt = 0; rt < S::RT; ++rt) {
                    st.o[rt][v][j][0] = fmaf(st.o[rt][v][j][0], corr[rt], c[rt][0] + c[rt][1]);
                    st.o[rt][v][j][1] = fmaf(st.o[rt][v][j][1], corr[rt], c[rt][2] + c[rt][3]);
                }
            }
        }
    }
}

// The warp's rows as a record in shared memory: [ROWS] maxima, [ROWS] sums, [ROWS][DV] weighted values.
template <class S> __device__ __forceinline__ void write_record(State<S> &st, bool lost, float *rec) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int rt = 0; rt < S::RT; ++rt) {
        float l = st.l[rt];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        const int r = 4 * rt + t;
        if (g == 0) {
            rec[r] = st.m[rt];
            rec[S::ROWS + r] = lost ? __int_as_float(0x7fc00000) : l;
        }
        float *o = rec + 2 * S::ROWS + r * S::DV;
#pragma unroll
        for (int v = 0; v < S::PV; ++v) {
            if constexpr (S::I4) {
                float mn = st.mn[rt][v];
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) mn += __shfl_xor_sync(0xffffffffu, mn, x);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    *reinterpret_cast<float2 *>(o + 64 * v + 8 * g + 2 * j) =
                        make_float2(fmaf(st.o[rt][v][j][0], 16777216.f, mn), fmaf(st.o[rt][v][j][1], 1048576.f, mn));
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    o[64 * v + 16 * j + g] = st.o[rt][v][j][0];
                    o[64 * v + 16 * j + 8 + g] = st.o[rt][v][j][1];
                }
            }
        }
    }
    __syncwarp();
}

struct Segment {                                        // what a warp leaves for the join
    long long key;                                      // first unit of the (sequence, head, row block), -1: nothing
    int begins, ends;                                   // whether it holds its first and its last tile
    int n, h, rb, pad;
    long long last;                                     // last unit
};

// weight of a record with maximum m under the common maximum top
__device__ __forceinline__ float weight(float m, float top) { return m == -INFINITY ? 0.f : exp2f(m - top); }

template <class S> __global__ void __launch_bounds__(S::WARPS * 32, 1) kernel(const __grid_constant__ Args A) {
    extern __shared__ __align__(128) char smem[];
    constexpr int W = S::WARPS, THREADS = W * 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem);                                   // [W][STAGES]
    Segment *segs = reinterpret_cast<Segment *>(smem + 1024);                              // [2 W]
    long long *pre = reinterpret_cast<long long *>(smem + 1024 + 2 * W * sizeof(Segment)); // [THREADS + 1]
    static_assert(sizeof(Segment) == 48 || sizeof(Segment) == 40, "segment");
    char *mine = smem + S::COMMON + warp * S::WARP_BYTES;
    float *rec0 = reinterpret_cast<float *>(mine + S::STAGES * S::STAGE), *rec1 = rec0 + S::RECORD;
    const uint32_t bar = tc::smem_u32(bars + warp * S::STAGES);
    __shared__ long long part_sum[W];
    __shared__ unsigned arrived;

    // ---- the call's units, and where each thread's sequences begin in their row
    const int per = (A.P.N + THREADS - 1) / THREADS;
    const int n_lo = min(A.P.N, (int)threadIdx.x * per), n_hi = min(A.P.N, n_lo + per);
    long long own = 0;
    for (int n = n_lo; n < n_hi; ++n) own += load_seq<S>(A, n).units(A.P.heads);
    long long run = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += y;
    }
    if (lane == 31) part_sum[warp] = run;
    if (lane == 0) {
#pragma unroll
        for (int s = 0; s < S::STAGES; ++s) tc::mbar_init(bar + 8 * s, 1);
        tc::fence_mbar_init();
        segs[2 * warp].key = segs[2 * warp + 1].key = -1;
    }
    __syncthreads();
    long long before = 0, U = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        before += w < warp ? part_sum[w] : 0;
        U += part_sum[w];
    }
    pre[threadIdx.x] = before + run - own;
    if (threadIdx.x == 0) pre[THREADS] = U;
    __syncthreads();
    if (U == 0) return;
    // few units: as few CTAs as give every warp one, so that fewer joins leave the CTA
    const long long C = min((long long)gridDim.x, (U + W - 1) / W);
    if ((long long)blockIdx.x >= C) return;
    const long long gw = (long long)blockIdx.x * W + warp, GW = C * W;
    const long long u0 = gw * U / GW, u1 = (gw + 1) * U / GW;
    const int total = (int)(u1 - u0);

    if (total > 0) {
        Cursor pc;                                       // runs ahead: the tile whose copies come next
        {
            int at = -1;
            for (int i = lane; i < THREADS; i += 32)
                if (pre[i] <= u0 && u0 < pre[i + 1]) at = i;
            at = __reduce_max_sync(0xffffffffu, at);
            long long rest = u0 - pre[at];
            pc.n = at * per;
            pc.s = load_seq<S>(A, pc.n);
            while (rest >= pc.s.units(A.P.heads)) {
                rest -= pc.s.units(A.P.heads);
                pc.s = load_seq<S>(A, ++pc.n);
            }
            const long long pair = rest / pc.s.tiles;
            pc.t = (int)(rest - pair * pc.s.tiles);
            pc.h = (int)(pair / pc.s.rbs);
            pc.rb = (int)(pair - (long long)pc.h * pc.s.rbs);
        }
        Cursor cc = pc;
        int issued = 0;
        unsigned bad_strips = 0;                         // NS bits a stage
        int page = -2;                                   // lane s: page of strip s of the next tile; -1 bad, -2 none
        int page_at = 0, page_h = 0;                     // its strip in the page, its head
        auto look_up = [&]() {
            page = -2;
            const int tok = pc.t * S::TILE + 16 * lane;
            if (lane < S::NS && tok < min(pc.s.len, pc.template seen_most<S>(A))) {
                page = paged_page(A.P, pc.n, tok);
                page_at = tok % A.P.page_size / kStrip;
                page_h = pc.h;
            }
        };
        auto issue = [&]() {
            const int s = issued % S::STAGES;
            const unsigned have = __ballot_sync(0xffffffffu, page >= 0), bad = __ballot_sync(0xffffffffu, page == -1);
            bad_strips = (bad_strips & ~(((1u << S::NS) - 1) << (s * S::NS))) | (bad << (s * S::NS));
            if (lane == 0) tc::mbar_arrive_expect_tx(bar + 8 * s, __popc(have) * S::STRIP);
            __syncwarp();
            if (page >= 0)
                tc::bulk_g2s(tc::smem_u32(mine + s * S::STAGE + lane * S::STRIP),
                             A.P.pool + (int64_t)page * A.P.page_bytes + (int64_t)page_h * A.P.block_bytes + (int64_t)page_at * S::STRIP,
                             S::STRIP, bar + 8 * s);
            if (++issued < total) {
                pc.advance<S>(A);
                look_up();
            }
        };
        look_up();
        while (issued < total && issued < S::STAGES) issue();

        State<S> st;
        bool dead = false;                               // a wait ran out: nothing more is issued or used
        long long first_unit = u0 - cc.t;                // first unit of the current segment
        bool begins = true;
        for (int k = 0; k < total; ++k) {
            if (k == 0 || cc.t == 0) {
                begins = cc.t == 0;
                first_unit = u0 + k - cc.t;
                load_rows<S>(A, cc, rec1, st);
            }
            const int s = k % S::STAGES;
            if (!dead && !tc::mbar_wait_bounded(bar + 8 * s, (k / S::STAGES) & 1, kWaitTries)) {
                dead = true;
                if (lane == 0) atomicOr(A.status, 2u);
            }
            dead = __any_sync(0xffffffffu, dead);
            const int j0 = cc.t * S::TILE, most = cc.template seen_most<S>(A);
            const unsigned bad = (bad_strips >> (s * S::NS)) & ((1u << S::NS) - 1);
            if (!dead && j0 < min(cc.s.len, most)) {
                if (bad || j0 + S::TILE > min(cc.s.len, cc.template seen_least<S>(A)))
                    tile<S, true>(A, mine + s * S::STAGE, j0, cc.s.len, bad, st);
                else
                    tile<S, false>(A, mine + s * S::STAGE, j0, cc.s.len, 0, st);
            }
            __syncwarp();
            if (!dead && issued < total) issue();
            const bool ends = cc.t == cc.s.tiles - 1;
            if (ends || k == total - 1) {
                const bool lost = cc.s.len < 0;
                if (begins && ends) {
                    write_record<S>(st, lost, rec1);
                    for (int x = lane; x < S::ROWS * S::DV / 4; x += 32) {
                        const int r = x / (S::DV / 4), ch = 4 * (x - r * (S::DV / 4));
                        store4<S>(A, cc, r, ch, *reinterpret_cast<const float4 *>(rec1 + 2 * S::ROWS + r * S::DV + ch), rec1[S::ROWS + r]);
                    }
                    __syncwarp();
                } else {
                    write_record<S>(st, lost, begins ? rec1 : rec0);
                    if (lane == 0)
                        segs[2 * warp + (begins ? 1 : 0)] = Segment{first_unit, begins, ends, cc.n, cc.h, cc.rb, 0, first_unit + cc.s.tiles - 1};
                }
            }
            if (k + 1 < total) cc.advance<S>(A);
        }
        if (dead)                                        // copies in flight land before their memory goes
            for (int k = 0; k < issued; ++k)
                if (k + S::STAGES >= issued) tc::mbar_wait_bounded(bar + 8 * (k % S::STAGES), (k / S::STAGES) & 1, kWaitTries);
    }
    __syncthreads();

    // ---- join the warps' records; those of (sequence, head, row block)s that reach into other CTAs go on
    long long out_key[2], out_last[2];
    Cursor out_at[2];
    int outs = 0;
    float *const my_partial = A.partial + (size_t)blockIdx.x * 2 * S::RECORD;
    for (int i = 0; i < 2 * W;) {
        const long long key = segs[i].key;
        if (key < 0) { ++i; continue; }
        int j = i + 1, last = i;
        for (; j < 2 * W && (segs[j].key < 0 || segs[j].key == key); ++j)
            if (segs[j].key == key) last = j;
        const bool begins = segs[i].begins != 0, ends = segs[last].ends != 0;
        Cursor c;
        c.n = segs[i].n; c.h = segs[i].h; c.rb = segs[i].rb; c.t = 0;
        c.s = load_seq<S>(A, c.n);
        float *dst = my_partial + (begins ? S::RECORD : 0);
        for (int x = threadIdx.x; x < S::ROWS * S::DV / 4; x += THREADS) {
            const int r = x / (S::DV / 4), ch = 4 * (x - r * (S::DV / 4));
            float top = -INFINITY;
            for (int y = i; y <= last; ++y)
                if (segs[y].key == key) {
                    const float *rec = reinterpret_cast<const float *>(smem + S::COMMON + (y >> 1) * S::WARP_BYTES + S::STAGES * S::STAGE) + (y & 1) * S::RECORD;
                    top = fmaxf(top, rec[r]);
                }
            float l = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int y = i; y <= last; ++y)
                if (segs[y].key == key) {
                    const float *rec = reinterpret_cast<const float *>(smem + S::COMMON + (y >> 1) * S::WARP_BYTES + S::STAGES * S::STAGE) + (y & 1) * S::RECORD;
                    const float f = weight(rec[r], top);
                    const float4 v = *reinterpret_cast<const float4 *>(rec + 2 * S::ROWS + r * S::DV + ch);
                    l = fmaf(f, rec[S::ROWS + r], l);
                    o.x = fmaf(f, v.x, o.x); o.y = fmaf(f, v.y, o.y); o.z = fmaf(f, v.z, o.z); o.w = fmaf(f, v.w, o.w);
                }
            if (begins && ends) {
                store4<S>(A, c, r, ch, o, l);
            } else {
                *reinterpret_cast<float4 *>(dst + 2 * S::ROWS + r * S::DV + ch) = o;
                if (ch == 0) { dst[r] = top; dst[S::ROWS + r] = l; }
            }
        }
        if (!(begins && ends) && outs < 2) {
            out_key[outs] = key;
            out_last[outs] = segs[i].last;
            out_at[outs++] = c;
        }
        i = j;
    }
    for (int i = 0; i < outs; ++i) {
        // the CTA that holds unit u: the largest c with c U / C <= u
        const long long first = ((out_key[i] + 1) * C - 1) / U, last = ((out_last[i] + 1) * C - 1) / U;
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0) arrived = atomicAdd(A.counters + first, 1u);
        __syncthreads();
        if ((long long)arrived != last - first) continue;
        __threadfence();
        if (threadIdx.x == 0) A.counters[first] = 0;     // as the next call needs it
        for (int x = threadIdx.x; x < S::ROWS * S::DV / 4; x += THREADS) {
            const int r = x / (S::DV / 4), ch = 4 * (x - r * (S::DV / 4));
            auto rec = [&](long long c) { return A.partial + ((size_t)c * 2 + (c == first ? 1 : 0)) * S::RECORD; };
            float top = -INFINITY;
#pragma unroll 4
            for (long long c = first; c <= last; ++c) top = fmaxf(top, __ldcg(rec(c) + r));
            float l = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (long long c = first; c <= last; ++c) {
                const float f = weight(__ldcg(rec(c) + r), top);
                const float4 v = __ldcg(reinterpret_cast<const float4 *>(rec(c) + 2 * S::ROWS + r * S::DV + ch));
                l = fmaf(f, __ldcg(rec(c) + S::ROWS + r), l);
                o.x = fmaf(f, v.x, o.x); o.y = fmaf(f, v.y, o.y); o.z = fmaf(f, v.z, o.z); o.w = fmaf(f, v.w, o.w);
            }
            store4<S>(A, out_at[i], r, ch, o, l);
        }
    }
}

template <class S> cudaError_t launch(const Args &A, int max_new, cudaStream_t stream) {
    static std::atomic<uint64_t> done{0};
    cudaError_t e = smem_attr_once((const void *)kernel<S>, S::SMEM, done);
    if (e != cudaSuccess) return e;
    int dev = 0, sms = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    // no more CTAs than the longest lengths could give a unit for each warp
    const double most = (double)A.P.N * A.P.heads * (((double)max_new * A.G + S::ROWS - 1) / S::ROWS) *
                        (((double)A.P.max_pages * A.P.page_size + S::TILE - 1) / S::TILE + 1);
    const double ctas = most / S::WARPS + 1;
    int grid = sms < kMaxCtas ? sms : kMaxCtas;
    if (ctas < grid) grid = (int)ctas;
    kernel<S><<<grid, S::WARPS * 32, S::SMEM, stream>>>(A);
    count_launch();
    return cudaGetLastError();
}

template <bool I4, int RT, int DQK> cudaError_t pick_dv(int dv, const Args &A, int max_new, cudaStream_t s) {
    if (dv == 64) return launch<Shape<DQK, 64, RT, I4>>(A, max_new, s);
    if (dv == 128) return launch<Shape<DQK, 128, RT, I4>>(A, max_new, s);
    return launch<Shape<DQK, 256, RT, I4>>(A, max_new, s);
}
template <bool I4, int RT> cudaError_t pick(int dqk, int dv, const Args &A, int max_new, cudaStream_t s) {
    if (dqk == 64) return pick_dv<I4, RT, 64>(dv, A, max_new, s);
    if (dqk == 128) return pick_dv<I4, RT, 128>(dv, A, max_new, s);
    if (dqk == 192) return pick_dv<I4, RT, 192>(dv, A, max_new, s);
    return pick_dv<I4, RT, 256>(dv, A, max_new, s);
}

// one translation unit each
cudaError_t run_i4_r4(int dqk, int dv, const Args &A, int max_new, cudaStream_t s);
cudaError_t run_i4_r8(int dqk, int dv, const Args &A, int max_new, cudaStream_t s);
cudaError_t run_bf16_r4(int dqk, int dv, const Args &A, int max_new, cudaStream_t s);
cudaError_t run_bf16_r8(int dqk, int dv, const Args &A, int max_new, cudaStream_t s);

}  // namespace attend
}  // namespace k3kda
