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
//   The running maximum is that of a tile's s plus the exponent of its largest scale less 14, which bounds p scale by
//   2^14: nothing overflows fp16, and what is far below it keeps 2^-38 of that.
// A tile's products start at 0 and are added to O in FP32 by fma (which also rescales O): tensor-core sums of
// few terms, ordinary rounding over the long axis.
//
// Measured, 4-bit pages, 128 + 128 channels.  64 sequences of 4 to 8,153 tokens, 32 heads, a query row each: 1,218 MB in 221 us,
// 5.5 TB/s (81 % of a copy's rate); the copies alone took 220 us and the arithmetic alone, in an earlier state, 248: both bind.
// One sequence of 250,008 tokens, 8 heads of 4 query rows: 288 MB in 68 us, of which some 12,000 cycles pass before the
// first product and 8,000 in the join.
#pragma once

#include "paged.cuh"
#include "tc_ptx.cuh"

namespace k3kda {
namespace attend {

constexpr int kMaxCtas = 160;                          // partials and counters of a workspace
constexpr size_t kHeadBytes = 256 + 4096;              // status word, counters (4 B a CTA)
constexpr int kMaxRows = 8;
constexpr int kExtra = 2, kRowsExtra = 10;             // units of a block's start and end, in tiles: few rows, 128-row blocks
constexpr int kRowsTile = 64;                          // keys of a tile of 128-row blocks
constexpr unsigned kWaitTries = 1u << 22;              // each try suspends for a while: seconds in all
static_assert(kMaxCtas * 4 <= 4096, "counters");

struct Args {
    Paged P;
    View q, gate;
    int in_bf16, out_bf16, Hq, G, T;
    const int32_t *cu;
    Rope r;
    float qmul;                                        // scale * log2(e)
    int per_page;                                      // strips of a page
    unsigned per_page_inv;                             // ceil(2^32 / per_page), exact for fewer than 2^28 strips; 0: one strip
    void *out;
    unsigned *status, *counters;
    float *partial;                                    // [kMaxCtas][2] records
    unsigned test_limit;                               // 128-row blocks: 0; else the armed test hook's tries (common.cuh)
};

// strips of a tile of the few-row kernel, pages with pl planes
constexpr int few_strips(bool i4, int pl) { return i4 ? (pl <= 4 ? 4 : 2) : (pl <= 2 ? 2 : 1); }

template <int DQK_, int DV_, int RT_, bool I4_> struct Shape {
    static constexpr int DQK = DQK_, DV = DV_, RT = RT_;
    static constexpr bool I4 = I4_;
    static constexpr int PK = DQK / 64, PV = DV / 64, PL = PK + PV;
    static constexpr int ROWS = 4 * RT;
    static constexpr int PLANE = I4 ? kPlaneI4 : kPlaneBf16, STRIP = PL * PLANE;
    static constexpr int NS = few_strips(I4, PL);                              // strips of a tile
    static constexpr int TILE = NS * kStrip, STAGE = NS * STRIP;
    static constexpr int WARPS = I4 ? (PL <= 4 ? 8 : RT == 1 ? 8 : 4) : (PL <= 4 ? 6 : 4);
    static constexpr int EXTRA = kExtra;
    static constexpr int QS = DQK + 8;                                          // floats between staged rows
    static constexpr int RECORD = ROWS * (DV + 2);                              // floats: m, l, O
    static constexpr int STAGED = ROWS * (QS + PK + 1);                         // floats: rows, their sums and exponents
    static constexpr int WORK = RECORD > STAGED ? RECORD : STAGED;
    static constexpr int FIXED = ((RECORD + WORK) * 4 + 127) / 128 * 128;       // bytes of a warp beside its ring
    static constexpr int COMMON = 1024 + 2 * WARPS * 32 + (WARPS * 32 + 4) * 4; // barriers, segments, prefix sums
    static constexpr int ROOM = (232448 - 256 - COMMON) / WARPS / 128 * 128;
    static constexpr int FIT = (ROOM - FIXED) / STAGE;
    static constexpr int STAGES = FIT > 6 ? 6 : FIT;
    static_assert(STAGES >= 2 && STAGES * WARPS * 8 <= 1024 && STAGES * NS <= 32, "ring");
    static constexpr int WARP_BYTES = STAGES * STAGE + FIXED;
    static constexpr int SMEM = COMMON + WARPS * WARP_BYTES;
    static_assert(STAGES * STAGE >= RECORD * 4 && STAGE % 64 == 0, "the ring holds a record at the end");
};

// c = (FIRST ? 0 : c) + A B
template <bool F16, bool FIRST> __device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    const float x = FIRST ? 0.f : c[0], y = FIRST ? 0.f : c[1], z = FIRST ? 0.f : c[2], w = FIRST ? 0.f : c[3];
    if constexpr (F16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
            : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(x), "f"(y), "f"(z), "f"(w));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
            : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(x), "f"(y), "f"(z), "f"(w));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&a)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]) : "r"(addr));
}
__device__ __forceinline__ void ldmatrix4t(uint32_t (&a)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]) : "r"(addr));
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
// the same of two values
template <bool F16> __device__ __forceinline__ void split_two(float x, float y, uint32_t &px, uint32_t &py) {
    uint32_t hi, lo;
    if constexpr (F16) {
        const __half2 h = __floats2half2_rn(x, y);
        const float2 f = __half22float2(h);
        const __half2 r = __floats2half2_rn(x - f.x, y - f.y);
        hi = *reinterpret_cast<const uint32_t *>(&h);
        lo = *reinterpret_cast<const uint32_t *>(&r);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        hi = *reinterpret_cast<const uint32_t *>(&h);
        const __nv_bfloat162 r = __floats2bfloat162_rn(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xffff0000u));
        lo = *reinterpret_cast<const uint32_t *>(&r);
    }
    px = __byte_perm(hi, lo, 0x5410);
    py = __byte_perm(hi, lo, 0x7632);
}
// the high (part 0) or low parts of two values
template <bool F16> __device__ __forceinline__ uint32_t pack_part(float x, float y, int part) {
    const uint32_t a = split_pair<F16>(x), b = split_pair<F16>(y);
    return __byte_perm(a, b, part ? 0x7632 : 0x5410);
}

// one sequence's share of the work
struct Seq {
    int len, q0, cnt, tiles, rbs;
    __device__ __forceinline__ unsigned pairs(int heads) const { return (unsigned)rbs * heads; }
};
template <class S> __device__ __forceinline__ Seq load_seq(const Args &A, int n) {
    Seq s;
    int b = n, e = n + 1;
    if (A.cu) seq_bounds(A.cu, n, A.T, b, e);
    s.len = paged_len(A.P, n);
    s.q0 = b;
    s.cnt = e - b;
    s.tiles = s.len > 0 ? (s.len + S::TILE - 1) / S::TILE : 1;   // an empty or bad sequence still writes its rows
    s.rbs = (int)(((unsigned)s.cnt * (unsigned)A.G + S::ROWS - 1) / S::ROWS);
    return s;
}

// a place in the row of units
struct Cursor {
    int n, h, rb, t;
    Seq s;
    int most, least;                                   // keys that some row of the block, and that its first row sees
    template <class S> __device__ __forceinline__ void enter(const Args &A) {
        const int r = rb * S::ROWS, last = min(s.cnt - 1, (r + S::ROWS - 1) / A.G);   // rows: below 2^28 (checked)
        most = min(s.len, s.len - s.cnt + last + 1);
        least = min(s.len, s.len - s.cnt + r / A.G + 1);
    }
    template <class S> __device__ __forceinline__ void advance(const Args &A) {
        if (++t < s.tiles) return;
        t = 0;
        if (++rb >= s.rbs) {
            rb = 0;
            if (++h >= A.P.heads) {
                h = 0;
                while (++n < A.P.N) {
                    s = load_seq<S>(A, n);
                    if (s.rbs > 0) break;
                }
            }
        }
        enter<S>(A);
    }
};

// Whether sequence n begins behind its end.  Without such a sequence the sequences' rows lie apart, T at most, and the units are as many as
// the call was checked for; with one, sums of them could pass 32 bits.
__device__ __forceinline__ bool decreases(const Args &A, int n) { return A.cu && A.cu[n + 1] < A.cu[n]; }

// A call whose cu_seqlens decreases: NaN for all rows.
__device__ __forceinline__ void all_nan(const Args &A, int dv) {
    const unsigned x = A.out_bf16 ? 0x7fc07fc0u : 0x7fc00000u;
    const int64_t pieces = (int64_t)A.T * A.Hq * dv / (A.out_bf16 ? 8 : 4);
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < pieces; i += (int64_t)gridDim.x * blockDim.x)
        reinterpret_cast<uint4 *>(A.out)[i] = make_uint4(x, x, x, x);
}

// out = O / l (* sigmoid(gate)) for channels ch .. ch + 3 of row R of a (sequence, key head) whose new tokens begin at q0, behind `past`
// keys.  l = 0: a row that sees no key gives 0, one whose keys all score minus infinity 0 / 0.
__device__ __forceinline__ void store4(const Args &A, int dv, int q0, int past, int h, int R, int ch, float4 o, float l) {
    const int i = R / A.G, hq = h * A.G + R - i * A.G;
    const float inv = l == 0.f ? (past + i >= 0 ? __int_as_float(0x7fc00000) : 0.f) : 1.f / l;
    float x[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
    if (A.gate.p) {
        const int64_t at = (int64_t)(q0 + i) * A.gate.ts + (int64_t)hq * A.gate.hs + ch;
        float g[4];
        if (A.in_bf16) {
#pragma unroll
            for (int e = 0; e < 4; ++e) g[e] = load_elt(A.gate.p, at + e, 1);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) g[e] = load_elt(A.gate.p, at + e, 0);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] *= sigmoidf_(g[e]);
    }
    const int64_t at = ((int64_t)(q0 + i) * A.Hq + hq) * dv + ch;
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

// A block's query rows and the rotation's phases on their way to registers.
template <class S> struct Rows {
    float x[S::ROWS][S::DQK / 32];        // lane's channels lane, lane + 32, ...
    uint64_t phase[S::DQK / 64];          // of pairs lane, lane + 32, ...
};
template <class S> __device__ __forceinline__ void fetch_rows(const Args &A, const Cursor &c, Rows<S> &f) {
    const int lane = threadIdx.x & 31, size = A.in_bf16 ? 2 : 4;
    const int rows = c.s.cnt * A.G, R0 = c.rb * S::ROWS;
    int i = R0 / A.G, g = R0 - i * A.G;                  // the row's token and head of the group
    const char *src[S::ROWS];
#pragma unroll
    for (int r = 0; r < S::ROWS; ++r) {
        src[r] = R0 + r < rows ? A.q.p + ((int64_t)(c.s.q0 + i) * A.q.ts + (int64_t)(c.h * A.G + g) * A.q.hs + lane) * size : nullptr;
        if (++g == A.G) { g = 0; ++i; }
    }
    if (A.in_bf16) {
#pragma unroll
        for (int r = 0; r < S::ROWS; ++r)
#pragma unroll
            for (int k = 0; k < S::DQK / 32; ++k) f.x[r][k] = src[r] ? load_elt(src[r], 32 * k, 1) : 0.f;
    } else {
#pragma unroll
        for (int r = 0; r < S::ROWS; ++r)
#pragma unroll
            for (int k = 0; k < S::DQK / 32; ++k) f.x[r][k] = src[r] ? load_elt(src[r], 32 * k, 0) : 0.f;
    }
#pragma unroll
    for (int k = 0; k < S::DQK / 64; ++k) f.phase[k] = lane + 32 * k < A.r.half ? A.r.phase[lane + 32 * k] : 0;
}

// Rows of a block: rotated, scaled, split and laid out as the operand.
template <class S> __device__ __forceinline__ void load_rows(const Args &A, const Cursor &c, const Rows<S> &f, float *qs, State<S> &st) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int rows = c.s.cnt * A.G, R0 = c.rb * S::ROWS;
    __syncwarp();
#pragma unroll
    for (int r = 0; r < S::ROWS; ++r)
#pragma unroll
        for (int k = 0; k < S::DQK / 32; ++k) qs[r * S::QS + lane + 32 * k] = f.x[r][k] * A.qmul;
    __syncwarp();
    if (A.r.dim > 0) {
#pragma unroll
        for (int k = 0; k < S::DQK / 64; ++k) {
            const int p = lane + 32 * k;
            if (p >= A.r.half) break;
            float *a = qs + A.r.off + (A.r.inter ? 2 * p : p);
            const int apart = A.r.inter ? 1 : A.r.half;
            int head = R0 % A.G, pos = c.s.len - c.s.cnt + R0 / A.G;
            float2 cs = rope_cs(f.phase[k], pos);
            float u[S::ROWS], v[S::ROWS];
#pragma unroll
            for (int r = 0; r < S::ROWS; ++r) {
                u[r] = a[r * S::QS] * A.r.mscale;
                v[r] = a[r * S::QS + apart] * A.r.mscale;
            }
#pragma unroll
            for (int r = 0; r < S::ROWS; ++r) {
                a[r * S::QS] = u[r] * cs.x - v[r] * cs.y;
                a[r * S::QS + apart] = v[r] * cs.x + u[r] * cs.y;
                if (++head == A.G) {                     // the next row is another token's
                    head = 0;
                    cs = rope_cs(f.phase[k], ++pos);
                }
            }
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
        const int R = R0 + 4 * rt + t;
        st.vis[rt] = R < rows ? c.s.len - c.s.cnt + R / A.G + 1 : 0;
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
                uint32_t *f = st.qf[rt][p][i];
                if constexpr (S::I4) {
                    const float *x = row + 64 * p + 16 * t + (i >> 1) * 8 + (i & 1) * 2;
                    f[0] = pack_part<true>(x[0] * mul * 16.f, x[4] * mul * 16.f, g & 1);
                    f[1] = pack_part<true>(x[1] * mul, x[5] * mul, g & 1);
                } else {
                    const float *x = row + 64 * p + 16 * i + 2 * t;
                    f[0] = pack_part<false>(x[0], x[1], g & 1);
                    f[1] = pack_part<false>(x[8], x[9], g & 1);
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
        if constexpr (S::I4) {
            float ps[S::RT][2], pm[S::RT][2];
#pragma unroll
            for (int k = 0; k < S::PK; ++k) {
                const char *pl = sp + k * kPlaneI4;
                const uint2 wa = *reinterpret_cast<const uint2 *>(pl + ta * 32 + 8 * t);
                const uint2 wb = *reinterpret_cast<const uint2 *>(pl + ta * 32 + 256 + 8 * t);
                const float2 ka = __half22float2(*reinterpret_cast<const __half2 *>(pl + 512 + ta * 4));
                const float2 kb = __half22float2(*reinterpret_cast<const __half2 *>(pl + 544 + ta * 4));
                float c[S::RT][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t ua = (i < 2 ? wa.x : wa.y) >> (8 * (i & 1)), ub = (i < 2 ? wb.x : wb.y) >> (8 * (i & 1));
#pragma unroll
                    for (int rt = 0; rt < S::RT; ++rt) {
                        const uint32_t *q = st.qf[rt][k][i];
                        if (i == 0) mma<true, true>(c[rt], ua & 0x000F000Fu, ub & 0x000F000Fu, ua & 0x00F000F0u, ub & 0x00F000F0u, q[0], q[1]);
                        else mma<true, false>(c[rt], ua & 0x000F000Fu, ub & 0x000F000Fu, ua & 0x00F000F0u, ub & 0x00F000F0u, q[0], q[1]);
                    }
                }
#pragma unroll
                for (int rt = 0; rt < S::RT; ++rt) {
                    const float sa = ka.x * (c[rt][0] + c[rt][1]), sb = kb.x * (c[rt][2] + c[rt][3]);
                    ps[rt][0] = k ? ps[rt][0] + sa : sa;
                    ps[rt][1] = k ? ps[rt][1] + sb : sb;
                    pm[rt][0] = k ? fmaf(ka.y, st.qsum[rt][k], pm[rt][0]) : ka.y * st.qsum[rt][k];
                    pm[rt][1] = k ? fmaf(kb.y, st.qsum[rt][k], pm[rt][1]) : kb.y * st.qsum[rt][k];
                }
            }
#pragma unroll
            for (int v = 0; v < S::PV; ++v) {
                const char *pl = sp + (S::PK + v) * kPlaneI4;
                vp[s][v][0] = *reinterpret_cast<const __half2 *>(pl + 512 + ta * 4);
                vp[s][v][1] = *reinterpret_cast<const __half2 *>(pl + 544 + ta * 4);
            }
#pragma unroll
            for (int rt = 0; rt < S::RT; ++rt) {
                p[s][rt][0] = fmaf(ps[rt][0], st.fac[rt], pm[rt][0]);
                p[s][rt][1] = fmaf(ps[rt][1], st.fac[rt], pm[rt][1]);
            }
        } else {
            constexpr int CH = S::PK;                    // a chain of products for each plane
            float ch[CH][S::RT][4], c[S::RT][4];
            const int tok = lane & 15, odd = lane >> 4;
#pragma unroll
            for (int k = 0; k < S::PK; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t a[4];
                    ldmatrix4(a, tc::smem_u32(sp + k * kPlaneBf16 + tok * 128 + (((2 * i + odd) ^ (tok & 7)) << 4)));
#pragma unroll
                    for (int rt = 0; rt < S::RT; ++rt) {
                        const uint32_t *q = st.qf[rt][k][i];
                        if (i == 0) mma<false, true>(ch[k][rt], a[0], a[1], a[2], a[3], q[0], q[1]);
                        else mma<false, false>(ch[k][rt], a[0], a[1], a[2], a[3], q[0], q[1]);
                    }
                }
#pragma unroll
            for (int rt = 0; rt < S::RT; ++rt) {
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    c[rt][x] = ch[0][rt][x];
#pragma unroll
                    for (int k = 1; k < CH; ++k) c[rt][x] += ch[k][rt][x];
                }
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
            top[rt] = fmaxf(top[rt], fmaxf(p[s][rt][0], p[s][rt][1]));
        }
    }
    // 4-bit: every value scale that the row sees here is below 2^e (their fp16 bits order as integers; NaN drops out)
    [[maybe_unused]] float e[S::RT];
    if constexpr (S::I4) {
#pragma unroll
        for (int rt = 0; rt < (MASK ? S::RT : 1); ++rt) {
            __half2 big = __float2half2_rn(0.f);
#pragma unroll
            for (int s = 0; s < S::NS; ++s)
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int v = 0; v < S::PV; ++v)
                        if (!MASK || j0 + 16 * s + ta + 8 * x < st.vis[rt]) big = __hmax2(big, vp[s][v][x]);
            unsigned bits = *reinterpret_cast<const uint32_t *>(&big) & 0xffffu;
            if (MASK) {                                  // the row's own tokens only: lanes of the same t
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) bits = max(bits, __shfl_xor_sync(0xffffffffu, bits, o));
            } else {
                bits = __reduce_max_sync(0xffffffffu, bits);
            }
            e[rt] = (float)max((int)(bits >> 10), 1) - 14.f;
        }
#pragma unroll
        for (int rt = MASK ? S::RT : 1; rt < S::RT; ++rt) e[rt] = e[0];
    }
    float corr[S::RT];
#pragma unroll
    for (int rt = 0; rt < S::RT; ++rt) {
        top[rt] = fmaxf(top[rt], __shfl_xor_sync(0xffffffffu, top[rt], 4));
        top[rt] = fmaxf(top[rt], __shfl_xor_sync(0xffffffffu, top[rt], 8));
        top[rt] = fmaxf(top[rt], __shfl_xor_sync(0xffffffffu, top[rt], 16));
        const float m = fmaxf(st.m[rt], S::I4 ? top[rt] + (e[rt] - 14.f) : top[rt]);
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
                for (int s = 0; s < S::NS; ++s) {
                    float2 qa = __half22float2(vp[s][v][0]), qb = __half22float2(vp[s][v][1]);
                    if (MASK) {                          // a key the row does not see weighs 0 even against a NaN
                        if (j0 + 16 * s + ta >= st.vis[rt]) qa = make_float2(0.f, 0.f);
                        if (j0 + 16 * s + ta + 8 >= st.vis[rt]) qb = make_float2(0.f, 0.f);
                    }
                    mn = fmaf(p[s][rt][0], qa.y, mn);
                    mn = fmaf(p[s][rt][1], qb.y, mn);
                    uint32_t pa, pb;
                    split_two<true>(p[s][rt][0] * qa.x, p[s][rt][1] * qb.x, pa, pb);
                    b[s][rt][0] = transpose8x8(pa);
                    b[s][rt][1] = transpose8x8(pb);
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
                for (int s = 0; s < S::NS; ++s) {
                    const uint32_t u0 = (j < 2 ? lo0[s] : hi0[s]) >> (8 * (j & 1)), u1 = (j < 2 ? lo1[s] : hi1[s]) >> (8 * (j & 1));
#pragma unroll
                    for (int rt = 0; rt < S::RT; ++rt) {
                        if (s == 0)
                            mma<true, true>(c[rt], u0 & 0x000F000Fu, u0 & 0x00F000F0u, u1 & 0x000F000Fu, u1 & 0x00F000F0u, b[s][rt][0], b[s][rt][1]);
                        else
                            mma<true, false>(c[rt], u0 & 0x000F000Fu, u0 & 0x00F000F0u, u1 & 0x000F000Fu, u1 & 0x00F000F0u, b[s][rt][0], b[s][rt][1]);
                    }
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
                    uint32_t pa, pb;
                    split_two<false>(p[s][rt][0], p[s][rt][1], pa, pb);
                    b[s][rt][0] = transpose8x8(pa);
                    b[s][rt][1] = transpose8x8(pb);
                }
            const int tok = (lane & 7) + ((lane >> 4) << 3), odd = (lane >> 3) & 1;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float c[S::RT][4];
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
                                float d[4];
                                mma<false, true>(d, flag[0] & 0x3f803f80u, flag[1] & 0x3f803f80u, flag[2] & 0x3f803f80u, flag[3] & 0x3f803f80u, s0, s1);
                                if (d[0] > 0.f) st.o[rt][v][j][0] = __int_as_float(0x7fc00000);
                                if (d[2] > 0.f) st.o[rt][v][j][1] = __int_as_float(0x7fc00000);
                            }
                        }
                    }
#pragma unroll
                    for (int rt = 0; rt < S::RT; ++rt) {
                        if (s == 0) mma<false, true>(c[rt], a[0], a[1], a[2], a[3], b[s][rt][0], b[s][rt][1]);
                        else mma<false, false>(c[rt], a[0], a[1], a[2], a[3], b[s][rt][0], b[s][rt][1]);
                    }
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
    int key;                                            // units before the (sequence, head, row block)'s tiles, -1: nothing
    int last;                                           // its last tile's unit
    int flags;                                          // 1: it holds its first tile, 2: its last
    int h, rb, q0, rows;                                // key head, row block, first token and rows of the sequence
    int past;                                           // keys before its first new token (negative: it has fewer than new ones)
};

// The row of units.  A (sequence, head, row block) takes `extra` units for its start and end (rows loaded, rotated and
// split; sums joined and stored) and one for each tile; with short sequences the former are most of the work.
struct Line {
    unsigned extra;
    const unsigned *pre;                                // [THREADS + 1]: units before each thread's sequences
    int per;                                            // sequences of a thread
    // Where unit u lies: its sequence, the (head, row block) in it, the unit in that one.
    template <class S> __device__ __forceinline__ void find(const Args &A, unsigned u, int threads, Seq &s, int &n, unsigned &pair, unsigned &at) const {
        int slot = -1;
        for (int i = threadIdx.x & 31; i < threads; i += 32)
            if (pre[i] <= u && u < pre[i + 1]) slot = i;
        slot = __reduce_max_sync(0xffffffffu, slot);
        unsigned rest = u - pre[slot];
        n = slot * per;
        s = load_seq<S>(A, n);
        unsigned have;
        while (rest >= (have = s.pairs(A.P.heads) * (s.tiles + extra))) {
            rest -= have;
            s = load_seq<S>(A, ++n);
        }
        pair = rest / (s.tiles + extra);
        at = rest - pair * (s.tiles + extra);
    }
};

// U units in equal runs over GW warps: the first `more` of them get one more than the others.
struct Split {
    unsigned base, more;
    __device__ __forceinline__ Split(unsigned U, unsigned GW) : base(U / GW), more(U - U / GW * GW) {}
    __device__ __forceinline__ unsigned begin(unsigned w) const { return w * base + min(w, more); }
    __device__ __forceinline__ unsigned owner(unsigned u) const {
        const unsigned edge = more * (base + 1);
        return u < edge ? u / (base + 1) : more + (u - edge) / base;     // (base = 0: every unit is below the edge)
    }
};

// weight of a record with maximum m under the common maximum top
__device__ __forceinline__ float weight(float m, float top) { return m == -INFINITY ? 0.f : exp2f(m - top); }

template <class S> __global__ void __launch_bounds__(S::WARPS * 32, 1) attend_kernel(const __grid_constant__ Args A) {
    extern __shared__ __align__(128) char smem[];
    constexpr int W = S::WARPS, THREADS = W * 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem);                                   // [W][STAGES]
    Segment *segs = reinterpret_cast<Segment *>(smem + 1024);                              // [2 W]
    unsigned *pre = reinterpret_cast<unsigned *>(smem + 1024 + 2 * W * sizeof(Segment));   // [THREADS + 1]
    char *mine = smem + S::COMMON + warp * S::WARP_BYTES;
    // a warp's memory: its ring (at the end its last record), its first record, and where rows are prepared and blocks finished
    float *rec0 = reinterpret_cast<float *>(mine + S::STAGES * S::STAGE), *work = rec0 + S::RECORD;
    const uint32_t bar = tc::smem_u32(bars + warp * S::STAGES);
    __shared__ unsigned part_sum[W], part_tiles[W];
    __shared__ unsigned arrived;

    // ---- the call's units, and where each thread's sequences begin in their row
    const int per = (A.P.N + THREADS - 1) / THREADS;
    const int n_lo = min(A.P.N, (int)threadIdx.x * per), n_hi = min(A.P.N, n_lo + per);
    unsigned own = 0, own_tiles = 0;                     // (sequence, head, row block)s, tiles
    bool bent = false;
    for (int n = n_lo; n < n_hi; ++n) {
        const Seq q = load_seq<S>(A, n);
        bent = bent || decreases(A, n);
        own += q.pairs(A.P.heads);
        own_tiles += q.pairs(A.P.heads) * q.tiles;
    }
    unsigned run = own, run_tiles = own_tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned y = __shfl_up_sync(0xffffffffu, run, o), z = __shfl_up_sync(0xffffffffu, run_tiles, o);
        if (lane >= o) {
            run += y;
            run_tiles += z;
        }
    }
    if (lane == 31) {
        part_sum[warp] = run;
        part_tiles[warp] = run_tiles;
    }
    if (lane == 0) {
#pragma unroll
        for (int s = 0; s < S::STAGES; ++s) tc::mbar_init(bar + 8 * s, 1);
        tc::fence_mbar_init();
        segs[2 * warp].key = segs[2 * warp + 1].key = -1;
    }
    if (__syncthreads_or(bent)) return all_nan(A, S::DV);
    unsigned pairs = 0, tiles = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        run += w < warp ? part_sum[w] : 0;
        run_tiles += w < warp ? part_tiles[w] : 0;
        pairs += part_sum[w];
        tiles += part_tiles[w];
    }
    // (a call with few tiles has a warp for each, and no runs to balance)
    const unsigned extra = tiles > 2 * gridDim.x * W ? S::EXTRA : 0, U = tiles + extra * pairs;
    pre[threadIdx.x] = run_tiles - own_tiles + extra * (run - own);
    if (threadIdx.x == 0) pre[THREADS] = U;
    __syncthreads();
    if (U == 0) return;
    // few units: as few CTAs as give every warp one, so that fewer joins leave the CTA
    const unsigned C = min(gridDim.x, (U + W - 1) / W);
    if (blockIdx.x >= C) return;
    const Split split(U, C * W);
    const Line line{extra, pre, per};
    const unsigned gw = blockIdx.x * W + warp, u0 = split.begin(gw), u1 = split.begin(gw + 1);
    Cursor pc;                                           // runs ahead: the tile whose copies come next
    unsigned base = 0;                                   // units before its (sequence, head, row block)
    if (u1 > u0) {
        unsigned pair, at;
        line.find<S>(A, u0, THREADS, pc.s, pc.n, pair, at);
        base = u0 - at;
        pc.t = at > extra ? (int)(at - extra) : 0;
        pc.h = (int)(pair / pc.s.rbs);
        pc.rb = (int)(pair - pc.h * pc.s.rbs);
        pc.enter<S>(A);
    }
    // (a run may hold nothing but a block's start)
    if (u1 > u0 && base + extra + pc.t < u1) {
        unsigned pbase = base;                           // pc's
        Cursor cc = pc;
        int issued = 0;                                  // tiles
        unsigned bad_strips = 0;                         // NS bits a stage
        // lane s: strip s of a tile, its page (not looked at before the copy: the load is on its way), its place in the
        // page (-1: no strip) and the head; a tile's pages are asked for while the one before it is issued
        struct Where { int page, at, h; } now, next;
        bool ahead = true;                               // pc is in the run
        auto look_up = [&]() {
            next.at = -1;
            const int strip = pc.t * S::NS + lane;
            if (ahead && lane < S::NS && 16 * strip < pc.most) {
                const int j = A.per_page_inv ? (int)__umulhi((unsigned)strip, A.per_page_inv) : strip;
                next.page = A.P.table[(int64_t)pc.n * A.P.max_pages + j];
                next.at = strip - j * A.per_page;
                next.h = pc.h;
            }
        };
        bool ready = true;                               // `now` is a tile of the run
        auto next_tile = [&]() {
            now = next;
            ready = ahead;
            if (ahead) {
                const unsigned then = pbase + pc.s.tiles + extra;
                if (pc.t == pc.s.tiles - 1) pbase = then;
                // the last unit of the run, or nothing but the next block's start after it
                ahead = (pc.t == pc.s.tiles - 1 ? pbase + extra : pbase + extra + pc.t + 1) < u1;
                if (ahead) pc.advance<S>(A);
            }
            look_up();
        };
        auto issue = [&]() {
            const int s = issued % S::STAGES;
            const bool good = now.at >= 0 && now.page >= 0 && now.page < A.P.num_pages;
            const unsigned have = __ballot_sync(0xffffffffu, good), bad = __ballot_sync(0xffffffffu, now.at >= 0 && !good);
            bad_strips = (bad_strips & ~(((1u << S::NS) - 1) << (s * S::NS))) | (bad << (s * S::NS));
            if (lane == 0) tc::mbar_arrive_expect_tx(bar + 8 * s, __popc(have) * S::STRIP);
            __syncwarp();
            // strips of one page lie together: the first of them brings all
            if (good && (lane == 0 || now.at == 0)) {
                const int run = min(A.per_page - now.at, __popc(have >> lane));
                tc::bulk_g2s(tc::smem_u32(mine + s * S::STAGE + lane * S::STRIP),
                             A.P.pool + (int64_t)now.page * A.P.page_bytes + (int64_t)now.h * A.P.block_bytes + (int64_t)now.at * S::STRIP,
                             run * S::STRIP, bar + 8 * s);
            }
            ++issued;
            next_tile();
        };
        Rows<S> rows;
        look_up();
        fetch_rows<S>(A, cc, rows);                      // under the pages' and the copies' latency
        next_tile();
        while (ready && issued < S::STAGES) issue();

        State<S> st;
        bool dead = false;                               // a wait ran out: nothing more is issued or used
        bool begins = cc.t == 0, fresh = true;           // fresh: the rows of a new block are on their way
        for (int k = 0;; ++k) {
            if (fresh) load_rows<S>(A, cc, rows, work, st);
            fresh = false;
            const int s = k % S::STAGES;
            const char *stage = mine + s * S::STAGE;
            const unsigned bad = (bad_strips >> (s * S::NS)) & ((1u << S::NS) - 1);
            if (!dead && !tc::mbar_wait_bounded(bar + 8 * s, (k / S::STAGES) & 1, kWaitTries)) {
                dead = true;
                if (lane == 0) atomicOr(A.status, 2u);
            }
            dead = __any_sync(0xffffffffu, dead);
            const int j0 = cc.t * S::TILE;
            if (!dead && j0 < cc.most) {
                if (bad || j0 + S::TILE > cc.least) tile<S, true>(A, stage, j0, cc.s.len, bad, st);
                else tile<S, false>(A, stage, j0, cc.s.len, 0, st);
            }
            __syncwarp();
            const bool ends = cc.t == cc.s.tiles - 1, stop = k + 1 == issued && !ready;
            if (!dead && ready) issue();
            if (!ends && !stop) {
                ++cc.t;
                continue;
            }
            const bool lost = cc.s.len < 0;
            const Segment done{(int)(base + extra), (int)(base + extra) + cc.s.tiles - 1, (begins ? 1 : 0) | (ends ? 2 : 0), cc.h, cc.rb,
                               cc.s.q0, cc.s.cnt * A.G, cc.s.len - cc.s.cnt};
            const bool last = stop || dead;              // (a dead warp leaves its run: its outputs are invalid)
            if (!last) {
                base += cc.s.tiles + extra;
                cc.advance<S>(A);
                fetch_rows<S>(A, cc, rows);
            }
            if (done.flags == 3) {
                write_record<S>(st, lost, work);
#pragma unroll 1
                for (int x = lane; x < S::ROWS * S::DV / 4; x += 32) {
                    const int r = x / (S::DV / 4), ch = 4 * (x - r * (S::DV / 4)), R = done.rb * S::ROWS + r;
                    if (R < done.rows)
                        store4(A, S::DV, done.q0, done.past, done.h, R, ch, *reinterpret_cast<const float4 *>(work + 2 * S::ROWS + r * S::DV + ch), work[S::ROWS + r]);
                }
                __syncwarp();
            } else {
                // (a block that begins but does not end here is the run's last: its tiles are read)
                write_record<S>(st, lost, begins ? reinterpret_cast<float *>(mine) : rec0);
                if (lane == 0) segs[2 * warp + (begins ? 1 : 0)] = done;
            }
            if (last) break;
            begins = fresh = true;
        }
        if (dead)                                        // copies in flight land before their memory goes
            for (int k = 0; k < issued; ++k)
                if (k + S::STAGES >= issued) tc::mbar_wait_bounded(bar + 8 * (k % S::STAGES), (k / S::STAGES) & 1, kWaitTries);
    }
    __syncthreads();

    // ---- join the warps' records, a (sequence, head, row block)'s run of them by one warp; what reaches into other CTAs
    // goes on to the workspace
    static_assert(2 * W <= 32, "a lane for each record");
    auto record = [&](int y) {
        return reinterpret_cast<const float *>(smem + S::COMMON + (y >> 1) * S::WARP_BYTES + (y & 1 ? 0 : S::STAGES * S::STAGE));
    };
    const int key = lane < 2 * W ? segs[lane].key : -1;
    const unsigned same = __match_any_sync(0xffffffffu, key);
    const unsigned heads = __ballot_sync(0xffffffffu, key >= 0 && lane == __ffs(same) - 1);    // first records of runs
    float *const my_partial = A.partial + (size_t)blockIdx.x * 2 * S::RECORD;
    // a warp's item: 32 pieces of 4 channels of a run, in one row (or two of 64 channels)
    constexpr int PIECES = S::DV / 4, PARTS = S::ROWS * PIECES / 32;
    int part = 0;
    unsigned left = heads;
    for (int i = 0; part < PARTS && heads; ++i) {        // the runs' first pieces before their second ones: late rows may be empty
        const int head = __ffs(left) - 1, x = 32 * part + lane;
        left &= left - 1;
        if (left == 0) {
            left = heads;
            ++part;
        }
        if (i % W != warp) continue;
        const int r = x / PIECES, ch = 4 * (x - r * PIECES);
        const unsigned members = __shfl_sync(0xffffffffu, same, head);
        const Segment sg = segs[head];
        const int R = sg.rb * S::ROWS + r;
        if (sg.rb * S::ROWS + (x - lane) / PIECES >= sg.rows) continue;
        const bool begins = sg.flags & 1, whole = begins && (segs[31 - __clz(members)].flags & 2);
        float *dst = my_partial + (begins ? S::RECORD : 0);
        // in the records' order, the maximum first
        float top = -INFINITY, l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        const int y0 = head, y1 = 31 - __clz(members);
#pragma unroll 4
        for (int y = y0; y <= y1; ++y)
            if ((members >> y) & 1) top = fmaxf(top, record(y)[r]);
#pragma unroll 4
        for (int y = y0; y <= y1; ++y)
            if ((members >> y) & 1) {
                const float *rec = record(y);
                const float f = weight(rec[r], top);
                const float4 v = *reinterpret_cast<const float4 *>(rec + 2 * S::ROWS + r * S::DV + ch);
                l = fmaf(f, rec[S::ROWS + r], l);
                o.x = fmaf(f, v.x, o.x); o.y = fmaf(f, v.y, o.y); o.z = fmaf(f, v.z, o.z); o.w = fmaf(f, v.w, o.w);
            }
        if (R >= sg.rows) continue;
        if (whole) {
            store4(A, S::DV, sg.q0, sg.past, sg.h, R, ch, o, l);
        } else {
            *reinterpret_cast<float4 *>(dst + 2 * S::ROWS + r * S::DV + ch) = o;
            if (ch == 0) {
                dst[r] = top;
                dst[S::ROWS + r] = l;
            }
        }
    }
    // a run that reaches out is the CTA's first (it began earlier) or its last (it goes on)
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
        if (heads == 0) break;
        const int head = i ? 31 - __clz(heads) : __ffs(heads) - 1;
        const Segment sg = segs[head];
        const unsigned members = __shfl_sync(0xffffffffu, same, head);
        const bool begins = sg.flags & 1, ends = segs[31 - __clz(members)].flags & 2;
        if ((begins && ends) || begins != (i == 1)) continue;
        const unsigned first = split.owner(sg.key) / W, last = split.owner(sg.last) / W;
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0) arrived = atomicAdd(A.counters + first, 1u);
        __syncthreads();
        if (arrived != last - first) continue;
        __threadfence();
        if (threadIdx.x == 0) A.counters[first] = 0;     // as the next call needs it
        auto rec = [&](unsigned b) { return A.partial + ((size_t)b * 2 + (b == first ? 1 : 0)) * S::RECORD; };
        for (int x = threadIdx.x; x < S::ROWS * S::DV / 4; x += THREADS) {
            const int r = x / (S::DV / 4), ch = 4 * (x - r * (S::DV / 4)), R = sg.rb * S::ROWS + r;
            if (R >= sg.rows) continue;
            // eight records on their way at a time, under a running maximum
            float top = -INFINITY, l = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
            for (unsigned b0 = first; b0 <= last; b0 += 8) {
                float m[8], sum[8];
                float4 v[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const float *from = rec(min(b0 + q, last));
                    m[q] = __ldcg(from + r);
                    sum[q] = __ldcg(from + S::ROWS + r);
                    v[q] = __ldcg(reinterpret_cast<const float4 *>(from + 2 * S::ROWS + r * S::DV + ch));
                }
                float next = top;
#pragma unroll
                for (int q = 0; q < 8; ++q) next = fmaxf(next, m[q]);          // (the last one again changes no maximum)
                const float old = weight(top, next);
                top = next;
                l *= old;
                o.x *= old; o.y *= old; o.z *= old; o.w *= old;
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    if (b0 + q > last) break;
                    const float f = weight(m[q], top);
                    l = fmaf(f, sum[q], l);
                    o.x = fmaf(f, v[q].x, o.x); o.y = fmaf(f, v[q].y, o.y); o.z = fmaf(f, v[q].z, o.z); o.w = fmaf(f, v[q].w, o.w);
                }
            }
            store4(A, S::DV, sg.q0, sg.past, sg.h, R, ch, o, l);
        }
    }
}

template <class S> cudaError_t launch(const Args &A, int max_new, cudaStream_t stream) {
    static std::atomic<uint64_t> done{0};
    cudaError_t e = smem_attr_once((const void *)attend_kernel<S>, S::SMEM, done);
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
    attend_kernel<S><<<grid, S::WARPS * 32, S::SMEM, stream>>>(A);
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
