// paged_rows.cuh -- attention of many new tokens over the paged cache on sm_103a: the same function as
// paged_attend.cuh for blocks of 128 query rows (prompts in chunks, several tokens checked at once, large head groups), on tcgen05.
//
// With this many rows the products bound the time, not the cache's bytes, and a tile's unpacking is shared by 128 rows.
// A CTA takes a run of 64-key tiles of (sequence, key head, row block)s (the same equal split, with partial results joined by the
// CTA that finishes last) and its warps pass them on through mbarriers:
//   producer (1 warp)  bulk copies of whole strips, whose pages it looks up
//   helpers (8 warps)  4-bit: codes to fp16 operand tiles by one AND (paged_attend.cuh), scales and minima to FP32;
//                      and, two tiles later, O = O corr + (the tile's product), 128 rows by half the channels a warpgroup, in registers
//   MMA (1 warp)       S = Q K^T, O_tile = P V, each with Q and P as a high and a low 16-bit part: A = Q from TMEM where it
//                      fits there (32 cycles a product of N = 64 against 48 from shared memory, and as much room there for
//                      the ring), P from TMEM where it took S's columns
//   softmax            a row a thread: S out of TMEM, scales, running maximum, weights back in.  bf16 pages 4 warps; 4-bit
//                      pages, with 30 instructions a key, 8 warps with half the tile's keys each, whose scores stay in registers
// 4-bit: a score group (64 channels) has columns of its own, s = sum_g scale_gj S_g + min_gj sum(q_g) on the way out; a
// value group has weights of its own, p_j scale_gj, and sum_j p_j min_gj stays in FP32.  bf16 pages hold 64-channel planes
// in the operands' own 128-byte swizzle (include/k3kda.h), so their strips are copied straight to the operand tiles.
// What bounds it, measured in cycles a tile of 64 keys and 128 rows: 4-bit pages of 128 + 128 channels, the softmax warps (2900 beside
// 1600 of products; with 4 warps and both passes forming the scores it was 4100); bf16 pages of 192 + 128, the products (1700)
// and the softmax (2100) in turn.  A block's start, its rows' rotation and split, takes 8,000 to 12,000, the join of a shared
// block 15,000.  462 new tokens of 4 sequences (13,365 cached), 8 heads of 4 query heads, 4-bit pages: 113 us.  153 new tokens of 48
// sequences (82,739 cached), 4 heads of 8 query heads of 192 + 128 channels, bf16 pages: 217 MB in 88 us.
// A row block's tiles are those of the whole sequence; those that none of its rows sees are skipped, but the division into runs counts
// them, so that a prompt from position 0 leaves the CTAs unevenly loaded: 8,192 tokens, 8 heads of 4 query heads, 4-bit pages 2,801 us.
#pragma once

#include "paged_attend.cuh"

namespace k3kda {
namespace attend {

template <int DQK_, int DV_, bool I4_> struct RowsShape {
    static constexpr int DQK = DQK_, DV = DV_;
    static constexpr bool I4 = I4_;
    static constexpr int PK = DQK / 64, PV = DV / 64, PL = PK + PV;
    static constexpr int ROWS = 128, NS = 4, TILE = kRowsTile;
    static constexpr int EXTRA = kRowsExtra;                                    // (few tokens, bf16 pages: 4: 112 us, 6: 97, 10: 89, 14: 89)
    static constexpr int STRIP = PL * (I4 ? kPlaneI4 : kPlaneBf16);
    static constexpr int GK = I4 ? PK : 1, GV = I4 ? PV : 1;                    // groups of scores, of weights
    static constexpr int SB = 64 * (GK > GV ? GK : GV);                         // TMEM columns of a tile's scores, then weights
    static constexpr bool QT = 2 * SB + DQK + DV <= 512;                        // the rows' operand stands in TMEM where it fits
    static constexpr int COL_Q = 2 * SB, COL_O = COL_Q + (QT ? DQK : 0);
    static constexpr int OB = COL_O + 2 * DV <= 512 ? 2 : 1;                    // buffers of a tile's product
    static_assert(COL_O + OB * DV <= 512, "TMEM");
    // softmax warpgroups (each takes its share of a tile's keys), two of helpers, one of producer, MMA and idle warps
    static constexpr int SW = I4 ? 2 : 1, KEYS = 64 / SW;
    static constexpr int HELP = 4 * SW, PROD = HELP + 8, WARPS = PROD + 4, THREADS = WARPS * 32;
    // Registers a thread: at launch (65,536 over the threads, in eights), then of each role; what the last warpgroup gives up the others take.
    static constexpr int LAUNCH = 65536 / THREADS / 8 * 8, R_SOFT = SW == 2 ? 112 : 192, R_HELP = SW == 2 ? 104 : 128, R_REST = SW == 2 ? 48 : 64;
    static_assert(4 * SW * R_SOFT + 8 * R_HELP + 4 * R_REST <= WARPS * LAUNCH, "registers");
    static constexpr int RECORD = ROWS * (DV + 2);
    // shared memory, in bytes from a 1024-byte boundary
    static constexpr int Q_PART = PK * 16384, KV = PL * 8192;
    static constexpr int RS = I4 ? 2 : 1, RAW = I4 ? NS * STRIP : 0;
    static constexpr int PARAMS = I4 ? PL * 512 : 0;                            // scale[64], minimum[64] of each plane
    static constexpr int SMALL = 4 * 128 * 4 + (2 + PV) * 128 * 4 + 128 * (PK + 1) * 4 + 1024 + 64 + 8 * PV * 8 + (THREADS + 4) * 4 + (SW > 1 ? 4 * 128 * 4 : 0);
    static constexpr int FIT = (232448 - 1024 - 256 - (QT ? 0 : 2 * Q_PART) - RS * RAW - SMALL) / (KV + PARAMS + 64);
    static constexpr int KB = FIT > 4 ? 4 : FIT;                                // operand tiles
    static_assert(KB >= 2 && KV >= WARPS * DQK * 4 && KB * KV >= ROWS * (DV + 4) * 4 && (!QT || KB * KV >= WARPS * DQK * 4 + 2 * Q_PART), "operand tiles");
    // (rows on their way to TMEM pass through the operand tiles, behind the warps' floats)
    static constexpr int AT_KV = QT ? 0 : 2 * Q_PART, AT_Q = QT ? WARPS * DQK * 4 : 0, AT_RAW = AT_KV + KB * KV, AT_PAR = AT_RAW + RS * RAW, AT_TOP = AT_PAR + KB * PARAMS;
    static constexpr int AT_CORR = AT_TOP + KB * 64, AT_FIN = AT_CORR + 4 * 128 * 4, AT_INFO = AT_FIN + (2 + PV) * 128 * 4;
    static constexpr int AT_BAR = AT_INFO + 128 * (PK + 1) * 4, AT_BAD = AT_BAR + 512, AT_PRE = AT_BAD + 64 + 8 * PV * 8;
    static constexpr int AT_XCH = AT_PRE + (THREADS + 4) * 4;                   // what the softmax warpgroups tell one another: [4][128]
    // the join's weights of records: over the operand tiles where they end before the barriers, else behind everything
    static constexpr int USED = AT_XCH + (SW > 1 ? 4 * 128 * 4 : 0), JOIN = (kMaxCtas + 1) * 128 * 4;
    static constexpr int AT_JOIN = AT_BAR >= JOIN ? 0 : USED, SMEM = (AT_JOIN ? USED + JOIN : USED) + 1024;
    static_assert(SMEM + 256 <= 232448, "shared memory");
};

// kind::f16 instruction descriptor with fp16 (or bf16) operands, FP32 sums
__host__ __device__ constexpr uint32_t idesc16(bool f16, int M, int N, bool b_mn) {
    return f16 ? tc::idesc_bf16_f32(M, N, false, false, b_mn) & ~((1u << 7) | (1u << 10)) : tc::idesc_bf16_f32(M, N, false, false, b_mn);
}

// packed pairs of FP32
using F2 = unsigned long long;
__device__ __forceinline__ F2 pk(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 up(F2 x) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

template <int N> __device__ __forceinline__ void take_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(N)); }
template <int N> __device__ __forceinline__ void give_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(N)); }

// A pair as two 16-bit parts of each: rounded, and what that left (exact in FP32) rounded.
template <bool F16> __device__ __forceinline__ void split2(float2 w, uint32_t &hi, uint32_t &lo) {
    float a, b;
    if constexpr (F16) {
        const __half2 h = __floats2half2_rn(w.x, w.y);
        hi = *reinterpret_cast<const uint32_t *>(&h);
        asm("fma.rn.f32.f16 %0, %1, %2, %3;" : "=f"(a) : "h"(__half_as_ushort(__low2half(h))), "h"((uint16_t)0xBC00), "f"(w.x));
        asm("fma.rn.f32.f16 %0, %1, %2, %3;" : "=f"(b) : "h"(__half_as_ushort(__high2half(h))), "h"((uint16_t)0xBC00), "f"(w.y));
        const __half2 rest = __floats2half2_rn(a, b);
        lo = *reinterpret_cast<const uint32_t *>(&rest);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(w.x, w.y);
        hi = *reinterpret_cast<const uint32_t *>(&h);
        const __nv_bfloat162 rest = __floats2bfloat162_rn(w.x - __uint_as_float(hi << 16), w.y - __uint_as_float(hi & 0xffff0000u));
        lo = *reinterpret_cast<const uint32_t *>(&rest);
    }
}

// x as a bf16 pair, the high part in the low half, with parts of the same sign and none 0 but for x = 0: each times an infinite key is
// the same infinity, as x times it is.  The high part is cut off, not rounded, so together they have 16 bits; 2^-100 adds nothing.
__device__ __forceinline__ uint32_t split_same_sign(float x) {
    const uint32_t hi = __float_as_uint(x) & 0xffff0000u;
    const float rest = x - __uint_as_float(hi);
    const uint32_t lo = __bfloat16_as_ushort(__float2bfloat16_rn(rest == 0.f && hi << 1 ? __uint_as_float((hi & 0x80000000u) | 0x0d800000u) : rest));
    return hi >> 16 | lo << 16;
}

// A bounded wait that also ends when another warp of the CTA has given up.
__device__ __forceinline__ bool wait_for(uint32_t bar, int parity, volatile int *dead, unsigned *status) {
    for (unsigned i = 0; i < kWaitTries; ++i) {
        if (tc::mbar_try_wait(bar, parity & 1)) return true;
        if ((i & 63) == 63 && *dead) return false;
    }
    *dead = 1;
    atomicOr(status, 2u);
    return false;
}

__device__ __forceinline__ bool elect() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

template <class S> __global__ void __launch_bounds__(S::THREADS, 1) rows_kernel(const __grid_constant__ Args A) {
    extern __shared__ char smem_raw[];
    char *const sm = reinterpret_cast<char *>(tc::smem_align1024(reinterpret_cast<uint8_t *>(smem_raw)));
    const uint32_t sm32 = tc::smem_u32(sm);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float *corr = reinterpret_cast<float *>(sm + S::AT_CORR), *fin = reinterpret_cast<float *>(sm + S::AT_FIN);
    float *info = reinterpret_cast<float *>(sm + S::AT_INFO);                  // [128][PK sums, factor]
    int *bad_of = reinterpret_cast<int *>(sm + S::AT_BAD);                     // [8] tiles' strips on pages outside the pool, [8] whether values were put to 0
    unsigned long long *poison = reinterpret_cast<unsigned long long *>(sm + S::AT_BAD + 64);   // [8][PV]: tokens whose value group is not finite
    unsigned *pre = reinterpret_cast<unsigned *>(sm + S::AT_PRE);
    __shared__ unsigned part_sum[S::WARPS], part_tiles[S::WARPS], arrived, tslot;
    __shared__ int dead_flag;
    volatile int *dead = &dead_flag;
    // barriers
    const uint32_t bar = sm32 + S::AT_BAR;
    const uint32_t raw_full = bar, raw_free = bar + 16, kv_full = bar + 32, kv_free = bar + 64, v_ok = bar + 96, s_full = bar + 128,
                   p_full = bar + 144, o_full = bar + 160, o_free = bar + 176;

    // ---- the call's units (as in paged_attend.cuh, a CTA a run)
    const int per = (A.P.N + S::THREADS - 1) / S::THREADS;
    const int n_lo = min(A.P.N, (int)threadIdx.x * per), n_hi = min(A.P.N, n_lo + per);
    unsigned own = 0, own_tiles = 0;
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
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(raw_full + 8 * i, 1);
            tc::mbar_init(raw_free + 8 * i, 256);
            tc::mbar_init(s_full + 8 * i, 1);
            tc::mbar_init(p_full + 8 * i, 128 * S::SW);
            tc::mbar_init(o_full + 8 * i, 1);
            tc::mbar_init(o_free + 8 * i, 256);
        }
        for (int i = 0; i < 4; ++i) {
            tc::mbar_init(kv_full + 8 * i, S::I4 ? 256 : 1);
            tc::mbar_init(kv_free + 8 * i, 1);
            tc::mbar_init(v_ok + 8 * i, 256);
        }
        tc::fence_mbar_init();
        dead_flag = 0;
    }
    if (__syncthreads_or(bent)) return all_nan(A, S::DV);
    unsigned pairs = 0, tiles = 0;
    for (int w = 0; w < S::WARPS; ++w) {
        run += w < warp ? part_sum[w] : 0;
        run_tiles += w < warp ? part_tiles[w] : 0;
        pairs += part_sum[w];
        tiles += part_tiles[w];
    }
    const unsigned extra = S::EXTRA, U = tiles + extra * pairs;
    pre[threadIdx.x] = run_tiles - own_tiles + extra * (run - own);
    if (threadIdx.x == 0) pre[S::THREADS] = U;
    __syncthreads();
    if (pairs == 0) return;
    const unsigned C = min(gridDim.x, max(pairs, U / 8));                      // runs of 8 units at least, a block a CTA at most
    if (blockIdx.x >= C) return;
    const Split split(U, C);
    const Line line{extra, pre, per};
    const unsigned u0 = split.begin(blockIdx.x), u1 = split.begin(blockIdx.x + 1);
    if (u0 == u1) return;
    if (warp == 0) {
        tc::tmem_alloc(tc::smem_u32(&tslot), 512);
        tc::tmem_relinquish();
    }
    Cursor start;
    unsigned pair, at;
    line.find<S>(A, u0, S::THREADS, start.s, start.n, pair, at);
    const unsigned base0 = u0 - at;
    start.t = at > extra ? (int)(at - extra) : 0;
    start.h = (int)(pair / start.s.rbs);
    start.rb = (int)(pair - start.h * start.s.rbs);
    start.enter<S>(A);
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tb = tslot;

    // The rows of a block: rotated, scaled, split to the operand tiles (softmax and helper warps, each through DQK floats of its own).
    auto prepare = [&](const Cursor &c) {
        const int rows = c.s.cnt * A.G, R0 = c.rb * S::ROWS;
        {
            float *x = reinterpret_cast<float *>(sm + S::AT_KV) + warp * S::DQK;
            const int size = A.in_bf16 ? 2 : 4;
            uint64_t phase[(S::DQK / 2 + 31) / 32];
#pragma unroll
            for (int k = 0; k < (S::DQK / 2 + 31) / 32; ++k) phase[k] = lane + 32 * k < A.r.half ? A.r.phase[lane + 32 * k] : 0;
            float v[S::DQK / 32], next[S::DQK / 32];     // the next row is on its way while one is prepared
            auto fetch = [&](int r, float (&f)[S::DQK / 32]) {
                const int R = R0 + r, i = R / A.G, hq = c.h * A.G + R - i * A.G;
                const char *src = A.q.p + ((int64_t)(c.s.q0 + i) * A.q.ts + (int64_t)hq * A.q.hs + lane) * size;
                if (A.in_bf16) {
#pragma unroll
                    for (int k = 0; k < S::DQK / 32; ++k) f[k] = load_elt(src, 32 * k, 1);
                } else {
#pragma unroll
                    for (int k = 0; k < S::DQK / 32; ++k) f[k] = load_elt(src, 32 * k, 0);
                }
            };
            const int live = min(S::ROWS, rows - R0), each = (live + S::PROD - 1) / S::PROD, r1 = min(live, (warp + 1) * each);
            float2 cs[(S::DQK / 2 + 31) / 32];
            int turned = -1;                             // the token whose cosines and sines they are
            for (int r = live + warp; r < S::ROWS; r += S::PROD) {             // rows of nothing
                for (int w = lane; w < S::DQK / 8; w += 32) {
                    char *dst = sm + S::AT_Q + (w >> 3) * 16384 + r * 128 + (((w & 7) ^ (r & 7)) << 4);
                    *reinterpret_cast<uint4 *>(dst) = *reinterpret_cast<uint4 *>(dst + S::Q_PART) = make_uint4(0, 0, 0, 0);
                }
                if (S::I4 && lane <= S::PK) info[r * (S::PK + 1) + lane] = 0.f;
            }
            if (warp * each < r1) fetch(warp * each, next);
#pragma unroll 1
            for (int r = warp * each; r < r1; ++r) {
                const int i = (R0 + r) / A.G;
#pragma unroll
                for (int k = 0; k < S::DQK / 32; ++k) v[k] = next[k];
                if (r + 1 < r1) fetch(r + 1, next);
                __syncwarp();
#pragma unroll
                for (int k = 0; k < S::DQK / 32; ++k) x[lane + 32 * k] = v[k] * A.qmul;
                __syncwarp();
                if (A.r.dim > 0) {
                    const int pos = c.s.len - c.s.cnt + i, apart = A.r.inter ? 1 : A.r.half;
#pragma unroll
                    for (int k = 0; k < (S::DQK / 2 + 31) / 32; ++k) {
                        const int p = lane + 32 * k;
                        if (p >= A.r.half) break;
                        if (turned != i) cs[k] = rope_cs(phase[k], pos);
                        float *a = x + A.r.off + (A.r.inter ? 2 * p : p);
                        const float u = a[0] * A.r.mscale, w = a[apart] * A.r.mscale;
                        a[0] = u * cs[k].x - w * cs[k].y;
                        a[apart] = w * cs[k].x + u * cs[k].y;
                    }
                    turned = i;
                    __syncwarp();
                }
                float mul = 1.f;
                if constexpr (S::I4) {
                    float big = 0.f;
#pragma unroll
                    for (int p = 0; p < S::PK; ++p) {
                        const float a = x[64 * p + lane], b = x[64 * p + 32 + lane];
                        big = fmaxf(big, fmaxf(fabsf(a), fabsf(b)));
                        const float sum = warp_sum(a + b);
                        if (lane == 0) info[r * (S::PK + 1) + p] = sum;
                    }
                    big = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(big)));   // (magnitudes order as integers)
                    const int e = min(max(9 - ((int)(__float_as_uint(big) >> 23) - 127), -100), 120);
                    mul = __int_as_float((e + 127) << 23);
                    if (lane == 0) info[r * (S::PK + 1) + S::PK] = __int_as_float((20 - e + 127) << 23);
                }
                // 16-byte pieces: 8 channels (4-bit: in the order the codes come out, even ones by 16)
                for (int w = lane; w < S::DQK / 8; w += 32) {
                    const float *y = x + 8 * w;
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float a = S::I4 ? y[q] * mul * (q & 1 ? 1.f : 16.f) : y[2 * q], b = S::I4 ? y[q + 4] * mul * (q & 1 ? 1.f : 16.f) : y[2 * q + 1];
                        const uint32_t pa = S::I4 ? split_pair<true>(a) : split_same_sign(a), pb = S::I4 ? split_pair<true>(b) : split_same_sign(b);
                        hi[q] = __byte_perm(pa, pb, 0x5410);
                        lo[q] = __byte_perm(pa, pb, 0x7632);
                    }
                    char *dst = sm + S::AT_Q + (w >> 3) * 16384 + r * 128 + (((w & 7) ^ (r & 7)) << 4);
                    *reinterpret_cast<uint4 *>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4 *>(dst + S::Q_PART) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
            }
        }
        if constexpr (S::QT) {                           // thread r copies row r to TMEM: the high parts, the low parts
            tc::named_bar(4, 32 * S::PROD);
            if (warp < S::HELP) {
                const int r = threadIdx.x & 127;
#pragma unroll 1
                for (int part = S::SW > 1 ? (int)(threadIdx.x >> 7) : 0; part < (S::SW > 1 ? (int)(threadIdx.x >> 7) + 1 : 2); ++part)
#pragma unroll 2
                    for (int w = 0; w < S::DQK / 8; w += 2) {
                        const char *src = sm + S::AT_Q + part * S::Q_PART + (w >> 3) * 16384 + r * 128;
                        const uint4 a = *reinterpret_cast<const uint4 *>(src + (((w & 7) ^ (r & 7)) << 4)), b = *reinterpret_cast<const uint4 *>(src + ((((w + 1) & 7) ^ (r & 7)) << 4));
                        const uint32_t x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
                        tc::tmem_st8(tb + ((uint32_t)((warp & 3) * 32) << 16) + S::COL_Q + part * (S::DQK / 2) + 4 * w, x);
                    }
                tc::tmem_wait_st();
                tc::tc_fence_before();
            }
        }
        tc::fence_async_smem();
    };
    // A role's way through the run: a segment is tiles t0 .. t1 of one block, of which the first T have keys that some row sees.
    // Every warp of the CTA passes the same three barriers a segment; each role has a loop of its own, so that its registers
    // are its own.
    auto segments = [&](auto &&role, auto &&finish, bool rows_too) {
        Cursor c = start;
        unsigned base = base0, done = 0;                                       // done: tiles of earlier segments
        while (base + extra + c.t < u1) {
            const int t0 = c.t, t1 = (int)min((unsigned)c.s.tiles, u1 - (base + extra));
            const int T = max(0, min(t1, (c.most + 63) / 64) - t0);
            if (rows_too) prepare(c);
            tc::named_bar(1, S::THREADS);
            role(c, t0, T, done);
            tc::named_bar(1, S::THREADS);
            finish(c, base, t0, t1);
            done += T;
            base += c.s.tiles + extra;
            c.t = c.s.tiles - 1;
            const bool stop = *dead != 0;
            tc::named_bar(1, S::THREADS);
            if (stop || base + extra >= u1) break;
            c.advance<S>(A);
        }
    };
    auto nothing = [](const Cursor &, unsigned, int, int) {};

    if (warp < S::HELP) {
        take_registers<S::R_SOFT>();
        segments([&](const Cursor &c, int t0, int T, unsigned done) {
            const int rows = c.s.cnt * A.G, R0 = c.rb * S::ROWS;
            // ---- softmax: thread r has row r, with two warpgroups the first or the last 32 keys of a tile
            const int r = threadIdx.x & 127, R = R0 + r, wg = S::SW > 1 ? threadIdx.x >> 7 : 0, b0 = wg * (S::KEYS / 16);
            float *xch = reinterpret_cast<float *>(sm + S::AT_XCH);
            bool ok = true;
            const int vis = R < rows ? c.s.len - c.s.cnt + R / A.G + 1 : 0;
            float m = -INFINITY, l = 0.f, mn[S::PV];
            F2 qs[S::PK];
            float fac = 1.f;
#pragma unroll
            for (int v = 0; v < S::PV; ++v) mn[v] = 0.f;
            if constexpr (S::I4) {
#pragma unroll
                for (int p = 0; p < S::PK; ++p) qs[p] = pk(info[r * (S::PK + 1) + p], info[r * (S::PK + 1) + p]);
                fac = info[r * (S::PK + 1) + S::PK];
            }
            for (int k = 0; k < T; ++k) {
                const unsigned use = done + k;
                // (a warp that gave up still comes to the warpgroups' barriers)
                ok = ok && __all_sync(0xffffffffu, wait_for(s_full + 8 * (use & 1), use >> 1, dead, A.status));
                if (!ok) {
                    if (S::SW == 1) break;
                    tc::named_bar(3, 256);
                    continue;
                }
                tc::tc_fence_after();
                const int j0 = (t0 + k) * 64, slot = use % S::KB;
                const int bad = bad_of[use & 7];
                const bool mask = bad || j0 + 64 > c.least;
                const uint32_t ts = tb + ((uint32_t)((warp & 3) * 32) << 16) + (use & 1) * S::SB;
                const float *par = reinterpret_cast<const float *>(sm + S::AT_PAR + slot * S::PARAMS);
                // 16 keys' scores out of TMEM
                uint32_t x[S::GK][16];
                auto bring = [&](int b) {
#pragma unroll
                    for (int g = 0; g < S::GK; ++g) tc::tmem_ld16(ts + 64 * g + 16 * b, x[g]);
                };
                auto scores = [&](int b, F2 (&sc)[8]) {
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        if constexpr (S::I4) {
                            F2 a, z;
#pragma unroll
                            for (int g = 0; g < S::GK; ++g) {
                                // four tokens' scales and minima a load, the same for all rows
                                const float4 s = *reinterpret_cast<const float4 *>(par + g * 128 + 16 * b + 4 * (q / 2)), m = *reinterpret_cast<const float4 *>(par + g * 128 + 64 + 16 * b + 4 * (q / 2));
                                const F2 s2 = q & 1 ? pk(s.z, s.w) : pk(s.x, s.y), m2 = q & 1 ? pk(m.z, m.w) : pk(m.x, m.y);
                                const F2 y = pk(__uint_as_float(x[g][2 * q]), __uint_as_float(x[g][2 * q + 1]));
                                a = g ? fma2(s2, y, a) : mul2(s2, y);
                                z = g ? fma2(m2, qs[g], z) : mul2(m2, qs[g]);
                            }
                            sc[q] = fma2(a, pk(fac, fac), z);
                        } else {
                            sc[q] = pk(__uint_as_float(x[0][2 * q]), __uint_as_float(x[0][2 * q + 1]));
                        }
                    }
                    if (mask) {
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            float2 f = up(sc[q]);
                            if ((bad >> b) & 1) f.x = f.y = __int_as_float(0x7fc00000);
                            if (j0 + 16 * b + 2 * q >= vis) f.x = -INFINITY;
                            if (j0 + 16 * b + 2 * q + 1 >= vis) f.y = -INFINITY;
                            sc[q] = pk(f.x, f.y);
                        }
                    }
                };
                // With 32 keys a thread their scores stay in registers; with 64 (bf16: they are what TMEM holds) both passes read
                // them, in loops short enough for the instruction cache.
                constexpr int BLOCKS = S::KEYS / 16;
                F2 kept[S::SW > 1 ? BLOCKS : 1][8];
                float top = -INFINITY, e = 0.f;
                bring(b0);
#pragma unroll(S::SW > 1 ? BLOCKS : 1)
                for (int i = 0; i < BLOCKS; ++i) {
                    F2 (&sc)[8] = kept[S::SW > 1 ? i : 0];
                    scores(b0 + i, sc);
                    if (i + 1 < BLOCKS) bring(b0 + i + 1);
                    else if (S::SW == 1) bring(b0);              // (for the second pass)
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        const float2 f = up(sc[q]);
                        top = fmaxf(top, fmaxf(f.x, f.y));
                    }
                }
                if constexpr (S::SW > 1) {
                    float *at2 = xch + (use & 1) * 256;
                    at2[wg * 128 + r] = top;
                    tc::named_bar(3, 256);
                    top = fmaxf(top, at2[(wg ^ 1) * 128 + r]);
                }
                if constexpr (S::I4) {
                    // every value scale that the row sees here is below 2^e (as in paged_attend.cuh)
                    float big = 0.f;
                    if (mask) {
#pragma unroll 4
                        for (int j = 0; j < 64; ++j)
                            if (j0 + j < vis)
#pragma unroll
                                for (int v = 0; v < S::PV; ++v) big = fmaxf(big, par[(S::PK + v) * 128 + j]);
                    } else {
                        const float *tops = reinterpret_cast<const float *>(sm + S::AT_TOP) + slot * 16;
#pragma unroll
                        for (int w = 0; w < 8; ++w) big = fmaxf(big, tops[w]);
                    }
                    e = (float)(max((int)(__float_as_uint(big) >> 23), 113) - 126) - 14.f;
                }
                const float mnew = fmaxf(m, top + e), at_base = mnew == -INFINITY ? 0.f : mnew, cr = ex2(m - at_base);
                m = mnew;
                if (wg == 0) corr[(use & 3) * 128 + r] = cr;
                F2 lsum = pk(0.f, 0.f), ms[S::PV];
#pragma unroll
                for (int v = 0; v < S::PV; ++v) ms[v] = pk(0.f, 0.f);
                const F2 nb = pk(-at_base, -at_base);
#pragma unroll(S::SW > 1 ? BLOCKS : 1)
                for (int i = 0; i < BLOCKS; ++i) {
                    const int b = b0 + i;
                    uint32_t hi[S::GV][8], lo[S::GV][8];
                    F2 (&sc)[8] = kept[S::SW > 1 ? i : 0];
                    if constexpr (S::SW == 1) {
                        scores(b, sc);
                        if (i + 1 < BLOCKS) bring(b + 1);
                    }
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        const float2 d = up(add2(sc[q], nb));
                        const F2 p = pk(ex2(d.x), ex2(d.y));
                        lsum = add2(lsum, p);
#pragma unroll
                        for (int g = 0; g < S::GV; ++g) {
                            F2 w = p;
                            if constexpr (S::I4) {
                                const float4 s = *reinterpret_cast<const float4 *>(par + (S::PK + g) * 128 + 16 * b + 4 * (q / 2)), mm = *reinterpret_cast<const float4 *>(par + (S::PK + g) * 128 + 64 + 16 * b + 4 * (q / 2));
                                const F2 s2 = q & 1 ? pk(s.z, s.w) : pk(s.x, s.y), m2 = q & 1 ? pk(mm.z, mm.w) : pk(mm.x, mm.y);
                                w = mul2(p, s2);
                                ms[g] = fma2(p, m2, ms[g]);
                            }
                            split2<S::I4>(up(w), hi[g][q], lo[g][q]);
                        }
                    }
#pragma unroll
                    for (int g = 0; g < S::GV; ++g) {
                        // the columns of these keys' scores: 8 of the high parts, 8 of the low ones, one step of the product
                        tc::tmem_st8(ts + 64 * g + 16 * b, hi[g]);
                        tc::tmem_st8(ts + 64 * g + 16 * b + 8, lo[g]);
                    }
                }
                const float2 ls = up(lsum);
                l = fmaf(l, cr, ls.x + ls.y);
                if constexpr (S::I4) {
#pragma unroll
                    for (int v = 0; v < S::PV; ++v) {
                        const float2 x = up(ms[v]);
                        mn[v] = fmaf(mn[v], cr, x.x + x.y);
                        // value groups that are not finite were put to 0: the rows that see one
                        const unsigned long long gone = poison[(use & 7) * S::PV + v];
                        if (gone) {
                            const int n = vis - j0;
                            if (gone & (n >= 64 ? ~0ull : n <= 0 ? 0ull : (1ull << n) - 1)) mn[v] = __int_as_float(0x7fc00000);
                        }
                    }
                }
                tc::tmem_wait_st();
                tc::tc_fence_before();
                tc::mbar_arrive(p_full + 8 * (use & 1));
            }
            if constexpr (S::SW > 1) {                       // the last keys' sums to the first warpgroup
                tc::named_bar(3, 256);
                if (wg == 1) {
                    xch[r] = l;
#pragma unroll
                    for (int v = 0; v < S::PV; ++v) xch[(1 + v) * 128 + r] = mn[v];
                }
                tc::named_bar(3, 256);
                if (wg == 1) return;
                l += xch[r];
#pragma unroll
                for (int v = 0; v < S::PV; ++v) mn[v] += xch[(1 + v) * 128 + r];
            }
            fin[r] = m;
            fin[128 + r] = c.s.len < 0 ? __int_as_float(0x7fc00000) : l;
#pragma unroll
            for (int v = 0; v < S::PV; ++v) fin[(2 + v) * 128 + r] = mn[v];
        }, nothing, true);
        tc::named_bar(1, S::THREADS);
        if (warp == 0) tc::tmem_dealloc(tb, 512);
    } else if (warp < S::PROD) {
        if constexpr (S::R_HELP > S::LAUNCH) take_registers<S::R_HELP>();
        float o[S::DV / 2];                                                    // a row, half the channels
        Segment out[2];                                                        // what reaches out: the first segment, the last
        out[0].key = out[1].key = -1;
        segments([&](const Cursor &c, int t0, int T, unsigned done) {
            const int rows = c.s.cnt * A.G, R0 = c.rb * S::ROWS;
            // ---- helpers
            const int ht = threadIdx.x - 32 * S::HELP, r = 32 * (warp & 3) + lane, half = (warp - S::HELP) >> 2;
            const int vis = R0 + r < rows ? c.s.len - c.s.cnt + (R0 + r) / A.G + 1 : 0;
#pragma unroll
            for (int x = 0; x < S::DV / 2; ++x) o[x] = 0.f;
            bool ok = true;
            for (int k = 0; k < T + 2 && ok; ++k) {
                if (k < T) {
                    const unsigned use = done + k;
                    const int slot = use % S::KB, j0 = (t0 + k) * 64;
                    char *kv = sm + S::AT_KV + slot * S::KV;
                    if constexpr (S::I4) {
                        ok = wait_for(raw_full + 8 * (use & 1), use >> 1, dead, A.status);
                        if (ok && use >= S::KB) ok = wait_for(kv_free + 8 * slot, use / S::KB - 1, dead, A.status);
                        ok = __all_sync(0xffffffffu, ok);    // (a warp gives up as one: what follows is the whole warp's)
                        if (!ok) break;
                        const char *raw = sm + S::AT_RAW + (use & 1) * S::RAW;
                        for (int x = ht; x < S::PL * 128; x += 256) {
                            const int p = x >> 7, tok = (x >> 1) & 63, hh = x & 1;
                            const uint4 w = *reinterpret_cast<const uint4 *>(raw + (tok >> 4) * S::STRIP + p * kPlaneI4 + (tok & 15) * 32 + 16 * hh);
                            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
                            char *dst = kv + p * 8192 + tok * 128;
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                const uint32_t v = u[q] >> 8;
                                *reinterpret_cast<uint4 *>(dst + (((4 * hh + q) ^ (tok & 7)) << 4)) =
                                    make_uint4(u[q] & 0x000F000Fu, u[q] & 0x00F000F0u, v & 0x000F000Fu, v & 0x00F000F0u);
                            }
                        }
                        float *par = reinterpret_cast<float *>(sm + S::AT_PAR + slot * S::PARAMS);
                        float big = 0.f;
                        for (int x = ht; x < S::PL * 64; x += 256) {
                            const int p = x >> 6, tok = x & 63;
                            float2 v = make_float2(0.f, 0.f);
                            if (j0 + tok < c.most) v = __half22float2(*reinterpret_cast<const __half2 *>(raw + (tok >> 4) * S::STRIP + p * kPlaneI4 + 512 + (tok & 15) * 4));
                            if (p >= S::PK) {            // a weight of 0 must not meet a NaN: such a group is 0 here and remembered
                                const bool gone = !(fabsf(v.x) < INFINITY && fabsf(v.y) < INFINITY);
                                if (gone) {
                                    v = make_float2(0.f, 0.f);
                                    atomicOr(&poison[(use & 7) * S::PV + p - S::PK], 1ull << tok);
                                }
                            }
                            par[p * 128 + tok] = v.x;
                            par[p * 128 + 64 + tok] = v.y;
                            if (p >= S::PK) big = fmaxf(big, v.x);
                        }
                        big = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(big)));   // (not negative)
                        if (lane == 0) reinterpret_cast<float *>(sm + S::AT_TOP)[slot * 16 + warp - S::HELP] = big;
                        tc::fence_async_smem();
                        tc::mbar_arrive(kv_full + 8 * slot);
                        tc::mbar_arrive(raw_free + 8 * (use & 1));
                    } else {
                        ok = __all_sync(0xffffffffu, wait_for(kv_full + 8 * slot, use / S::KB, dead, A.status));
                        if (!ok) break;
                        if (bad_of[use & 7] || j0 + 64 > c.least) {
                            // value rows past what was brought hold anything, and a value that is not finite must not meet a
                            // weight of 0: both go to 0 here, the latter remembered by the rows that see it
                            const int t = ht >> 2, q4 = ht & 3;          // a token, a quarter of its channels
                            const bool gone = j0 + t >= c.most || ((bad_of[use & 7] >> (t >> 4)) & 1);
                            uint32_t found = 0;
#pragma unroll
                            for (int p = 0; p < S::PV; ++p)
#pragma unroll
                                for (int q = 0; q < 2; ++q) {
                                    uint4 *at4 = reinterpret_cast<uint4 *>(kv + (S::PK + p) * 8192 + t * 128 + (((2 * q4 + q) ^ (t & 7)) << 4));
                                    uint4 w = *at4;
                                    uint32_t *u = &w.x;
                                    bool touched = gone;
#pragma unroll
                                    for (int x = 0; x < 4; ++x) {
                                        const uint32_t f = gone ? 0xffffffffu : __vcmpeq2(u[x] & 0x7f807f80u, 0x7f807f80u);
                                        touched = touched || f;
                                        u[x] &= ~f;
                                        if (!gone) found |= f;
                                    }
                                    if (touched) *at4 = w;
                                }
                            if (found) atomicOr(bad_of + 8 + (use & 7), 1);
                        }
                        tc::fence_async_smem();
                        tc::mbar_arrive(v_ok + 8 * slot);
                    }
                }
                if (k >= 2) {
                    const unsigned use = done + k - 2;
                    const int ob = use % S::OB;
                    ok = __all_sync(0xffffffffu, wait_for(o_full + 8 * ob, use / S::OB, dead, A.status));
                    if (!ok) break;
                    tc::tc_fence_after();
                    const float cr = corr[(use & 3) * 128 + r];
                    const uint32_t to = tb + ((uint32_t)(32 * (warp & 3)) << 16) + S::COL_O + ob * S::DV + half * (S::DV / 2);
#pragma unroll
                    for (int b = 0; b < S::DV / 32; ++b) {
                        uint32_t x[16];
                        tc::tmem_ld16(to + 16 * b, x);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int q = 0; q < 16; ++q) o[16 * b + q] = fmaf(o[16 * b + q], cr, __uint_as_float(x[q]));
                    }
                    if (!S::I4 && bad_of[8 + (use & 7)]) {   // values that are not finite: from memory, for the rows that see them
                        const int j0 = (t0 + k - 2) * 64;
#pragma unroll 1
                        for (int j = j0; j < min(j0 + 64, min(vis, c.most)); ++j) {
                            const int pgi = j / A.P.page_size, pg = A.P.table[(int64_t)c.n * A.P.max_pages + pgi];
                            if (pg < 0 || pg >= A.P.num_pages) continue;
                            const char *plane = A.P.pool + (int64_t)pg * A.P.page_bytes + (int64_t)c.h * A.P.block_bytes +
                                                (int64_t)((j - pgi * A.P.page_size) / kStrip) * S::STRIP + S::PK * kPlaneBf16;
#pragma unroll
                            for (int x = 0; x < S::DV / 2; ++x) {
                                const int ch = half * (S::DV / 2) + x;
                                const uint16_t v = *reinterpret_cast<const uint16_t *>(plane + (ch >> 6) * kPlaneBf16 + (j & 15) * 128 + ((((ch & 63) >> 3) ^ (j & 7)) << 4) + (ch & 7) * 2);
                                if ((v & 0x7f80) == 0x7f80) o[x] = __int_as_float(0x7fc00000);
                            }
                        }
                    }
                    tc::tc_fence_before();
                    tc::mbar_arrive(o_free + 8 * ob);
                }
            }
        }, [&](const Cursor &c, unsigned base, int t0, int t1) {
            // the segment's end: O through shared memory (over the operand tiles) to the output, or to the workspace
            const int rows = c.s.cnt * A.G, R0 = c.rb * S::ROWS, ht = threadIdx.x - 32 * S::HELP;
            const bool begins = t0 == 0, ends = t1 == c.s.tiles;
            float *stage = reinterpret_cast<float *>(sm + S::AT_KV);           // rows of DV + 4
            const int r = 32 * (warp & 3) + lane, half = (warp - S::HELP) >> 2;
#pragma unroll
            for (int w = 0; w < S::DV / 16; ++w) {
                const int ch = half * (S::DV / 2) + 8 * w;
                float x[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    if constexpr (S::I4) x[q] = fmaf(o[8 * w + (q < 4 ? 2 * q : 2 * q - 7)], q & 1 ? 1048576.f : 16777216.f, fin[(2 + ch / 64) * 128 + r]);
                    else x[q] = o[8 * w + q];
                }
                float4 *dst = reinterpret_cast<float4 *>(stage + r * (S::DV + 4) + ch);
                dst[0] = make_float4(x[0], x[1], x[2], x[3]);
                dst[1] = make_float4(x[4], x[5], x[6], x[7]);
            }
            tc::named_bar(2, 256);
            float *rec = A.partial + ((size_t)blockIdx.x * 2 + (begins ? 1 : 0)) * S::RECORD;
            const int live = min(S::ROWS, rows - R0);
#pragma unroll 1
            for (int x = ht; x < live * (S::DV / 4); x += 256) {
                const int rr = x / (S::DV / 4), ch = 4 * (x - rr * (S::DV / 4));
                const float4 v = *reinterpret_cast<const float4 *>(stage + rr * (S::DV + 4) + ch);
                if (begins && ends) {
                    store4(A, S::DV, c.s.q0, c.s.len - c.s.cnt, c.h, R0 + rr, ch, v, fin[128 + rr]);
                } else {
                    *reinterpret_cast<float4 *>(rec + 256 + rr * S::DV + ch) = v;
                    if (ch == 0) {
                        rec[rr] = fin[rr];
                        rec[128 + rr] = fin[128 + rr];
                    }
                }
            }
            if (!(begins && ends)) {
                const int key = (int)(base + extra);
                const Segment sg{key, key + c.s.tiles - 1, (begins ? 1 : 0) | (ends ? 2 : 0), c.h, c.rb, c.s.q0, rows, c.s.len - c.s.cnt};
                if (begins) out[1] = sg;
                else out[0] = sg;
            }
        }, true);
        tc::named_bar(1, S::THREADS);

        // blocks that several CTAs share: the last of them to get here joins the records, in the row's order
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
            const Segment sg = i ? out[1] : out[0];
            if (sg.key < 0) continue;
            const unsigned first = split.owner(sg.key), last = split.owner(sg.last);
            __threadfence();
            tc::named_bar(2, 256);
            if (threadIdx.x == 32 * S::HELP) arrived = atomicAdd(A.counters + first, 1u);
            tc::named_bar(2, 256);
            if (arrived != last - first) continue;
            __threadfence();
            if (threadIdx.x == 32 * S::HELP) A.counters[first] = 0;
            auto rec = [&](unsigned b) { return A.partial + ((size_t)b * 2 + (b == first ? 1 : 0)) * S::RECORD; };
            // each row's weights of the records, then the weighted sums, several loads on their way at a time
            float *wt = reinterpret_cast<float *>(sm + S::AT_JOIN);            // [records][128], then the rows' sums
            const int ht = threadIdx.x - 32 * S::HELP, live = min(S::ROWS, sg.rows - sg.rb * S::ROWS);
            const unsigned count = last - first + 1;
            if (ht < live) {
                float top = -INFINITY, l = 0.f;
#pragma unroll 8
                for (unsigned b = 0; b < count; ++b) top = fmaxf(top, __ldcg(rec(first + b) + ht));
#pragma unroll 4
                for (unsigned b = 0; b < count; ++b) {
                    const float f = weight(__ldcg(rec(first + b) + ht), top);
                    l = fmaf(f, __ldcg(rec(first + b) + 128 + ht), l);
                    wt[b * 128 + ht] = f;
                }
                wt[count * 128 + ht] = l;
            }
            tc::named_bar(2, 256);
            constexpr int C4 = S::DV / 4, ITEMS = 4;
            for (int x0 = ht; x0 < live * C4; x0 += 256 * ITEMS) {
                float4 v4[ITEMS];
#pragma unroll
                for (int q = 0; q < ITEMS; ++q) v4[q] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
                for (unsigned b = 0; b < count; ++b) {
                    const float4 *from = reinterpret_cast<const float4 *>(rec(first + b) + 256);
                    float4 v[ITEMS];
                    float f[ITEMS];
#pragma unroll
                    for (int q = 0; q < ITEMS; ++q) {
                        const int x = min(x0 + 256 * q, live * C4 - 1);
                        v[q] = __ldcg(from + x);
                        f[q] = wt[b * 128 + x / C4];
                    }
#pragma unroll
                    for (int q = 0; q < ITEMS; ++q) {
                        v4[q].x = fmaf(f[q], v[q].x, v4[q].x); v4[q].y = fmaf(f[q], v[q].y, v4[q].y); v4[q].z = fmaf(f[q], v[q].z, v4[q].z); v4[q].w = fmaf(f[q], v[q].w, v4[q].w);
                    }
                }
#pragma unroll
                for (int q = 0; q < ITEMS; ++q) {
                    const int x = x0 + 256 * q, r = x / C4;
                    if (x < live * C4) store4(A, S::DV, sg.q0, sg.past, sg.h, sg.rb * S::ROWS + r, 4 * (x - r * C4), v4[q], wt[count * 128 + r]);
                }
            }
            tc::named_bar(2, 256);
        }
    } else {
        give_registers<S::R_REST>();
        const bool starve = A.test_limit != 0 && blockIdx.x == 0;
        unsigned issued = 0, scored = 0, weighed = 0;    // tiles whose copies, scores' and outputs' products are issued
        segments([&](const Cursor &c, int t0, int T, unsigned done) {
            if (warp == S::PROD) {
                // ---- producer
                for (int k = 0; k < T; ++k) {
                    const unsigned use = done + k;
                    const int strip = (t0 + k) * 4 + (S::I4 ? lane : lane / S::PL), slot = use % S::KB;
                    const bool mine = (S::I4 ? lane < 4 : lane < 4 * S::PL) && 16 * strip < c.most;
                    int pg = -1, j = 0;
                    if (mine) {
                        j = A.per_page_inv ? (int)__umulhi((unsigned)strip, A.per_page_inv) : strip;
                        pg = A.P.table[(int64_t)c.n * A.P.max_pages + j];
                    }
                    bool ok = true;
                    if (S::I4 ? use >= 2 : use >= S::KB)
                        ok = S::I4 ? wait_for(raw_free + 8 * (use & 1), (use >> 1) - 1, dead, A.status) : wait_for(kv_free + 8 * slot, use / S::KB - 1, dead, A.status);
                    if (!__all_sync(0xffffffffu, ok)) break;
                    const bool good = mine && pg >= 0 && pg < A.P.num_pages;
                    const unsigned have = __ballot_sync(0xffffffffu, good), wrong = __ballot_sync(0xffffffffu, mine && !good);
                    const uint32_t full = S::I4 ? raw_full + 8 * (use & 1) : kv_full + 8 * slot;
                    const bool skip = starve && use == 0;
                    if (lane == 0) {
                        int bits = 0;
                        for (int s = 0; s < 4; ++s) bits |= ((wrong >> (S::I4 ? s : s * S::PL)) & 1) << s;
                        bad_of[use & 7] = bits;
                        bad_of[8 + (use & 7)] = 0;
                        if constexpr (S::I4)
                            for (int v = 0; v < S::PV; ++v) poison[(use & 7) * S::PV + v] = 0;
                        if (!skip) tc::mbar_arrive_expect_tx(full, __popc(have) * (S::I4 ? S::STRIP : kPlaneBf16));
                    }
                    __syncwarp();
                    issued = use + 1;
                    if (good && !skip) {
                        const char *src = A.P.pool + (int64_t)pg * A.P.page_bytes + (int64_t)c.h * A.P.block_bytes + (int64_t)(strip - j * A.per_page) * S::STRIP;
                        if constexpr (S::I4) {
                            tc::bulk_g2s(sm32 + S::AT_RAW + (use & 1) * S::RAW + lane * S::STRIP, src, S::STRIP, full);
                        } else {
                            const int p = lane % S::PL, s = lane / S::PL;
                            tc::bulk_g2s(sm32 + S::AT_KV + slot * S::KV + p * 8192 + s * kPlaneBf16, src + p * kPlaneBf16, kPlaneBf16, full);
                        }
                    }
                    if (starve && use == 1) {            // (with the second tile's copies in flight)
                        if (!tc::mbar_wait_bounded(S::I4 ? raw_full : kv_full, 0, A.test_limit) && lane == 0) {
                            *dead = 1;
                            atomicOr(A.status, 2u);
                        }
                        break;
                    }
                }
            } else if (warp == S::PROD + 1) {
                // ---- MMA: the whole warp comes along, so that addresses are uniform, and one thread issues
                constexpr uint32_t id_s = idesc16(S::I4, 128, 64, false), id_o = idesc16(S::I4, 128, S::I4 ? 64 : S::DV, true);
                const uint32_t tu = __shfl_sync(0xffffffffu, tb, 0);
                for (int k = 0; k < T + 1; ++k) {
                    if (k < T) {
                        const unsigned use = done + k;
                        const int slot = use % S::KB;
                        if (!__all_sync(0xffffffffu, wait_for(kv_full + 8 * slot, use / S::KB, dead, A.status))) break;
                        tc::tc_fence_after();
                        const uint32_t ts = tu + __shfl_sync(0xffffffffu, (use & 1) * S::SB, 0), kv = __shfl_sync(0xffffffffu, sm32 + S::AT_KV + slot * S::KV, 0);
                        if (elect()) {
#pragma unroll
                            for (int p = 0; p < S::PK; ++p) {
                                const uint64_t dk = tc::sdesc_kmajor_sw128(kv + p * 8192);
                                const uint32_t d = ts + (S::I4 ? 64 * p : 0);
#pragma unroll
                                for (int i = 0; i < 4; ++i)
#pragma unroll
                                    for (int part = 0; part < 2; ++part) {
                                        const uint32_t more = i != 0 || part != 0 || (!S::I4 && p != 0);
                                        if constexpr (S::QT) tc::mma_bf16_ta(d, tu + S::COL_Q + part * (S::DQK / 2) + 32 * p + 8 * i, tc::dadd(dk, 32 * i), id_s, more);
                                        else tc::mma_bf16(d, tc::dadd(tc::sdesc_kmajor_sw128(sm32 + part * S::Q_PART + p * 16384), 32 * i), tc::dadd(dk, 32 * i), id_s, more);
                                    }
                            }
                            tc::mma_commit(s_full + 8 * (use & 1));
                        }
                        scored = use + 1;
                    }
                    if (k >= 1) {
                        const unsigned use = done + k - 1;
                        const int slot = use % S::KB, ob = use % S::OB;
                        bool ok = wait_for(p_full + 8 * (use & 1), use >> 1, dead, A.status);
                        if (ok && use >= S::OB) ok = wait_for(o_free + 8 * ob, use / S::OB - 1, dead, A.status);
                        if (ok && !S::I4) ok = wait_for(v_ok + 8 * slot, use / S::KB, dead, A.status);
                        if (!__all_sync(0xffffffffu, ok)) break;
                        tc::tc_fence_after();
                        const uint32_t ts = tu + __shfl_sync(0xffffffffu, (use & 1) * S::SB, 0), kv = __shfl_sync(0xffffffffu, sm32 + S::AT_KV + slot * S::KV, 0),
                                       to = tu + __shfl_sync(0xffffffffu, S::COL_O + ob * S::DV, 0);
                        if (elect()) {
#pragma unroll
                            for (int v = 0; v < S::GV; ++v) {    // (bf16: all value channels at once)
                                const uint64_t dv = tc::sdesc_mnmajor_sw128(kv + (S::PK + v) * 8192, 8192);
#pragma unroll
                                for (int i = 0; i < 4; ++i)
#pragma unroll
                                    for (int part = 0; part < 2; ++part)
                                        tc::mma_bf16_ta(to + 64 * v, ts + 64 * v + 16 * i + 8 * part, tc::dadd(dv, 2048 * i), id_o, i != 0 || part != 0);
                            }
                            tc::mma_commit(o_full + 8 * ob);
                            tc::mma_commit(kv_free + 8 * slot);
                        }
                        weighed = use + 1;
                    }
                }
            }
        }, [&](const Cursor &, unsigned, int, int) {
            if (*dead == 0) return;
            // the CTA gives up: what is in flight ends before its shared and tensor memory go
            constexpr unsigned RING = S::I4 ? 2 : S::KB;
            if (warp == S::PROD)
                for (unsigned use = issued > RING ? issued - RING : 0; use < issued; ++use) {
                    if (starve && use == 0) continue;
                    tc::mbar_wait_bounded((S::I4 ? raw_full : kv_full) + 8 * (use % RING), (use / RING) & 1, kWaitTries);
                }
            if (warp == S::PROD + 1) {
                const unsigned s = scored - 1, o = weighed - 1;
                if (scored > 0) tc::mbar_wait_bounded(s_full + 8 * (s & 1), (s >> 1) & 1, kWaitTries);
                if (weighed > 0) {
                    tc::mbar_wait_bounded(o_full + 8 * (o % S::OB), (o / S::OB) & 1, kWaitTries);
                    tc::mbar_wait_bounded(kv_free + 8 * (o % S::KB), (o / S::KB) & 1, kWaitTries);
                }
            }
        }, false);
        tc::named_bar(1, S::THREADS);
    }
}

template <class S> cudaError_t launch_rows(const Args &A, cudaStream_t stream) {
    static std::atomic<uint64_t> done{0};
    static std::atomic<bool> fits{false};
    cudaError_t e;
    if (!fits.load(std::memory_order_acquire)) {         // roles take registers that others give: the launch must have had them
        cudaFuncAttributes attr;
        if ((e = cudaFuncGetAttributes(&attr, (const void *)rows_kernel<S>)) != cudaSuccess) return e;
        if (attr.numRegs < S::LAUNCH) return cudaErrorInvalidConfiguration;
        fits.store(true, std::memory_order_release);
    }
    if ((e = smem_attr_once((const void *)rows_kernel<S>, S::SMEM, done)) != cudaSuccess) return e;
    int dev = 0, sms = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    rows_kernel<S><<<sms < kMaxCtas ? sms : kMaxCtas, S::THREADS, S::SMEM, stream>>>(A);
    count_launch();
    return cudaGetLastError();
}

// up to 192 and 128 channels: what fits tensor memory
template <bool I4> cudaError_t pick_rows(int dqk, int dv, const Args &A, cudaStream_t s) {
    if (dqk == 64) return dv == 64 ? launch_rows<RowsShape<64, 64, I4>>(A, s) : launch_rows<RowsShape<64, 128, I4>>(A, s);
    if (dqk == 128) return dv == 64 ? launch_rows<RowsShape<128, 64, I4>>(A, s) : launch_rows<RowsShape<128, 128, I4>>(A, s);
    return dv == 64 ? launch_rows<RowsShape<192, 64, I4>>(A, s) : launch_rows<RowsShape<192, 128, I4>>(A, s);
}

cudaError_t run_i4_rows(int dqk, int dv, const Args &A, cudaStream_t s);
cudaError_t run_bf16_rows(int dqk, int dv, const Args &A, cudaStream_t s);

}  // namespace attend
}  // namespace k3kda
