// paged_append.cu -- new key and value rows into the paged cache (keys rotated on the way), and rows
// back out of it as values, on sm_103a.
//
// Both move every element once; what they have to beat is their own arithmetic, appending some 34 instructions a channel (by the
// profile: the slow paths below take a whole warp of eight groups when one group needs them).  Four lanes hold a group (64
// channels of a token and head), 16 channels each; a lane keeps its head and channels and goes through its CTA's tokens, so
// that addresses, the rotation's layout and its table's place are worked out once.  Lanes of
// a warp hold the same channels of eight heads, so that keys that turn and values that do not seldom share one.
// A CTA finds its tokens' sequences and pages once (a 32-way search of cu_seqlens, one warp a token) and forms their cosines
// and sines once for all heads.  Pairs of channels go through packed FP32 instructions (fma.rn.f32x2).
//
// 4-bit rounding.  The stored values are those of the definition in exact arithmetic, so that what
// the cache holds does not hang on how FP32 rounds:
//   - The plain path rounds t = (x - m) / s to the nearest whole number by FP32 and keeps the largest distance to it; with
//     that below 1/2 by more than FP32's error every code is right.  It also wants fp16's roundings of the minimum and
//     the scale to be clear, and codes that need no clamp (a scale that is a normal fp16 number, a minimum whose rounding is
//     small next to it).
//   - Else, in a group of channels that are not turned (exact in FP32: m is one rounding, s was clear), a code is decided
//     by the sign of (x - m) - (c + 1/2) s, where (c + 1/2) s has at most 16 bits: one fma and, next to a tie, the
//     rounding error of x - m.  Ties are common there (bf16 values): one group in 30.  c comes from t, or, where a clamp is
//     needed or m is more than 10^6 s (x / s - m / s has no fraction left), from x - m.
//   - Else (turned channels, FP32 errors of up to kSlack of the pair: about one group in 500; or a rotation that FP32 may
//     overflow) the warp repeats the group in double, two channels a lane, with the angle's sine and cosine in double.
//
// Measured (26,339 prompt tokens, 32 heads of 128 + 128 channels, 553 MB each way): append 248 us, 2.2 TB/s, where instruction
// issue is the bound (57 M warp instructions for a quarter of it, HBM at a fifth of its rate); read 113 us, 4.9 TB/s, 72 % of
// a copy's rate.  FP32 rows of 9,366 tokens, 8 heads of 192 + 128 channels, into bf16 pages and back: 50 us (append 34, read 19).
// CTAs of 128 and 64 threads, or scalar FP32 in place of the packed instructions: 385 to 612 us for the first append and read
// instead of 358.
#include <math.h>

#include "paged.cuh"

namespace k3kda {
namespace {

constexpr int kThreads = 256;
constexpr int kGroups = kThreads / 4;     // most groups of a CTA
constexpr int kDepth = 16;                // most tokens a lane goes through
constexpr int kTokens = 128;              // most tokens of a CTA
// Bound on the FP32 error of a turned channel, relative to the largest of the pair's two channels (times mscale).  The cosine
// and sine are off by at most 1.7e-7 each: 2^-24 from sincospif (1 ulp below 1), 4.7e-8 from the angle's own rounding
// (at most 1/8 turn, 24 bits), 2^-24 from the factor mscale; two products add 2^-24 of one and 2^-24 sqrt(2) of the sum.
constexpr float kSlack = 4.8e-7f;
constexpr float kSlackPlain = 3.6e-7f;    // without the factor: 1.1e-7 each

struct AppendArgs {
    Paged P;
    View k, v;
    const int32_t *cu;
    int T;
    Rope r;
    int tokens;                           // tokens of a CTA
    int parts;                            // CTAs that share the same tokens
    int groups;                           // groups of a CTA: its share of heads * planes, at most kGroups
    int warps, side;                      // warps for them, and how many tokens lie side by side (warps * side <= 8)
};

struct Place {                            // where a CTA's token goes; page < 0: nowhere
    int64_t at;                           // its strip in (page, head 0)'s block: bytes from the pool's start
    int pos, page;
};

// Sequence of token t: the last n with cu[n] <= t; each round looks at 32 entries at once.
__device__ __forceinline__ int find_seq(const int32_t *cu, int N, int t, int lane) {
    int lo = 0, hi = N;                   // cu[lo] <= t < cu[hi]
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int at = lo + lane * step;
        const unsigned m = __ballot_sync(0xffffffffu, at < hi && cu[at] <= t);
        const int last = 31 - __clz(m | 1u);
        lo += last * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

// One warp per token of the CTA: its place.  A malformed cu_seqlens cannot send it outside the table.
__device__ __forceinline__ void find_places(const Paged &P, const int32_t *cu, int T, int t0, int count, Place *place) {
    const int lane = threadIdx.x & 31;
    for (int i = threadIdx.x >> 5; i < count; i += (int)blockDim.x >> 5) {
        const int t = t0 + i;
        const int n = cu ? find_seq(cu, P.N, t, lane) : t;
        if (lane == 0) {
            Place w{0, -1, -1};
            int b = t, e = t + 1;
            if (cu) seq_bounds(cu, n, T, b, e);
            const int len = paged_len(P, n);
            const int64_t pos = (int64_t)len - e + t;
            if (len >= 0 && t >= b && t < e && pos >= 0) {
                w.pos = (int)pos;
                w.page = paged_page(P, n, w.pos);
                w.at = (int64_t)w.page * P.page_bytes + (int64_t)(w.pos % P.page_size / kStrip) * P.strip_bytes;
            }
            place[i] = w;
        }
    }
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
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// three-way maximum and minimum; a NaN stays
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
    float r;
    asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// 8 channels as they lie in memory
template <typename T, bool VEC> struct Raw {
    uint32_t w[2 * sizeof(T)];
    __device__ __forceinline__ void load(const T *p) {
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
                const uint4 x = __ldcs(reinterpret_cast<const uint4 *>(p) + i);
                w[4 * i] = x.x; w[4 * i + 1] = x.y; w[4 * i + 2] = x.z; w[4 * i + 3] = x.w;
            }
        } else if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = reinterpret_cast<const uint16_t *>(p)[2 * i] | (uint32_t)reinterpret_cast<const uint16_t *>(p)[2 * i + 1] << 16;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = reinterpret_cast<const uint32_t *>(p)[i];
        }
    }
    __device__ __forceinline__ F2 pair(int i) const {
        if constexpr (sizeof(T) == 2) return pk(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
        else return pk(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    }
};

// channel c's place in the rotation: its pair, its partner's channel and whether it is the second of the two
struct Turn { int pair, partner; bool second; };
__device__ __forceinline__ Turn turn_of(const Rope &r, int c) {
    const int i = c - r.off;
    if (r.inter) return Turn{i >> 1, r.off + (i ^ 1), (i & 1) != 0};
    const bool second = i >= r.half;
    return Turn{second ? i - r.half : i, second ? c - r.half : c + r.half, second};
}

// fp16 nearest to x, within +-65504
__device__ __forceinline__ float half_sat(float x) {
    return __half2float(__float2half_rn(fminf(fmaxf(x, -65504.f), 65504.f)));
}
__device__ __forceinline__ double half_sat(double x) {
    x = x < -65504.0 ? -65504.0 : x > 65504.0 ? 65504.0 : x;
    return (double)__half2float(__double2half(x));
}

// Whether the fp16 rounding h of x may differ from that of some value within d of x: x lies that close to the middle of two
// fp16 numbers, half their spacing (2^-11 of x's power of two, 2^-25 at least) away from h.
__device__ __forceinline__ bool half_unsure(float x, float h, float d) {
    const float gap = fmaxf(__uint_as_float((__float_as_uint(x) & 0x7f800000u) - (11u << 23)), 2.9802322e-8f);
    return fabsf(fabsf(x - h) - gap) <= d;
}

// A group in double by the whole warp: lane l takes channels 2l and 2l + 1 of the plane.  src: the (token, head) row's
// key or value; c0: the plane's first channel in it.
template <typename T> __device__ __noinline__ void group_in_double(const T *src, int c0, const Rope r, bool key, int pos, char *plane, int row) {
    const int lane = threadIdx.x & 31;
    double x[2];
    bool bad = false;                                     // a channel that is not finite
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int c = c0 + 2 * lane + e;
        x[e] = (double)load_elt(src, c, sizeof(T) == 2);
        if (key && c >= r.off && c < r.off + r.dim) {
            const Turn t = turn_of(r, c);
            const double y = (double)load_elt(src, t.partner, sizeof(T) == 2);
            double cs, sn;
            rope_cs_f64(r.phase[t.pair], pos, cs, sn);
            x[e] = (double)r.mscale * (t.second ? x[e] * cs + y * sn : x[e] * cs - y * sn);
        }
        bad = bad || !isfinite(x[e]);
    }
    bad = __any_sync(0xffffffffu, bad);
    double lo = fmin(x[0], x[1]), hi = fmax(x[0], x[1]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        lo = fmin(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = fmax(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    const double m = half_sat(lo), range = fmax(hi - m, 0.0);
    // fp16(range / 15): FP32's quotient is off by less than half a step of fp16, so the result is its rounding or the value next
    // to it; 15 times the value between two neighbours is exact, and the comparison decides (a tie to the even one)
    const float guess = half_sat((float)range * (1.f / 15.f));
    const unsigned bits = __half_as_ushort(__float2half_rn(guess));
    double s = guess;
    const double above = (double)__half2float(__ushort_as_half((unsigned short)(bits + 1))), below = (double)__half2float(__ushort_as_half((unsigned short)(bits - 1)));
    const double up_at = fma(-7.5, s + above, range), down_at = fma(-7.5, s + below, range);     // range - 15 (s + neighbour) / 2
    if (bits < 0x7bff && (up_at > 0.0 || (up_at == 0.0 && (bits & 1)))) s = above;
    else if (bits > 0 && (down_at < 0.0 || (down_at == 0.0 && (bits & 1)))) s = below;
    unsigned byte = 0;
    const float inv = s > 0.0 ? 1.f / (float)s : 0.f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        // FP32's quotient is within 1/4 of the exact one (or beyond the clamp): the code is f or f + 1 by the sign of
        // (x - m) - (f + 1/2) s, f its whole part less 1/4
        const double d = x[e] - m;
        const float f = fminf(fmaxf(rintf((float)d * inv - 0.5f), 0.f), 14.f);
        const double diff = fma(-((double)f + 0.5), s, d);
        const unsigned code = s > 0.0 ? (unsigned)f + (diff > 0.0 || (diff == 0.0 && ((int)f & 1)) ? 1u : 0u) : 0u;
        byte |= code << (4 * e);
    }
    const __half nan = __ushort_as_half(0x7e00);
    reinterpret_cast<uint8_t *>(plane)[row * 32 + lane] = bad ? 0 : (uint8_t)byte;
    if (lane == 0) reinterpret_cast<__half2 *>(plane + 512)[row] = bad ? __halves2half2(nan, nan) : __halves2half2(__double2half(s), __double2half(m));
}

// How a lane's 8 channels c .. c + 7 turn.
enum Mode { kStill, kPairs, kFirst, kSecond, kMixed };     // not; neighbours; as first or second halves; channel by channel
__device__ __forceinline__ Mode mode_of(const Rope &r, int c, bool vec) {
    const int end = r.off + r.dim;
    if (c >= end || c + 8 <= r.off) return kStill;
    const bool inside = vec && c >= r.off && c + 8 <= end;
    if (inside && r.inter && ((c - r.off) & 7) == 0) return kPairs;
    if (inside && !r.inter && (r.half & 7) == 0 && ((c - r.off) & 7) == 0) return c - r.off < r.half ? kFirst : kSecond;
    return kMixed;
}

template <typename T, bool VEC, bool I4>
__global__ void __launch_bounds__(kThreads, 3) append_kernel(const __grid_constant__ AppendArgs A) {
    extern __shared__ __align__(16) float table[];        // [tokens][dim/2 cosines, then as many sines], rows of a multiple of 4
    __shared__ Place place[kTokens];
    const Paged &P = A.P;
    const int part = (int)(blockIdx.x % A.parts);
    const int t0 = (int)(blockIdx.x / A.parts) * A.tokens, n = min(A.tokens, A.T - t0);
    find_places(P, A.cu, A.T, t0, n, place);
    // this lane's group: plane-major, so that a warp holds one plane of several heads
    const int kplanes = P.dqk / 64, lane4 = threadIdx.x & 3;
    const int row_set = (int)(threadIdx.x >> 5) / A.warps, mine = ((int)(threadIdx.x >> 5) - row_set * A.warps) * 8 + (int)(threadIdx.x & 31) / 4;
    const int gi = part * A.groups + mine;
    const bool inside = mine < A.groups && gi < P.heads * P.planes;
    const int plane = inside ? gi / P.heads : 0, head = inside ? gi - plane * P.heads : 0;
    const bool key = plane < kplanes;
    const int c0 = 64 * (key ? plane : plane - kplanes), c = c0 + 16 * lane4;
    const View &src = key ? A.k : A.v;
    const T *row = reinterpret_cast<const T *>(src.p) + (int64_t)t0 * src.ts + (int64_t)head * src.hs;
    const bool turned = key && A.r.dim > 0 && c0 < A.r.off + A.r.dim && c0 + 64 > A.r.off;   // some channel of the group
    const Mode mode0 = turned ? mode_of(A.r, c, VEC) : kStill, mode1 = turned ? mode_of(A.r, c + 8, VEC) : kStill;
    const bool any_turned = __any_sync(0xffffffffu, turned);
    const int tab_half = (A.r.half + 3) & ~3, tab_row = 2 * tab_half;
    char *dst = P.pool + (int64_t)head * P.block_bytes + plane * (I4 ? kPlaneI4 : kPlaneBf16);
    // the first token's rows are on their way before its angles are known
    Raw<T, VEC> r0, r1, y0, y1;
    auto fetch = [&](int t) {
        const T *p = row + (int64_t)t * src.ts;
        r0.load(p + c);
        r1.load(p + c + 8);
        if (mode0 == kFirst || mode0 == kSecond) y0.load(p + (mode0 == kFirst ? c + A.r.half : c - A.r.half));
        if (mode1 == kFirst || mode1 == kSecond) y1.load(p + 8 + (mode1 == kFirst ? c + A.r.half : c - A.r.half));
    };
    if (inside && row_set < n) fetch(row_set);
    __syncthreads();
    for (int i = threadIdx.x; i < n * A.r.half; i += blockDim.x) {
        const int t = i / A.r.half, p = i - t * A.r.half;
        const float2 v = rope_cs(A.r.phase[p], place[t].pos);
        table[t * tab_row + p] = v.x * A.r.mscale;
        table[t * tab_row + tab_half + p] = v.y * A.r.mscale;
    }
    __syncthreads();
#pragma unroll 1
    for (int t = row_set; t < n; t += A.side) {
        const Place w = place[t];
        F2 x[8];
        float mag = 0.f;                                  // largest channel of the lane's pairs that turn
        auto turn = [&](const Raw<T, VEC> &r, const Raw<T, VEC> &y, Mode mode, int cr, F2 *out) {
            if (mode == kStill || mode == kMixed) {
#pragma unroll
                for (int q = 0; q < 4; ++q) out[q] = r.pair(q);
                if (mode == kStill) return;
                float v[8];                               // some channels turn, or the rows are not aligned: one at a time, from memory
                const T *p = row + (int64_t)t * src.ts;
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    v[q] = load_elt(p, cr + q, sizeof(T) == 2);
                    if (cr + q < A.r.off || cr + q >= A.r.off + A.r.dim) continue;
                    const Turn tn = turn_of(A.r, cr + q);
                    const float u = load_elt(p, tn.partner, sizeof(T) == 2);
                    const float cs = table[t * tab_row + tn.pair], sn = table[t * tab_row + tab_half + tn.pair];
                    mag = fmaxf(mag, fmaxf(fabsf(v[q]), fabsf(u)));
                    v[q] = tn.second ? v[q] * cs + u * sn : v[q] * cs - u * sn;
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) out[q] = pk(v[2 * q], v[2 * q + 1]);
                return;
            }
            const int i = cr - A.r.off, p = mode == kPairs ? i / 2 : mode == kFirst ? i : i - A.r.half;
            const float *tc = table + t * tab_row + p, *ts = tc + tab_half;
            if (mode == kPairs) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const F2 a = r.pair(q);
                    const float2 b = up(a);
                    mag = fmaxf(mag, fmaxf(fabsf(b.x), fabsf(b.y)));
                    out[q] = fma2(a, pk(tc[q], tc[q]), mul2(pk(b.y, b.x), pk(-ts[q], ts[q])));
                }
            } else {
                const F2 sg = mode == kFirst ? pk(-1.f, -1.f) : pk(1.f, 1.f);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const F2 a = r.pair(q), b = y.pair(q);
                    const float2 fa = up(a), fb = up(b), cs = *reinterpret_cast<const float2 *>(tc + 2 * q), sn = *reinterpret_cast<const float2 *>(ts + 2 * q);
                    mag = fmaxf(mag, fmaxf(fmaxf(fabsf(fa.x), fabsf(fa.y)), fmaxf(fabsf(fb.x), fabsf(fb.y))));
                    out[q] = fma2(a, pk(cs.x, cs.y), mul2(mul2(b, sg), pk(sn.x, sn.y)));
                }
            }
        };
        if (w.page < 0) {                                 // (the warp agrees on it)
            if (inside && t + A.side < n) fetch(t + A.side);
            continue;
        }
        if (inside) {
            turn(r0, y0, mode0, c, x);
            turn(r1, y1, mode1, c + 8, x + 4);
            if (t + A.side < n) fetch(t + A.side);
        } else {
#pragma unroll
            for (int q = 0; q < 8; ++q) x[q] = 0;
        }
        char *pl = dst + w.at;
        const int r16 = w.pos & (kStrip - 1);
        if constexpr (!I4) {
            if (inside) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t o[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float2 v = up(x[4 * h + q]);
                        const __nv_bfloat162 b = __floats2bfloat162_rn(v.x, v.y);
                        o[q] = *reinterpret_cast<const uint32_t *>(&b);
                    }
                    *reinterpret_cast<uint4 *>(pl + r16 * 128 + (((2 * lane4 + h) ^ (r16 & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
        } else {
            float2 v = up(x[0]);
            float lo = v.x, hi = v.x;
            lo = min3(lo, v.y, v.y);
            hi = max3(hi, v.y, v.y);
#pragma unroll
            for (int q = 1; q < 8; ++q) {
                v = up(x[q]);
                lo = min3(lo, v.x, v.y);
                hi = max3(hi, v.x, v.y);
            }
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                const float a = __shfl_xor_sync(0xffffffffu, lo, o), b = __shfl_xor_sync(0xffffffffu, hi, o);
                lo = min3(lo, a, a);
                hi = max3(hi, b, b);
            }
            float err = 0.f;                              // of a channel's value
            if (any_turned) {
                mag = fmaxf(mag, __shfl_xor_sync(0xffffffffu, mag, 1));
                mag = fmaxf(mag, __shfl_xor_sync(0xffffffffu, mag, 2));
                err = turned ? fabsf(A.r.mscale) * mag * (A.r.mscale == 1.f ? kSlackPlain : kSlack) : 0.f;
            }
            const float m = half_sat(lo), range = fmaxf(hi - m, 0.f);
            const float sraw = range * (1.f / 15.f), s = half_sat(sraw);
            // what FP32 leaves open: the minimum, and the scale (its own roundings are within 2^-22 of it)
            const bool open_scale = half_unsure(sraw, s, fmaf(sraw, 2.4e-7f, err * 0.14f)) || (err > 0.f && half_unsure(lo, m, err));
            float inv;
            asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
            const float nm = -m * inv;
            const bool normal = s >= 6.2e-5f && s < 65504.f && fmaf(lo, inv, nm) >= -0.45f;
            // whole numbers next to t = x / s - m / s, and the largest distance to them
            constexpr float kMagic = 12582912.f;          // 1.5 * 2^23: adding it rounds to a whole number
            const F2 inv2 = pk(inv, inv), nm2 = pk(nm, nm), magic = pk(kMagic, kMagic), unmagic = pk(-kMagic, -kMagic);
            const F2 minus = pk(-1.f, -1.f);
            float away = 0.f;
            F2 cd[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const F2 tt = fma2(x[q], inv2, nm2);
                cd[q] = add2(add2(tt, magic), unmagic);
                const float2 r = up(fma2(cd[q], minus, tt));
                away = fmaxf(away, fmaxf(fabsf(r.x), fabsf(r.y)));
            }
            // t's own error, t below 15.1: 2^-23 of t from inv, 2^-24 of t from the fma, 2^-24 of m / s from nm
            const float window = fmaf(fabsf(nm), 1.2e-7f, 3e-6f) + err * inv;
            // (a group with a NaN, an infinity or a rotation that FP32 overflows has no normal scale, or a window too wide)
            const bool plain = normal && !open_scale && away < 0.5f - window;
            uint2 word;
            {   // four codes to 16 bits: sums of whole numbers below 2^16
                float h[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float2 u = up(fma2(cd[2 * q + 1], pk(256.f, 256.f), cd[2 * q]));
                    h[q] = fmaf(u.y, 16.f, u.x) + 8388608.f;
                }
                word.x = __byte_perm(__float_as_uint(h[0]), __float_as_uint(h[1]), 0x5410);
                word.y = __byte_perm(__float_as_uint(h[2]), __float_as_uint(h[3]), 0x5410);
            }
            __half2 pr = __halves2half2(__float2half_rn(s), __float2half_rn(m));
            const unsigned gmask = 0xfu << (threadIdx.x & 28);
            const unsigned rest = __ballot_sync(0xffffffffu, inside && !plain);
            unsigned open = 0;
            if (rest) {
                // wild: the rotation may have overflowed FP32 (or met an infinity: the path in double tells); bad: a NaN or an infinity
                const bool wild = turned && !(fabsf(A.r.mscale) * mag <= 8e37f);
                const bool bad = !wild && !(fabsf(lo) < INFINITY && fabsf(hi) < INFINITY);
                if ((rest & gmask) && !wild) {
                    if (bad) {
                        word = make_uint2(0, 0);
                        pr = __halves2half2(__ushort_as_half(0x7e00), __ushort_as_half(0x7e00));
                    } else if (err == 0.f && !open_scale && normal && fabsf(nm) < 1e6f) {
                        // ties, mostly: only the channels next to a border are looked at again (t is off by less than 1/8, so a code is the
                        // whole number next to it or the one on the other side of the border)
#pragma unroll
                        for (int q = 0; q < 16; ++q) {
                            const float2 xv = up(x[q / 2]), cv = up(cd[q / 2]);
                            const float xq = q & 1 ? xv.y : xv.x, c = q & 1 ? cv.y : cv.x, r = fmaf(xq, inv, nm) - c;
                            if (fabsf(r) < 0.5f - window) continue;
                            const float f = r > 0.f ? c : c - 1.f, d = xq - m;
                            const float back = xq - d, lost = (xq - (d + back)) + (back - m);   // x - m = d + lost, exactly
                            const float diff = (d - (f + 0.5f) * s) + lost;
                            const int more = (f < c ? -1 : 0) + (diff > 0.f || (diff == 0.f && ((int)f & 1)) ? 1 : 0);
                            (q < 8 ? word.x : word.y) += (unsigned)more << (4 * (q & 7));
                        }
                    } else if (err == 0.f && !open_scale) {
                        // codes that need a clamp, or a minimum of so many steps that t has lost its fraction: x - m first, which has not
                        word = make_uint2(0, 0);
                        const float iv = s > 0.f ? 1.f / s : 0.f;
#pragma unroll
                        for (int q = 0; q < 16; ++q) {
                            const float2 xv = up(x[q / 2]);
                            const float xq = q & 1 ? xv.y : xv.x, d = xq - m;
                            const float f = fminf(fmaxf(floorf(d * iv), 0.f), 14.f);
                            const float half = (f + 0.5f) * s;    // exact: 5 bits times 11
                            float diff = d - half;                // its sign decides f or f + 1
                            if (fabsf(diff) <= 1e-6f * fabsf(half)) {
                                const float back = xq - d, lost = (xq - (d + back)) + (back - m);   // x - m = d + lost, exactly
                                diff += lost;
                            }
                            const bool more = diff > 0.f || (diff == 0.f && ((int)f & 1));
                            const unsigned code = s > 0.f ? (unsigned)f + (more ? 1u : 0u) : 0u;
                            if (q < 8) word.x |= code << (4 * q);
                            else word.y |= code << (4 * (q - 8));
                        }
                    }
                }
                open = __ballot_sync(0xffffffffu, inside && (rest & gmask) && (wild || (!bad && !(err == 0.f && !open_scale))));
            }
            if (inside && !(open & gmask)) {
                reinterpret_cast<uint2 *>(pl)[r16 * 4 + lane4] = word;
                if (lane4 == 0) reinterpret_cast<__half2 *>(pl + 512)[r16] = pr;
            }
            for (unsigned left = open; left;) {
                const int at = __ffs(left) - 1;
                left &= ~(0xfu << (at & 28));
                const int ohead = __shfl_sync(0xffffffffu, head, at), oplane = __shfl_sync(0xffffffffu, plane, at);
                const bool okey = oplane < kplanes;
                const View &os = okey ? A.k : A.v;
                group_in_double<T>(reinterpret_cast<const T *>(os.p) + (int64_t)(t0 + t) * os.ts + (int64_t)ohead * os.hs,
                                   64 * (okey ? oplane : oplane - kplanes), A.r, okey, w.pos,
                                   P.pool + w.at + (int64_t)ohead * P.block_bytes + oplane * kPlaneI4, r16);
            }
        }
    }
}

// ---- read ------------------------------------------------------------------------------------------

template <typename T, bool VEC> __device__ __forceinline__ void store8(T *p, const F2 (&x)[4]) {
    if constexpr (sizeof(T) == 2) {
        uint32_t o[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float2 v = up(x[q]);
            const __nv_bfloat162 b = __floats2bfloat162_rn(v.x, v.y);
            o[q] = *reinterpret_cast<const uint32_t *>(&b);
        }
        if constexpr (VEC) *reinterpret_cast<uint4 *>(p) = make_uint4(o[0], o[1], o[2], o[3]);
        else
#pragma unroll
            for (int q = 0; q < 8; ++q) reinterpret_cast<uint16_t *>(p)[q] = (uint16_t)(o[q / 2] >> (16 * (q & 1)));
    } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float2 v = up(x[q]);
            if constexpr (VEC) {
                if (q & 1) continue;
                const float2 u = up(x[q + 1]);
                *reinterpret_cast<float4 *>(p + 2 * q) = make_float4(v.x, v.y, u.x, u.y);
            } else {
                p[2 * q] = v.x;
                p[2 * q + 1] = v.y;
            }
        }
    }
}

template <typename T, bool VEC, bool I4>
__global__ void __launch_bounds__(kThreads) read_kernel(const __grid_constant__ AppendArgs A) {
    __shared__ Place place[kTokens];
    const Paged &P = A.P;
    const int part = (int)(blockIdx.x % A.parts);
    const int t0 = (int)(blockIdx.x / A.parts) * A.tokens, n = min(A.tokens, A.T - t0);
    find_places(P, A.cu, A.T, t0, n, place);
    __syncthreads();
    const int kplanes = P.dqk / 64, lane4 = threadIdx.x & 3;
    const int row_set = (int)(threadIdx.x >> 5) / A.warps, mine = ((int)(threadIdx.x >> 5) - row_set * A.warps) * 8 + (int)(threadIdx.x & 31) / 4;
    const int gi = part * A.groups + mine;
    if (mine >= A.groups || gi >= P.heads * P.planes || row_set >= n) return;
    // plane-fastest here: neighbouring lanes write neighbouring channels
    const int head = gi / P.planes, plane = gi - head * P.planes;
    const bool key = plane < kplanes;
    const View &dst = key ? A.k : A.v;
    if (!dst.p) return;
    T *row = reinterpret_cast<T *>(dst.p) + (int64_t)t0 * dst.ts + (int64_t)head * dst.hs + 64 * (key ? plane : plane - kplanes) + 16 * lane4;
    const char *src = P.pool + (int64_t)head * P.block_bytes + plane * (I4 ? kPlaneI4 : kPlaneBf16);
    struct Held { uint4 a, b; uint32_t pr; };
    auto fetch = [&](int t, Held &h) {
        const Place w = place[t];
        if (w.page < 0) return;
        const char *pl = src + w.at;
        const int r16 = w.pos & (kStrip - 1);
        if constexpr (I4) {
            const uint2 v = reinterpret_cast<const uint2 *>(pl)[r16 * 4 + lane4];
            h.a.x = v.x;
            h.a.y = v.y;
            h.pr = reinterpret_cast<const uint32_t *>(pl + 512)[r16];
        } else {
            h.a = *reinterpret_cast<const uint4 *>(pl + r16 * 128 + (((2 * lane4) ^ (r16 & 7)) << 4));
            h.b = *reinterpret_cast<const uint4 *>(pl + r16 * 128 + (((2 * lane4 + 1) ^ (r16 & 7)) << 4));
        }
    };
    Held now, next;
    fetch(row_set, now);
#pragma unroll 1
    for (int t = row_set; t < n; t += A.side) {
        if (t + A.side < n) fetch(t + A.side, next);
        F2 x[2][4];
        if (place[t].page < 0) {
#pragma unroll
            for (int q = 0; q < 8; ++q) x[q / 4][q % 4] = pk(__int_as_float(0x7fc00000), __int_as_float(0x7fc00000));
        } else if constexpr (I4) {
            const float2 pr = __half22float2(*reinterpret_cast<const __half2 *>(&now.pr));
            const F2 s = pk(pr.x, pr.x), m = pk(pr.y, pr.y), off = pk(-8388608.f, -8388608.f);
            // s code is exact (15 bits), so the value is rounded once, then to the output's type
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const uint32_t w = (q < 4 ? now.a.x : now.a.y) >> (8 * (q & 3));
                const F2 c = pk(__uint_as_float((w & 15u) | 0x4B000000u), __uint_as_float(((w >> 4) & 15u) | 0x4B000000u));   // 2^23 + code
                x[q / 4][q % 4] = fma2(add2(c, off), s, m);
            }
        } else {
            const uint32_t u[8] = {now.a.x, now.a.y, now.a.z, now.a.w, now.b.x, now.b.y, now.b.z, now.b.w};
#pragma unroll
            for (int q = 0; q < 8; ++q) x[q / 4][q % 4] = pk(__uint_as_float(u[q] << 16), __uint_as_float(u[q] & 0xffff0000u));
        }
        T *p = row + (int64_t)t * dst.ts;
        store8<T, VEC>(p, x[0]);
        store8<T, VEC>(p + 8, x[1]);
        now = next;
    }
}

// A CTA's groups (an equal share of heads * planes), its warps and tokens.  A lane goes through as many tokens (up to
// kDepth) as leave about 16 CTAs for each of the GPU's 152 SMs (three are resident; with 8, appending and reading 9,366 tokens
// of 8 heads of 192 + 128 channels, bf16 pages, took 56 us instead of 49);
// the search for their places, their angles and a lane's addresses are shared by them.  With few groups several tokens lie side by side.
void plan(AppendArgs &A, unsigned &grid, unsigned &threads, size_t &table) {
    const int all = A.P.heads * A.P.planes;
    A.parts = (all + kGroups - 1) / kGroups;
    A.groups = (all + A.parts - 1) / A.parts;
    A.warps = (A.groups + 7) / 8;
    A.side = kThreads / 32 / A.warps;
    const size_t row = 2 * (size_t)((A.r.half + 3) & ~3) * sizeof(float);
    long long depth = (long long)A.T * A.parts / ((long long)A.side * 152 * 16);
    depth = depth < 1 ? 1 : depth > kDepth ? kDepth : depth;
    while (depth > 1 && (depth * A.side > kTokens || depth * A.side * row > 32768)) --depth;
    A.tokens = (int)depth * A.side;
    table = A.tokens * row;
    threads = (unsigned)(A.warps * A.side * 32);
    grid = (unsigned)(((long long)A.T + A.tokens - 1) / A.tokens * A.parts);
}

}  // namespace

cudaError_t launch_paged_append(const k3mla_paged_cache *c, const k3mla_view *k, const k3mla_view *v, int bf16, const int32_t *cu,
                                int T, const k3mla_rope_args *rope, cudaStream_t s) {
    AppendArgs A;
    A.P = make_paged(c);
    A.k = make_view(k);
    A.v = make_view(v);
    A.cu = cu;
    A.T = T;
    A.r = make_rope(rope);
    unsigned grid, threads;
    size_t table;
    plan(A, grid, threads, table);
    const int size = bf16 ? 2 : 4;
    const bool vec = view_vec(k, size, T, c->heads) && view_vec(v, size, T, c->heads), i4 = c->format == K3MLA_CACHE_I4;
    void (*fn)(const AppendArgs);
    if (bf16) fn = vec ? (i4 ? append_kernel<__nv_bfloat16, true, true> : append_kernel<__nv_bfloat16, true, false>)
                       : (i4 ? append_kernel<__nv_bfloat16, false, true> : append_kernel<__nv_bfloat16, false, false>);
    else fn = vec ? (i4 ? append_kernel<float, true, true> : append_kernel<float, true, false>)
                  : (i4 ? append_kernel<float, false, true> : append_kernel<float, false, false>);
    fn<<<grid, threads, table, s>>>(A);
    count_launch();
    return cudaGetLastError();
}

cudaError_t launch_paged_read(const k3mla_paged_cache *c, const k3mla_view *k, const k3mla_view *v, int bf16, const int32_t *cu,
                              int T, cudaStream_t s) {
    AppendArgs A;
    A.P = make_paged(c);
    A.k = make_view(k);
    A.v = make_view(v);
    A.cu = cu;
    A.T = T;
    A.r = make_rope(nullptr);
    unsigned grid, threads;
    size_t table;
    plan(A, grid, threads, table);
    const int size = bf16 ? 2 : 4;
    const bool vec = (!k || view_vec(k, size, T, c->heads)) && (!v || view_vec(v, size, T, c->heads)), i4 = c->format == K3MLA_CACHE_I4;
    void (*fn)(const AppendArgs);
    if (bf16) fn = vec ? (i4 ? read_kernel<__nv_bfloat16, true, true> : read_kernel<__nv_bfloat16, true, false>)
                       : (i4 ? read_kernel<__nv_bfloat16, false, true> : read_kernel<__nv_bfloat16, false, false>);
    else fn = vec ? (i4 ? read_kernel<float, true, true> : read_kernel<float, true, false>)
                  : (i4 ? read_kernel<float, false, true> : read_kernel<float, false, false>);
    fn<<<grid, threads, 0, s>>>(A);
    count_launch();
    return cudaGetLastError();
}

}  // namespace k3kda
