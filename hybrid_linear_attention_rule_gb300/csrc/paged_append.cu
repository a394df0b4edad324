// paged_append.cu -- new key and value rows into the paged cache (keys rotated on the way), and rows
// back out of it as values, on sm_103a.
//
// Both move every element once and are bound by HBM.  A unit is 8 channels of one (token, head): one
// 16-byte piece (bf16 in) or two (fp32 in); the 8 lanes of a group hold one plane's 64 channels of a token, whose
// minimum and maximum three shuffles find.  A CTA takes kTokens tokens (fewer when there are
// few), finds their sequence, position and page once (a 32-way search of cu_seqlens, one warp a
// token) and forms their cosines and sines once for all heads.
//
// 4-bit rounding.  The stored values are those of the definition in exact arithmetic, so that what
// the cache holds does not hang on how FP32 rounds:
//   - A group of channels that are not turned is exact in FP32: m = fp16(min) is one rounding, and a
//     code is decided by the sign of (x - m) - (c + 1/2) s, where (c + 1/2) s has at most 16 bits: one
//     fma and, only next to a tie, the rounding error of x - m.
//   - A group that holds turned channels carries FP32 errors of up to kSlack of its largest
//     magnitude.  Where m, s or a code lies that close to a rounding border (about one group in
//     1000, by the borders' spacing) the group goes to the warp, which repeats it in double, two channels a
//     lane, with the angle's sine and cosine in double.  The same path settles a scale next to a border.
#include <math.h>

#include "paged.cuh"

namespace k3kda {
namespace {

constexpr int kThreads = 256;
constexpr int kUnits = 4;                 // units a thread has in flight
constexpr int kTokens = 16;               // most tokens of a CTA
// bound on the FP32 error of a turned channel, relative to the largest |x| + |y| of the group's pairs: three
// roundings of the rotation and the error of the cosine and sine, 2^-22 in all, doubled
constexpr float kSlack = 4.8e-7f;

struct AppendArgs {
    Paged P;
    View k, v;
    const int32_t *cu;
    int T;
    Rope r;
    int tokens;                           // tokens of a CTA
    int parts;                            // CTAs that share the same tokens
    int units;                            // units per token: heads * planes * 8
};

struct Place {                            // where a CTA's token goes; page < 0: nowhere
    int n, pos, page;
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
    for (int i = threadIdx.x >> 5; i < count; i += kThreads / 32) {
        const int t = t0 + i;
        const int n = cu ? find_seq(cu, P.N, t, lane) : t;
        if (lane == 0) {
            Place w{n, -1, -1};
            int b = t, e = t + 1;
            if (cu) seq_bounds(cu, n, T, b, e);
            const int len = paged_len(P, n);
            const int64_t pos = (int64_t)len - e + t;
            if (len >= 0 && t >= b && t < e && pos >= 0) {
                w.pos = (int)pos;
                w.page = paged_page(P, n, w.pos);
            }
            place[i] = w;
        }
    }
}

__device__ __forceinline__ char *plane_at(const Paged &P, const Place &w, int head, int plane, int plane_bytes) {
    const int in_page = w.pos % P.page_size;
    return P.pool + (int64_t)w.page * P.page_bytes + (int64_t)head * P.block_bytes +
           (int64_t)(in_page / kStrip) * P.strip_bytes + plane * plane_bytes;
}

template <typename T, bool VEC> __device__ __forceinline__ void load8(const T *p, float (&x)[8]) {
    if constexpr (VEC && sizeof(T) == 2) {
        const uint4 w = *reinterpret_cast<const uint4 *>(p);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = __uint_as_float((e & 1) ? (u[e / 2] & 0xffff0000u) : (u[e / 2] << 16));
    } else if constexpr (VEC) {
        const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = load_elt(p, e, sizeof(T) == 2);
    }
}

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

// Whether the fp16 rounding of some value within d of x may differ from that of x.
__device__ __forceinline__ bool half_unsure(float x, float d) { return half_sat(x - d) != half_sat(x + d); }

// A group in double by the whole warp: lane l takes channels 2l and 2l + 1 of the plane.  src: the (token, head) row's
// key or value; c0: the plane's first channel in it.
template <typename T> __device__ __noinline__ void group_in_double(const T *src, int c0, const Rope r, bool key, int pos, char *plane, int row) {
    const int lane = threadIdx.x & 31;
    double x[2];
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
    }
    double lo = fmin(x[0], x[1]), hi = fmax(x[0], x[1]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        lo = fmin(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = fmax(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    const double m = half_sat(lo), s = half_sat(fmax(hi - m, 0.0) / 15.0);
    unsigned byte = 0;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const double c = s > 0.0 ? fmin(fmax(rint((x[e] - m) / s), 0.0), 15.0) : 0.0;
        byte |= (unsigned)c << (4 * e);
    }
    reinterpret_cast<uint8_t *>(plane)[row * 32 + lane] = (uint8_t)byte;
    if (lane == 0) reinterpret_cast<__half2 *>(plane + 512)[row] = __halves2half2(__double2half(s), __double2half(m));
}

template <typename T, bool VEC, bool I4>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ AppendArgs A) {
    extern __shared__ float2 cs[];                        // [tokens][dim/2]
    __shared__ Place place[kTokens];
    const Paged &P = A.P;
    const int part = (int)(blockIdx.x % A.parts);
    const int t0 = (int)(blockIdx.x / A.parts) * A.tokens, n = min(A.tokens, A.T - t0);
    find_places(P, A.cu, A.T, t0, n, place);
    __syncthreads();
    for (int i = threadIdx.x; i < n * A.r.half; i += kThreads) {
        const int t = i / A.r.half;
        const float2 v = rope_cs(A.r.phase[i - t * A.r.half], place[t].pos);
        cs[i] = make_float2(v.x * A.r.mscale, v.y * A.r.mscale);
    }
    __syncthreads();
    const int kplanes = P.dqk / 64, total = n * A.units;
    // every lane of a warp runs every round: a group that needs the double path gets the whole warp
    for (int base = part * kThreads; base < total; base += A.parts * kThreads) {
        const int i = base + threadIdx.x;
        const bool inside = i < total;
        const int t = inside ? i / A.units : 0;
        const int e = inside ? i - t * A.units : 0;
        const int g = e & 7, hp = e >> 3, head = hp / P.planes, plane = hp - head * P.planes;
        const bool key = plane < kplanes;
        const Place w = place[t];
        const bool live = inside && w.page >= 0;
        const int c0 = key ? plane * 64 : (plane - kplanes) * 64;
        const View &src = key ? A.k : A.v;
        const T *row = reinterpret_cast<const T *>(src.p) + (int64_t)(t0 + t) * src.ts + (int64_t)head * src.hs;
        float x[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) x[q] = 0.f;
        bool turned = false;                              // some channel of the group is
        float mag = 0.f;                                  // largest |x| + |y| of the pairs
        const int c = c0 + 8 * g, rend = A.r.off + A.r.dim;
        if (live) {
            load8<T, VEC>(row + c, x);
            if (key && A.r.dim > 0) {
                turned = c0 < rend && c0 + 64 > A.r.off;
                if (c < rend && c + 8 > A.r.off) {
                    const float2 *tab = cs + t * A.r.half;
                    // runs of 8 channels that turn together with 8 partners; else channel by channel
                    const bool whole = VEC && c >= A.r.off && c + 8 <= rend && (A.r.inter ? ((c - A.r.off) & 1) == 0 : (A.r.half & 7) == 0 && ((c - A.r.off) & 7) == 0);
                    if (whole && A.r.inter) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const float2 a = tab[(c - A.r.off) / 2 + q];
                            mag = fmaxf(mag, fabsf(x[2 * q]) + fabsf(x[2 * q + 1]));
                            const float u = x[2 * q] * a.x - x[2 * q + 1] * a.y, v = x[2 * q + 1] * a.x + x[2 * q] * a.y;
                            x[2 * q] = u;
                            x[2 * q + 1] = v;
                        }
                    } else if (whole) {
                        const bool second = c - A.r.off >= A.r.half;
                        const int pair = c - A.r.off - (second ? A.r.half : 0);
                        float y[8];
                        load8<T, VEC>(row + (second ? c - A.r.half : c + A.r.half), y);
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            const float2 a = tab[pair + q];
                            mag = fmaxf(mag, fabsf(x[q]) + fabsf(y[q]));
                            x[q] = second ? x[q] * a.x + y[q] * a.y : x[q] * a.x - y[q] * a.y;
                        }
                    } else {
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            if (c + q < A.r.off || c + q >= rend) continue;
                            const Turn tn = turn_of(A.r, c + q);
                            const float2 a = tab[tn.pair];
                            const float y = load_elt(row, tn.partner, sizeof(T) == 2);
                            // its own value again: a neighbour's turn must not read what this loop wrote
                            const float z = load_elt(row, c + q, sizeof(T) == 2);
                            mag = fmaxf(mag, fabsf(z) + fabsf(y));
                            x[q] = tn.second ? z * a.x + y * a.y : z * a.x - y * a.y;
                        }
                    }
                }
            }
        }
        const int r16 = w.pos & (kStrip - 1);
        if constexpr (!I4) {
            if (live) {
                uint32_t o[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * q], x[2 * q + 1]);
                    o[q] = *reinterpret_cast<const uint32_t *>(&b);
                }
                *reinterpret_cast<uint4 *>(plane_at(P, w, head, plane, kPlaneBf16) + r16 * 128 + ((g ^ (r16 & 7)) << 4)) =
                    make_uint4(o[0], o[1], o[2], o[3]);
            }
        } else {
            float lo = x[0], hi = x[0], sum = 0.f;        // sum: NaN when the group has a NaN or an infinity
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                lo = fminf(lo, x[q]);
                hi = fmaxf(hi, x[q]);
                sum = fmaf(x[q], 0.f, sum);
            }
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) {
                lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
                hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
                sum += __shfl_xor_sync(0xffffffffu, sum, o);
                mag = fmaxf(mag, __shfl_xor_sync(0xffffffffu, mag, o));
            }
            const float err = turned ? fabsf(A.r.mscale) * mag * kSlack : 0.f;    // of a channel's value
            const bool bad = !(sum == 0.f);
            const float m = half_sat(lo), range = fmaxf(hi - m, 0.f);
            const float sraw = range / 15.f, s = half_sat(sraw);
            // what FP32 leaves open: the minimum, the scale (its own roundings are within 2^-23 of it) and, for
            // turned channels, the codes
            bool unsure = err > 0.f && half_unsure(lo, err);
            unsure = unsure || half_unsure(sraw, fmaf(sraw, 2.4e-7f, err * 0.14f));
            const float inv = s > 0.f ? 1.f / s : 0.f;
            const float slack = err * inv;
            unsigned word = 0;
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const float d = x[q] - m;
                const float f = fminf(fmaxf(floorf(d * inv), 0.f), 14.f);
                const float half = (f + 0.5f) * s;        // exact: 5 bits times 11
                float diff = fmaf(-1.f, half, d);         // sign decides f or f + 1
                if (err > 0.f) {
                    unsure = unsure || fabsf(diff) * inv <= slack + 1.5e-7f * (f + 1.f);
                } else if (fabsf(diff) <= 1e-6f * fabsf(half)) {
                    const float back = x[q] - d, lost = (x[q] - (d + back)) + (back - m);   // x - m = d + lost, exactly
                    diff += lost;
                }
                const bool up = diff > 0.f || (diff == 0.f && ((int)f & 1));
                word |= (s > 0.f ? (unsigned)f + (up ? 1u : 0u) : 0u) << (4 * q);
            }
            const unsigned open = __ballot_sync(0xffffffffu, unsure && !bad && live);
            if (live) {
                char *pl = plane_at(P, w, head, plane, kPlaneI4);
                const unsigned mine = (open >> (threadIdx.x & 24)) & 0xffu;
                if (!mine) {
                    reinterpret_cast<uint32_t *>(pl)[r16 * 8 + g] = bad ? 0u : word;
                    if (g == 0) {
                        const __half2 pr = bad ? __halves2half2(__ushort_as_half(0x7e00), __ushort_as_half(0x7e00))
                                               : __halves2half2(__float2half_rn(s), __float2half_rn(m));
                        reinterpret_cast<__half2 *>(pl + 512)[r16] = pr;
                    }
                }
            }
            for (int q = 0; q < 32; q += 8) {
                if (!((open >> q) & 0xffu)) continue;
                const int ot = __shfl_sync(0xffffffffu, t, q), ohead = __shfl_sync(0xffffffffu, head, q),
                          oplane = __shfl_sync(0xffffffffu, plane, q);
                const bool okey = oplane < kplanes;
                const Place ow = place[ot];
                const View &os = okey ? A.k : A.v;
                group_in_double<T>(reinterpret_cast<const T *>(os.p) + (int64_t)(t0 + ot) * os.ts + (int64_t)ohead * os.hs,
                                   (okey ? oplane : oplane - kplanes) * 64, A.r, okey, ow.pos,
                                   plane_at(P, ow, ohead, oplane, kPlaneI4), ow.pos & (kStrip - 1));
            }
        }
    }
}

// ---- read ------------------------------------------------------------------------------------------

template <typename T, bool VEC> __device__ __forceinline__ void store8(T *p, const float (&x)[8]) {
    if constexpr (VEC && sizeof(T) == 2) {
        uint32_t o[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * q], x[2 * q + 1]);
            o[q] = *reinterpret_cast<const uint32_t *>(&b);
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(o[0], o[1], o[2], o[3]);
    } else if constexpr (VEC) {
        *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<float4 *>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) store_elt(p, e, x[e], sizeof(T) == 2);
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
    const int kplanes = P.dqk / 64, total = n * A.units;
    for (int i = part * kThreads + threadIdx.x; i < total; i += A.parts * kThreads) {
        const int t = i / A.units, e = i - t * A.units;
        const int g = e & 7, hp = e >> 3, head = hp / P.planes, plane = hp - head * P.planes;
        const bool key = plane < kplanes;
        const View &dst = key ? A.k : A.v;
        if (!dst.p) continue;
        const Place w = place[t];
        float x[8];
        if (w.page < 0) {
#pragma unroll
            for (int q = 0; q < 8; ++q) x[q] = __int_as_float(0x7fc00000);
        } else if (I4) {
            const char *pl = plane_at(P, w, head, plane, kPlaneI4);
            const int r16 = w.pos & (kStrip - 1);
            const uint32_t word = reinterpret_cast<const uint32_t *>(pl)[r16 * 8 + g];
            const float2 pr = __half22float2(reinterpret_cast<const __half2 *>(pl + 512)[r16]);
            // s code is exact (15 bits), so the value is rounded once, then to the output's type
#pragma unroll
            for (int q = 0; q < 8; ++q) x[q] = fmaf((float)((word >> (4 * q)) & 15u), pr.x, pr.y);
        } else {
            const int r16 = w.pos & (kStrip - 1);
            load8<__nv_bfloat16, true>(reinterpret_cast<const __nv_bfloat16 *>(plane_at(P, w, head, plane, kPlaneBf16) + r16 * 128 +
                                                                               ((g ^ (r16 & 7)) << 4)), x);
        }
        const int c = (key ? plane * 64 : (plane - kplanes) * 64) + 8 * g;
        store8<T, VEC>(reinterpret_cast<T *>(dst.p) + (int64_t)(t0 + t) * dst.ts + (int64_t)head * dst.hs + c, x);
    }
}

// Tokens of a CTA and CTAs of a token: about kUnits units a thread, more tokens to a CTA (up to
// kTokens) once all SMs have several CTAs, so that the places' search is shared.
void plan(AppendArgs &A, unsigned &grid) {
    A.units = A.P.heads * A.P.planes * 8;
    const long long total = (long long)A.T * A.units, full = (long long)kThreads * kUnits;
    const long long want = total / (full * 152 * 4);              // four CTAs of work for each SM
    int tokens = (int)(full / A.units > 1 ? full / A.units : 1);
    if (want > 1) tokens = (int)(tokens * (want > kTokens ? kTokens : want));
    A.tokens = tokens > kTokens ? kTokens : tokens;
    const long long per = (long long)A.tokens * A.units;
    A.parts = per > full * 4 ? (int)((per + full * 4 - 1) / (full * 4)) : 1;
    if (total < full * 152) A.parts = (int)((per + kThreads - 1) / kThreads);   // few rows: a unit a thread
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
    unsigned grid;
    plan(A, grid);
    const int size = bf16 ? 2 : 4;
    const bool vec = view_vec(k, size, T, c->heads) && view_vec(v, size, T, c->heads), i4 = c->format == K3MLA_CACHE_I4;
    void (*fn)(const AppendArgs);
    if (bf16) fn = vec ? (i4 ? append_kernel<__nv_bfloat16, true, true> : append_kernel<__nv_bfloat16, true, false>)
                       : (i4 ? append_kernel<__nv_bfloat16, false, true> : append_kernel<__nv_bfloat16, false, false>);
    else fn = vec ? (i4 ? append_kernel<float, true, true> : append_kernel<float, true, false>)
                  : (i4 ? append_kernel<float, false, true> : append_kernel<float, false, false>);
    fn<<<grid, kThreads, (size_t)A.tokens * A.r.half * sizeof(float2), s>>>(A);
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
    unsigned grid;
    plan(A, grid);
    const int size = bf16 ? 2 : 4;
    const bool vec = (!k || view_vec(k, size, T, c->heads)) && (!v || view_vec(v, size, T, c->heads)), i4 = c->format == K3MLA_CACHE_I4;
    void (*fn)(const AppendArgs);
    if (bf16) fn = vec ? (i4 ? read_kernel<__nv_bfloat16, true, true> : read_kernel<__nv_bfloat16, true, false>)
                       : (i4 ? read_kernel<__nv_bfloat16, false, true> : read_kernel<__nv_bfloat16, false, false>);
    else fn = vec ? (i4 ? read_kernel<float, true, true> : read_kernel<float, true, false>)
                  : (i4 ? read_kernel<float, false, true> : read_kernel<float, false, false>);
    fn<<<grid, kThreads, 0, s>>>(A);
    count_launch();
    return cudaGetLastError();
}

}  // namespace k3kda
