// block_norm.cuh -- the norms around a block with its gate and residual, and their gradients (block_norm_bf16.cu and
// block_norm_f32.cu hold the kernels of one element type each).
//
//     u = x r_x post,  r_x = rsqrt(mean x^2 + eps)      (u = x without post)
//     s = residual + alpha u act(gate)
//     y = s r_s pre,   r_s = rsqrt(mean s^2 + eps)
// Backwards, with ds the gradient of s from the residual stream and dy that of y:
//     d = ds + r_s (dy pre - h_s mean(dy pre h_s)),  h_s = s r_s            dresidual = d,  dpre = sum over rows dy h_s
//     dgate = alpha d u act'(gate),  du = alpha d act(gate)
//     dx = r_x (du post - h_x mean(du post h_x)),  h_x = x r_x              dpost = sum over rows du h_x
// Every array is read once and written once: a row is held in registers by its threads, up to 16 elements each.  HBM bounds the forward pass, issue as much
// as HBM the gradient; both work on all 16, so widths that fill them are the fastest.  Rows
// of up to 128 channels take 8 threads, of up to 16384 a CTA of 1024; arrays move in 16-byte pieces where the width and the
// addresses allow it, else element by element.  The gradient's rows are copied to shared memory two rounds ahead.  All arithmetic is FP32, each output is rounded once; y comes from the sum
// before its rounding.
//
// 16,384 rows of 4,096 in BF16, all parts: 114 us, 88 % of a plain copy's rate; 131,072 rows of 128 with a gate 22.5 us, 67 %.  Gradients of 8,192
// rows of 4,096: 123 us, 65 %, the issue slots half used; of 2,777 rows of 1,111 in FP32, whose rows begin off 16 bytes, 41 us, 36 %.
#pragma once

#include "common.cuh"
#include "tc_ptx.cuh"

namespace k3kda {
namespace blk {

constexpr int MOST_E = 16;             // elements of a row that one thread holds, at most
constexpr int MOST_D = 1024 * MOST_E;
constexpr int MOST_PARTS = 304;        // CTAs of the gradient: two an SM, each a partial sum of the weights' gradients

struct Args {
    const void *x, *gate, *residual;   // forward: in
    const void *s_in, *ds, *dy;        // gradient: in
    const float *post, *pre;
    void *s, *y;                       // forward: out
    void *dx, *dgate, *dresidual;      // gradient: out
    float *dpost, *dpre, *parts;       // parts [2][CTAs][D]
    long long rows;
    int D, silu;
    float alpha, eps;
};

inline int threads_a_row(int D) {
    const int need = (D + MOST_E - 1) / MOST_E;
    return need <= 8 ? 8 : need <= 32 ? 32 : need <= 128 ? 128 : need <= 256 ? 256 : need <= 512 ? 512 : 1024;
}
inline long long groups_of(int tpr) { return tpr < 256 ? 256 / tpr : 1; }
inline int parts_of(long long rows, int D) {
    const long long g = groups_of(threads_a_row(D)), need = (rows + g - 1) / g;
    return (int)(need < MOST_PARTS ? need : MOST_PARTS);
}

template <class T> constexpr int kVec = 16 / (int)sizeof(T);

template <class T> __device__ __forceinline__ float exp_of(float x) { return sizeof(T) == 2 ? __expf(x) : expf(x); }
template <class T> __device__ __forceinline__ float inverse(float x) { return sizeof(T) == 2 ? __fdividef(1.f, x) : 1.f / x; }
// sigmoid(z); where 1 + e^-z is too large for the fast division it gives 0, as it should
template <class T> __device__ __forceinline__ float sigmoid_of(float z) { return inverse<T>(1.f + exp_of<T>(-z)); }

// Thread t's elements of a row: pieces of VEC at (t + i TPR) VEC.
template <class T, int VEC, int TPR, int E> struct Slot {
    static constexpr int ITEMS = E / VEC, WORDS = VEC == 1 ? E : E * (int)sizeof(T) / 4;
    static __device__ __forceinline__ int column(int t, int e) { return (t + e / VEC * TPR) * VEC + e % VEC; }
    // As they lie in memory (BF16 pieces two to a word): half the registers until they are used.
    struct Raw { uint32_t w[WORDS]; };
    template <bool STREAM> static __device__ __forceinline__ void fetch(const T *row, int t, int D, Raw &r) {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int c = (t + i * TPR) * VEC;
            if constexpr (VEC == 1) {
                if constexpr (sizeof(T) == 2) r.w[i] = c < D ? (uint32_t)reinterpret_cast<const unsigned short *>(row)[c] << 16 : 0u;
                else r.w[i] = c < D ? reinterpret_cast<const uint32_t *>(row)[c] : 0u;
            } else {
                uint4 v = make_uint4(0, 0, 0, 0);
                if (c < D) v = STREAM ? __ldcs(reinterpret_cast<const uint4 *>(row + c)) : *reinterpret_cast<const uint4 *>(row + c);
                r.w[4 * i] = v.x;
                r.w[4 * i + 1] = v.y;
                r.w[4 * i + 2] = v.z;
                r.w[4 * i + 3] = v.w;
            }
        }
    }
    static __device__ __forceinline__ float value(const Raw &r, int e) {
        if constexpr (VEC == 1 || sizeof(T) == 4) return __uint_as_float(r.w[e]);
        else return __uint_as_float(e & 1 ? r.w[e / 2] & 0xffff0000u : r.w[e / 2] << 16);
    }
    static __device__ __forceinline__ void load(const void *p, long long at, int t, int D, Raw &r) { fetch<true>(static_cast<const T *>(p) + at, t, D, r); }
    static __device__ __forceinline__ void weights(const float *p, int t, int D, float (&v)[E]) {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int c = (t + i * TPR) * VEC;
            if constexpr (VEC == 1) {
                v[i] = c < D ? __ldg(p + c) : 0.f;
            } else {
#pragma unroll
                for (int u = 0; u < VEC / 4; ++u) {
                    const float4 w = c < D ? __ldg(reinterpret_cast<const float4 *>(p + c) + u) : make_float4(0.f, 0.f, 0.f, 0.f);
                    v[i * VEC + 4 * u] = w.x;
                    v[i * VEC + 4 * u + 1] = w.y;
                    v[i * VEC + 4 * u + 2] = w.z;
                    v[i * VEC + 4 * u + 3] = w.w;
                }
            }
        }
    }
    static __device__ __forceinline__ void store(void *p, long long at, int t, int D, const float (&v)[E]) {
        T *row = static_cast<T *>(p) + at;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int c = (t + i * TPR) * VEC;
            if (c >= D) continue;
            if constexpr (VEC == 1) {
                row[c] = (T)v[i];
            } else {
                uint32_t w[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    if constexpr (sizeof(T) == 2) {
                        const __nv_bfloat162 b = __floats2bfloat162_rn(v[i * VEC + 2 * u], v[i * VEC + 2 * u + 1]);
                        w[u] = *reinterpret_cast<const uint32_t *>(&b);
                    } else {
                        w[u] = __float_as_uint(v[i * VEC + u]);
                    }
                }
                __stcs(reinterpret_cast<uint4 *>(row + c), make_uint4(w[0], w[1], w[2], w[3]));
            }
        }
    }
};

// Sums of N values over the TPR threads of a row, the same in each of them and from run to run.  `room`: 4 floats a warp, twice; `turn`
// goes from one half to the other with each sum, so that one barrier a sum is enough.
template <int TPR, int N> __device__ __forceinline__ void row_sums(float (&v)[N], float *room, int &turn) {
    constexpr int WIDE = TPR < 32 ? TPR : 32;
#pragma unroll
    for (int o = WIDE / 2; o; o >>= 1)
#pragma unroll
        for (int u = 0; u < N; ++u) v[u] += __shfl_xor_sync(0xffffffffu, v[u], o);
    if constexpr (TPR > 32) {
        constexpr int WARPS = TPR / 32;
        room += (threadIdx.x / TPR * 2 + turn) * WARPS * 4;
        turn ^= 1;
        const int warp = threadIdx.x % TPR / 32, lane = threadIdx.x % 32;
        if (lane == 0)
#pragma unroll
            for (int u = 0; u < N; ++u) room[warp * 4 + u] = v[u];
        __syncthreads();
#pragma unroll
        for (int u = 0; u < N; ++u) {
            float s = lane < WARPS ? room[lane * 4 + u] : 0.f;
#pragma unroll
            for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            v[u] = s;
        }
    }
}

template <class T, int VEC, int TPR> __global__ void __launch_bounds__(TPR < 256 ? 256 : TPR, TPR > 256 ? 1024 / TPR : VEC == 8 ? 4 : 3) norm_kernel(const __grid_constant__ Args A) {
    constexpr int E = MOST_E;
    using S = Slot<T, VEC, TPR, E>;
    constexpr int THREADS = TPR < 256 ? 256 : TPR, GROUPS = THREADS / TPR;
    __shared__ float room[GROUPS * 2 * (TPR / 32 + 1) * 4];
    const int t = threadIdx.x % TPR;
    int turn = 0;
    const long long row = (long long)blockIdx.x * GROUPS + threadIdx.x / TPR;
    const bool in = row < A.rows;
    const int D = in ? A.D : 0;
    const long long at = in ? row * A.D : 0;
    typename S::Raw x, gate, res;
    S::load(A.x, at, t, D, x);
    if (A.gate) S::load(A.gate, at, t, D, gate);
    if (A.residual) S::load(A.residual, at, t, D, res);
    float z[E], w[E];
    float r = 1.f;
    if (A.post) {
        float sum[1] = {0.f};
#pragma unroll
        for (int e = 0; e < E; ++e) sum[0] = fmaf(S::value(x, e), S::value(x, e), sum[0]);
        row_sums<TPR>(sum, room, turn);
        r = rsqrtf(sum[0] / A.D + A.eps);
        S::weights(A.post, t, D, w);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
        z[e] = A.post ? S::value(x, e) * r * w[e] : S::value(x, e);
        if (A.gate) {
            const float g = S::value(gate, e), a = sigmoid_of<T>(g);
            z[e] *= A.silu ? g * a : a;
        }
        z[e] = A.residual ? fmaf(A.alpha, z[e], S::value(res, e)) : A.alpha * z[e];
    }
    if (A.s) S::store(A.s, at, t, D, z);
    if (A.pre) {
        float sum[1] = {0.f};
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (S::column(t, e) < D) sum[0] = fmaf(z[e], z[e], sum[0]);
        row_sums<TPR>(sum, room, turn);
        r = rsqrtf(sum[0] / A.D + A.eps);
        S::weights(A.pre, t, D, w);
#pragma unroll
        for (int e = 0; e < E; ++e) z[e] = z[e] * r * w[e];
        S::store(A.y, at, t, D, z);
    }
}

// Rows on their way: up to five arrays' next GROUPS rows (one stretch of memory) in shared memory, two deep, while those before are worked on.
// A copy starts and ends on 16 bytes, so it may hold up to 15 more on either side, never past the array's last whole 16; what lies behind is
// fetched by the threads.
template <class T, int TPR, int E> struct Ring {
    static constexpr int THREADS = TPR < 256 ? 256 : TPR, GROUPS = THREADS / TPR;
    static constexpr int ARRAYS = 5;
    static constexpr bool FITS = 2 * ARRAYS * (TPR * GROUPS * E * (int)sizeof(T) + 32) <= 220 * 1024;
    // Bytes of an array's rows (the weights' sums meet in their place).
    static __host__ __device__ int most(int D) { return ((GROUPS * D * (int)sizeof(T) + 15) & ~15) + 32; }
    static int bytes(int D) { const int n = 2 * ARRAYS * most(D), m = GROUPS > 1 ? GROUPS * TPR * E * 4 : 0; return n > m ? n : m; }
};

// The weights' gradients: a thread keeps its columns' sums over the rows of its CTA, in a fixed order.
template <class T, int VEC, int TPR, int E> __global__ void __launch_bounds__(TPR < 256 ? 256 : TPR, TPR <= 256 ? 2 : 1) norm_grad_kernel(const __grid_constant__ Args A) {
    using S = Slot<T, VEC, TPR, E>;
    using Q = Ring<T, TPR, E>;
    constexpr int THREADS = Q::THREADS, GROUPS = Q::GROUPS;
    extern __shared__ __align__(16) char ring[];
    __shared__ float room[GROUPS * 2 * (TPR / 32 + 1) * 4];
    __shared__ __align__(8) unsigned long long full[2];
    __shared__ int late;
    const int t = threadIdx.x % TPR, group = threadIdx.x / TPR, D0 = A.D, most = Q::most(D0);
    const long long step = (long long)gridDim.x * GROUPS;
    int turn = 0;
    const T *const arrays[5] = {static_cast<const T *>(A.ds), static_cast<const T *>(A.x), static_cast<const T *>(A.gate), static_cast<const T *>(A.s_in),
                                static_cast<const T *>(A.dy)};
    if (threadIdx.x == 0) {
        tc::mbar_init(tc::smem_u32(&full[0]), 1);
        tc::mbar_init(tc::smem_u32(&full[1]), 1);
        tc::fence_mbar_init();
        late = 0;
    }
    __syncthreads();
    // the copies of rows r0 .. r0 + GROUPS - 1 (one thread)
    auto ask = [&](long long r0, int s) {
        const long long n = min((long long)GROUPS, A.rows - r0);
        uint32_t bytes = 0;
        tc::fence_async_smem();
#pragma unroll
        for (int pass = 0; pass < 2; ++pass) {
            if (pass) tc::mbar_arrive_expect_tx(tc::smem_u32(&full[s]), bytes);
#pragma unroll
            for (int k = 0; k < 5; ++k) {
                if (!arrays[k]) continue;
                const uintptr_t a = reinterpret_cast<uintptr_t>(arrays[k] + r0 * D0), z = reinterpret_cast<uintptr_t>(arrays[k] + (r0 + n) * D0),
                                last = reinterpret_cast<uintptr_t>(arrays[k] + A.rows * D0) & ~(uintptr_t)15;
                // (the array may begin off 16 bytes: its first piece is then the threads' too)
                const uintptr_t first = (reinterpret_cast<uintptr_t>(arrays[k]) + 15) & ~(uintptr_t)15;
                const uintptr_t from = max(a & ~(uintptr_t)15, first), to = min((z + 15) & ~(uintptr_t)15, last);
                if (from >= to) continue;
                if (!pass) bytes += (uint32_t)(to - from);
                else tc::bulk_g2s(tc::smem_u32(ring + s * (Q::ARRAYS * most) + k * most + (from - (a & ~(uintptr_t)15))), reinterpret_cast<const void *>(from), (uint32_t)(to - from), tc::smem_u32(&full[s]));
            }
        }
    };
    const long long begin = (long long)blockIdx.x * GROUPS;
    if (Q::FITS && threadIdx.x == 0)
        for (int s = 0; s < 2; ++s)
            if (begin + s * step < A.rows) ask(begin + s * step, s);
    float sum_post[E], sum_pre[E];
#pragma unroll
    for (int e = 0; e < E; ++e) sum_post[e] = sum_pre[e] = 0.f;
    const float inv = 1.f / D0;
    int it = 0;
    for (long long r0 = begin; r0 < A.rows; r0 += step, ++it) {
        const int s = it & 1;
        const long long row = r0 + group;
        const bool in = row < A.rows;
        const int D = in ? D0 : 0;
        const long long at = in ? row * D0 : 0;
        if (Q::FITS) {
            bool there = false;
            for (uint32_t i = 0; i < 1u << 20 && !there; ++i) there = tc::mbar_try_wait(tc::smem_u32(&full[s]), it >> 1 & 1);
            if (!there) late = 1;
        }
        // array k's elements of this thread
        auto row_of = [&](int k, typename S::Raw &r) {
            if constexpr (Q::FITS) {
                const uintptr_t a = reinterpret_cast<uintptr_t>(arrays[k] + r0 * D0), own = reinterpret_cast<uintptr_t>(arrays[k] + at);
                S::template fetch<false>(reinterpret_cast<const T *>(ring + s * (Q::ARRAYS * most) + k * most + (own - (a & ~(uintptr_t)15))), t, D, r);
                if constexpr (VEC == 1) {
                    // the pieces of the array's ends that no copy holds
                    const uintptr_t first = (reinterpret_cast<uintptr_t>(arrays[k]) + 15) & ~(uintptr_t)15, last = reinterpret_cast<uintptr_t>(arrays[k] + A.rows * D0) & ~(uintptr_t)15;
                    if (own < first || own + D * sizeof(T) > last) S::template fetch<true>(arrays[k] + at, t, D, r);
                }
            } else {
                S::template fetch<true>(arrays[k] + at, t, D, r);
            }
        };
        typename S::Raw sr, dyr, xr;
        float d[E], w[E], sums[3] = {0.f, 0.f, 0.f};
        if (A.pre) {
            row_of(3, sr);
            row_of(4, dyr);
            S::weights(A.pre, t, D, w);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float v = S::value(sr, e);
                sums[0] = fmaf(v, v, sums[0]);
                sums[1] = fmaf(S::value(dyr, e) * w[e], v, sums[1]);
            }
        }
        if (A.x) row_of(1, xr);
        if (A.post)
#pragma unroll
            for (int e = 0; e < E; ++e) sums[2] = fmaf(S::value(xr, e), S::value(xr, e), sums[2]);
        if (A.pre || A.post) row_sums<TPR>(sums, room, turn);
        {
            typename S::Raw dsr;
            row_of(0, dsr);
#pragma unroll
            for (int e = 0; e < E; ++e) d[e] = S::value(dsr, e);
        }
        if (A.pre) {
            if (Q::FITS && sizeof(T) == 4) {                         // (fetched again rather than kept: 32 registers)
                row_of(3, sr);
                row_of(4, dyr);
            }
            // (a row that is not there has factors of 0: with an eps of 0 they would be infinite, and its zeros NaN in the weights' sums)
            const float r = in ? rsqrtf(sums[0] * inv + A.eps) : 0.f, m = sums[1] * inv * r;     // m: mean(dy pre h_s)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float h = S::value(sr, e) * r, y = S::value(dyr, e);
                sum_pre[e] = fmaf(y, h, sum_pre[e]);
                d[e] = fmaf(r, fmaf(-h, m, y * w[e]), d[e]);
            }
        }
        if (A.dresidual) S::store(A.dresidual, at, t, D, d);
#pragma unroll
        for (int e = 0; e < E; ++e) d[e] *= A.alpha;
        const float r = !A.post ? 1.f : in ? rsqrtf(sums[2] * inv + A.eps) : 0.f;
        if (A.post) S::weights(A.post, t, D, w);
        if (A.x && Q::FITS && sizeof(T) == 4) row_of(1, xr);
        if (A.gate) {
            typename S::Raw gr;
            float g[E];
            row_of(2, gr);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float z = S::value(gr, e), a = sigmoid_of<T>(z), x = S::value(xr, e), u = A.post ? x * r * w[e] : x;
                g[e] = d[e] * u * (A.silu ? a * fmaf(z, 1.f - a, 1.f) : a * (1.f - a));
                d[e] *= A.silu ? z * a : a;
            }
            S::store(A.dgate, at, t, D, g);
        }
        if (A.post) {
            float mean[1] = {0.f};
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float h = S::value(xr, e) * r;
                sum_post[e] = fmaf(d[e], h, sum_post[e]);
                d[e] *= w[e];
                mean[0] = fmaf(d[e], h, mean[0]);
            }
            row_sums<TPR>(mean, room, turn);
            mean[0] *= inv;
#pragma unroll
            for (int e = 0; e < E; ++e) d[e] = r * fmaf(-(S::value(xr, e) * r), mean[0], d[e]);
        }
        S::store(A.dx, at, t, D, d);
        if (Q::FITS) {
            __syncthreads();                                         // the stage has been read
            if (late) {
                // (a copy that did not come: rows that are not a number rather than wrong ones, and no more of them)
                const float nan = __int_as_float(0x7fffffff);
#pragma unroll
                for (int e = 0; e < E; ++e) d[e] = sum_pre[e] = sum_post[e] = nan;
                S::store(A.dx, at, t, D, d);
                break;
            }
            if (threadIdx.x == 0 && r0 + 2 * step < A.rows) ask(r0 + 2 * step, s);
        }
    }
    if (late && threadIdx.x == 0)                                    // (nothing may be on its way into shared memory when the CTA ends)
        for (int k = max(0, it - 1); k < it + 2; ++k)
            for (uint32_t i = 0; i < 1u << 20 && !tc::mbar_try_wait(tc::smem_u32(&full[k & 1]), k >> 1 & 1); ++i) {}
    __syncthreads();
    float *const meet = reinterpret_cast<float *>(ring);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        if (which ? !A.pre : !A.post) continue;
        float(&sum)[E] = which ? sum_pre : sum_post;
        float *to = A.parts + ((long long)which * gridDim.x + blockIdx.x) * D0;
        if constexpr (GROUPS > 1) {
            __syncthreads();
#pragma unroll
            for (int e = 0; e < E; ++e) meet[group * TPR * E + S::column(t, e)] = sum[e];
            __syncthreads();
            for (int c = threadIdx.x; c < D0; c += THREADS) {
                float v = 0.f;
                for (int g = 0; g < GROUPS; ++g) v += meet[g * TPR * E + c];
                to[c] = v;
            }
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (S::column(t, e) < D0) to[S::column(t, e)] = sum[e];
        }
    }
}

template <class T, int VEC, int TPR, int E> cudaError_t launch_grad(const Args &a, cudaStream_t s) {
    static std::atomic<uint64_t> attr{0};
    using Q = Ring<T, TPR, E>;
    const int bytes = Q::FITS ? Q::bytes(a.D) : 0;
    if (Q::FITS)
        if (cudaError_t e = smem_attr_once((const void *)norm_grad_kernel<T, VEC, TPR, E>, Q::bytes(TPR * E), attr)) return e;
    norm_grad_kernel<T, VEC, TPR, E><<<(unsigned)parts_of(a.rows, a.D), TPR < 256 ? 256 : TPR, bytes, s>>>(a);
    count_launch();
    return cudaGetLastError();
}
template <class T, int VEC, int TPR> cudaError_t launch(const Args &a, bool grad, cudaStream_t s) {
    constexpr int THREADS = TPR < 256 ? 256 : TPR, GROUPS = THREADS / TPR;
    if (grad) {
        // (single elements: all that a thread may hold is worked on, whether the row has it or not, and with 16 it does not fit
        // the registers: 2,777 rows of 1,111 in FP32 take 49 us with 16 and 41 with 12)
        if constexpr (VEC == 1 && TPR < 256) {
            if (a.D <= TPR * 8) return launch_grad<T, VEC, TPR, 8>(a, s);
            if (a.D <= TPR * 12) return launch_grad<T, VEC, TPR, 12>(a, s);
        }
        return launch_grad<T, VEC, TPR, MOST_E>(a, s);
    }
    norm_kernel<T, VEC, TPR><<<(unsigned)((a.rows + GROUPS - 1) / GROUPS), THREADS, 0, s>>>(a);
    count_launch();
    return cudaGetLastError();
}

template <class T, int VEC> cudaError_t launch_width(const Args &a, bool grad, cudaStream_t s) {
    switch (threads_a_row(a.D)) {
    case 8: return launch<T, VEC, 8>(a, grad, s);
    case 32: return launch<T, VEC, 32>(a, grad, s);
    case 128: return launch<T, VEC, 128>(a, grad, s);
    case 256: return launch<T, VEC, 256>(a, grad, s);
    case 512: return launch<T, VEC, 512>(a, grad, s);
    default: return launch<T, VEC, 1024>(a, grad, s);
    }
}

template <class T> cudaError_t launch_type(const Args &a, bool grad, cudaStream_t s) {
    uintptr_t all = 0;
    for (const void *p : {a.x, a.gate, a.residual, a.s_in, a.ds, a.dy, (const void *)a.post, (const void *)a.pre, (const void *)a.s, (const void *)a.y,
                          (const void *)a.dx, (const void *)a.dgate, (const void *)a.dresidual})
        all |= reinterpret_cast<uintptr_t>(p);
    if (a.D % kVec<T> == 0 && (all & 15) == 0) return launch_width<T, kVec<T>>(a, grad, s);
    return launch_width<T, 1>(a, grad, s);
}

cudaError_t launch_bf16(const Args &a, bool grad, cudaStream_t s);
cudaError_t launch_f32(const Args &a, bool grad, cudaStream_t s);

}  // namespace blk

size_t blk_norm_workspace(long long rows, int D);
cudaError_t launch_blk_norm(const blk::Args &a, int bf16, bool grad, cudaStream_t s);

}  // namespace k3kda
