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
// Every array is read once and written once: a row is held in registers by its threads, 16 elements each, so HBM bounds both.  Rows
// of up to 128 channels take 8 threads, of up to 16384 a CTA of 1024; arrays move in 16-byte pieces where the width and the
// addresses allow it, else element by element.  All arithmetic is FP32, each output is rounded once; y comes from the sum
// before its rounding.
#pragma once

#include "common.cuh"

namespace k3kda {
namespace blk {

constexpr int E = 16;                  // elements of a row that one thread holds
constexpr int MOST_D = 1024 * E;
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
    const int need = (D + E - 1) / E;
    return need <= 8 ? 8 : need <= 32 ? 32 : need <= 128 ? 128 : need <= 256 ? 256 : need <= 512 ? 512 : 1024;
}
inline long long groups_of(int tpr) { return tpr < 256 ? 256 / tpr : 1; }
inline int parts_of(long long rows, int D) {
    const long long g = groups_of(threads_a_row(D)), need = (rows + g - 1) / g;
    return (int)(need < MOST_PARTS ? need : MOST_PARTS);
}

template <class T> struct Raw;
template <> struct Raw<__nv_bfloat16> { static constexpr int VEC = 8; };
template <> struct Raw<float> { static constexpr int VEC = 4; };

template <class T> __device__ __forceinline__ float exp_of(float x) { return sizeof(T) == 2 ? __expf(x) : expf(x); }
template <class T> __device__ __forceinline__ float inverse(float x) { return sizeof(T) == 2 ? __fdividef(1.f, x) : 1.f / x; }
// sigmoid(z); where 1 + e^-z is too large for the fast division it gives 0, as it should
template <class T> __device__ __forceinline__ float sigmoid_of(float z) { return inverse<T>(1.f + exp_of<T>(-z)); }

// Thread t's elements of a row: pieces of VEC at (t + i TPR) VEC.
template <class T, int VEC, int TPR> struct Slot {
    static constexpr int ITEMS = E / VEC;
    static __device__ __forceinline__ int column(int t, int e) { return (t + e / VEC * TPR) * VEC + e % VEC; }
    static __device__ __forceinline__ void load(const void *p, long long at, int t, int D, float (&v)[E]) {
        const T *row = static_cast<const T *>(p) + at;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int c = (t + i * TPR) * VEC;
            if constexpr (VEC == 1) {
                v[i] = c < D ? (float)row[c] : 0.f;
            } else {
                uint4 r = make_uint4(0, 0, 0, 0);
                if (c < D) r = __ldcs(reinterpret_cast<const uint4 *>(row + c));
                const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    if constexpr (sizeof(T) == 2) {
                        v[i * VEC + 2 * u] = __uint_as_float(w[u] << 16);
                        v[i * VEC + 2 * u + 1] = __uint_as_float(w[u] & 0xffff0000u);
                    } else {
                        v[i * VEC + u] = __uint_as_float(w[u]);
                    }
                }
            }
        }
    }
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

template <class T, int VEC, int TPR> __global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) norm_kernel(const __grid_constant__ Args A) {
    using S = Slot<T, VEC, TPR>;
    constexpr int THREADS = TPR < 256 ? 256 : TPR, GROUPS = THREADS / TPR;
    __shared__ float room[GROUPS * 2 * (TPR / 32 + 1) * 4];
    const int t = threadIdx.x % TPR;
    int turn = 0;
    const long long row = (long long)blockIdx.x * GROUPS + threadIdx.x / TPR;
    const bool in = row < A.rows;
    const int D = in ? A.D : 0;
    const long long at = in ? row * A.D : 0;
    float z[E], gate[E], res[E], w[E];
    S::load(A.x, at, t, D, z);
    if (A.gate) S::load(A.gate, at, t, D, gate);
    if (A.residual) S::load(A.residual, at, t, D, res);
    if (A.post) {
        float sum[1] = {0.f};
        S::weights(A.post, t, D, w);
#pragma unroll
        for (int e = 0; e < E; ++e) sum[0] = fmaf(z[e], z[e], sum[0]);
        row_sums<TPR>(sum, room, turn);
        const float r = rsqrtf(sum[0] / A.D + A.eps);
#pragma unroll
        for (int e = 0; e < E; ++e) z[e] = z[e] * r * w[e];
    }
    if (A.gate) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float a = sigmoid_of<T>(gate[e]);
            z[e] *= A.silu ? gate[e] * a : a;
        }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) z[e] = A.residual ? fmaf(A.alpha, z[e], res[e]) : A.alpha * z[e];
    if (A.s) S::store(A.s, at, t, D, z);
    if (A.pre) {
        float sum[1] = {0.f};
        S::weights(A.pre, t, D, w);
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (S::column(t, e) < D) sum[0] = fmaf(z[e], z[e], sum[0]);
        row_sums<TPR>(sum, room, turn);
        const float r = rsqrtf(sum[0] / A.D + A.eps);
#pragma unroll
        for (int e = 0; e < E; ++e) z[e] = z[e] * r * w[e];
        S::store(A.y, at, t, D, z);
    }
}

// The weights' gradients: a thread keeps its columns' sums over the rows of its CTA, in a fixed order.
template <class T, int VEC, int TPR> __global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) norm_grad_kernel(const __grid_constant__ Args A) {
    using S = Slot<T, VEC, TPR>;
    constexpr int THREADS = TPR < 256 ? 256 : TPR, GROUPS = THREADS / TPR;
    __shared__ float room[GROUPS * 2 * (TPR / 32 + 1) * 4];
    __shared__ float meet[GROUPS > 1 ? THREADS * E : 1];
    const int t = threadIdx.x % TPR, group = threadIdx.x / TPR;
    int turn = 0;
    float sum_post[E], sum_pre[E];
#pragma unroll
    for (int e = 0; e < E; ++e) sum_post[e] = sum_pre[e] = 0.f;
    const float inv = 1.f / A.D;
    for (long long r0 = (long long)blockIdx.x * GROUPS; r0 < A.rows; r0 += (long long)gridDim.x * GROUPS) {
        const long long row = r0 + group;
        const bool in = row < A.rows;
        const int D = in ? A.D : 0;
        const long long at = in ? row * A.D : 0;
        float d[E], x[E], gate[E], s[E], dy[E], w[E];
        S::load(A.ds, at, t, D, d);
        if (A.x) S::load(A.x, at, t, D, x);
        if (A.gate) S::load(A.gate, at, t, D, gate);
        float sums[3] = {0.f, 0.f, 0.f};
        if (A.pre) {
            S::load(A.s_in, at, t, D, s);
            S::load(A.dy, at, t, D, dy);
            S::weights(A.pre, t, D, w);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                sums[0] = fmaf(s[e], s[e], sums[0]);
                sums[1] = fmaf(dy[e] * w[e], s[e], sums[1]);
            }
        }
        if (A.post)
#pragma unroll
            for (int e = 0; e < E; ++e) sums[2] = fmaf(x[e], x[e], sums[2]);
        if (A.pre || A.post) row_sums<TPR>(sums, room, turn);
        if (A.pre) {
            const float r = rsqrtf(sums[0] * inv + A.eps), m = sums[1] * inv * r;     // m: mean(dy pre h_s)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float h = s[e] * r;
                sum_pre[e] = fmaf(dy[e], h, sum_pre[e]);
                d[e] = fmaf(r, fmaf(-h, m, dy[e] * w[e]), d[e]);
            }
        }
        if (A.dresidual) S::store(A.dresidual, at, t, D, d);
#pragma unroll
        for (int e = 0; e < E; ++e) d[e] *= A.alpha;
        const float r = A.post ? rsqrtf(sums[2] * inv + A.eps) : 1.f;
        if (A.post) S::weights(A.post, t, D, w);
        if (A.gate) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float z = gate[e], a = sigmoid_of<T>(z), u = A.post ? x[e] * r * w[e] : x[e];
                gate[e] = d[e] * u * (A.silu ? a * fmaf(z, 1.f - a, 1.f) : a * (1.f - a));
                d[e] *= A.silu ? z * a : a;
            }
            S::store(A.dgate, at, t, D, gate);
        }
        if (A.post) {
            float mean[1] = {0.f};
#pragma unroll
            for (int e = 0; e < E; ++e) {
                x[e] *= r;
                sum_post[e] = fmaf(d[e], x[e], sum_post[e]);
                d[e] *= w[e];
                mean[0] = fmaf(d[e], x[e], mean[0]);
            }
            row_sums<TPR>(mean, room, turn);
            mean[0] *= inv;
#pragma unroll
            for (int e = 0; e < E; ++e) d[e] = r * fmaf(-x[e], mean[0], d[e]);
        }
        S::store(A.dx, at, t, D, d);
    }
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        if (which ? !A.pre : !A.post) continue;
        float(&sum)[E] = which ? sum_pre : sum_post;
        float *to = A.parts + ((long long)which * gridDim.x + blockIdx.x) * A.D;
        if constexpr (GROUPS > 1) {
            __syncthreads();
#pragma unroll
            for (int e = 0; e < E; ++e) meet[group * TPR * E + S::column(t, e)] = sum[e];
            __syncthreads();
            for (int c = threadIdx.x; c < A.D; c += THREADS) {
                float v = 0.f;
                for (int g = 0; g < GROUPS; ++g) v += meet[g * TPR * E + c];
                to[c] = v;
            }
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (S::column(t, e) < A.D) to[S::column(t, e)] = sum[e];
        }
    }
}

template <class T, int VEC, int TPR> cudaError_t launch(const Args &a, bool grad, cudaStream_t s) {
    constexpr int THREADS = TPR < 256 ? 256 : TPR, GROUPS = THREADS / TPR;
    if (grad) norm_grad_kernel<T, VEC, TPR><<<(unsigned)parts_of(a.rows, a.D), THREADS, 0, s>>>(a);
    else norm_kernel<T, VEC, TPR><<<(unsigned)((a.rows + GROUPS - 1) / GROUPS), THREADS, 0, s>>>(a);
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
    if (a.D % Raw<T>::VEC == 0 && (all & 15) == 0) return launch_width<T, Raw<T>::VEC>(a, grad, s);
    return launch_width<T, 1>(a, grad, s);
}

cudaError_t launch_bf16(const Args &a, bool grad, cudaStream_t s);
cudaError_t launch_f32(const Args &a, bool grad, cudaStream_t s);

}  // namespace blk

size_t blk_norm_workspace(long long rows, int D);
cudaError_t launch_blk_norm(const blk::Args &a, int bf16, bool grad, cudaStream_t s);

}  // namespace k3kda
