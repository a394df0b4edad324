// rope.cu -- rotary positions of the attention layers on sm_103a: forward and gradient.
//
//   (x, y) -> m (x cos - y sin, y cos + x sin),   angle = position * f_i            (forward)
//   (x, y) -> m (x cos + y sin, y cos - x sin)                                      (gradient: the transpose)
//
// Bound by HBM: each element is read and written once.  A thread's item is two 16-byte pieces of one
// (token, head) row: the two halves' pieces i and i + dim/2 (HALF), two neighbouring pieces
// (INTERLEAVED), or two pieces that pass through.  A CTA takes kThreads * kItems items of
// consecutive (token, head) rows, issues their loads, and only then forms its tokens' cosines and
// sines in shared memory, once for all heads, so that the angles' arithmetic lies under the loads.
// Rows that are not 16-byte aligned go one element at a time (V = 1) through the same code.
//
// A key head that all heads shared gets the sum of their gradients: the CTA's threads divide the
// heads among themselves, add their sums in shared memory in a fixed order and turn the total.
#include <math.h>

#include "rope.cuh"

namespace k3kda {
namespace {

constexpr int kThreads = 256;
constexpr int kItems = 2;                 // items of a thread
constexpr int kTable = 4096;              // most (cos, sin) pairs of a CTA's tokens (32 KB)
constexpr int kSplit = 8;                 // threads that divide a shared head's sum

struct RopeJob {                          // one array's rotation
    View in, out;
    int heads;
    int copy;                             // pieces that pass through (0 when in place)
    int pairs;                            // items per head that turn
    int items;                            // items per head
};

struct RopeArgs {
    RopeJob a, b;                         // b.heads = 0: none
    int shared;                           // b's output is one head, the sum over b.heads
    const int32_t *pos;
    int T;
    Rope r;
    int per_token;                        // items per token (a and, unless shared, b)
    int block_items;                      // items of a CTA
    unsigned main_blocks;                 // CTAs of the plain rotation; the rest form the shared sums
    int shared_tokens;                    // tokens of a CTA of the shared sums
    int table;                            // (cos, sin) pairs in shared memory
    float sgn;                            // +1 forward, -1 gradient
};

template <typename T, int V> struct Piece { T x[V]; };

template <typename T, int V> __device__ __forceinline__ Piece<T, V> ld(const T *p) {
    Piece<T, V> r;
    if constexpr (sizeof(T) * V == 16) *reinterpret_cast<uint4 *>(r.x) = __ldcs(reinterpret_cast<const uint4 *>(p));
    else r.x[0] = *p;
    return r;
}
template <typename T, int V> __device__ __forceinline__ void st(T *p, const Piece<T, V> &r) {
    if constexpr (sizeof(T) * V == 16) *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<const uint4 *>(r.x);
    else *p = r.x[0];
}
__device__ __forceinline__ float tof(float x) { return x; }
__device__ __forceinline__ float tof(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T> __device__ __forceinline__ T fromf(float x) {
    if constexpr (sizeof(T) == 4) return x;
    else return __float2bfloat16_rn(x);
}

// the channels of item `it`'s two pieces (second < 0: none); turned = whether they are a pair's
template <int V> __device__ __forceinline__ bool item_at(const Rope &r, const RopeJob &j, int it, int &c0, int &c1) {
    if (it < j.pairs) {
        c0 = r.off + (r.inter ? 2 * V * it : V * it);
        c1 = c0 + (r.inter ? V : r.half);
        return true;
    }
    const int first = 2 * (it - j.pairs), pre = r.off / V, skip = r.dim / V;
    c0 = V * (first < pre ? first : first + skip);
    c1 = first + 1 < j.copy ? V * (first + 1 < pre ? first + 1 : first + 1 + skip) : -1;
    return false;
}

// pairs of the two pieces: HALF turns a.x[e] with b.x[e], INTERLEAVED the neighbours of (a, b) in a row
template <int V> __device__ __forceinline__ void turn(float (&a)[V], float (&b)[V], const float2 *cs, int pair0, int inter, float sgn) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const float2 t = cs[pair0 + e];
        float &x = !inter ? a[e] : (V == 1 ? a[0] : (2 * e < V ? a[2 * e % V] : b[2 * e % V]));
        float &y = !inter ? b[e] : (V == 1 ? b[0] : (2 * e < V ? a[(2 * e + 1) % V] : b[(2 * e + 1) % V]));
        const float s = sgn * t.y, nx = x * t.x - y * s, ny = y * t.x + x * s;
        x = nx;
        y = ny;
    }
}

__device__ __forceinline__ void fill_table(const RopeArgs &A, float2 *cs, int t0, int n) {
    for (int i = threadIdx.x; i < n * A.r.half; i += kThreads) {
        const int t = i / A.r.half;
        const float2 v = rope_cs(A.r.phase[i - t * A.r.half], A.pos[t0 + t]);
        cs[i] = make_float2(v.x * A.r.mscale, v.y * A.r.mscale);
    }
}

template <typename T, int V> __device__ void plain_block(const RopeArgs &A, float2 *cs) {
    // items of all tokens in one row; a CTA's run of them spans at most block_items / per_token + 2 tokens
    const int64_t base = (int64_t)blockIdx.x * A.block_items, all = (int64_t)A.T * A.per_token;
    const int count = (int)min((int64_t)A.block_items, all - base);
    const int t0 = (int)(base / A.per_token), e0 = (int)(base - (int64_t)t0 * A.per_token);
    const int n = (e0 + count - 1) / A.per_token + 1;
    const int na = A.a.heads * A.a.items;
    T *dst[kItems];
    int c0[kItems], c1[kItems], pair[kItems];
    Piece<T, V> x[kItems], y[kItems];
#pragma unroll
    for (int u = 0; u < kItems; ++u) {
        const int i = u * kThreads + threadIdx.x;
        pair[u] = -2;
        if (i >= count) continue;
        const int t = (e0 + i) / A.per_token;
        int e = e0 + i - t * A.per_token;
        const bool second = e >= na;
        const RopeJob &j = second ? A.b : A.a;
        e -= second ? na : 0;
        const int h = e / j.items, it = e - h * j.items;
        const bool turned = item_at<V>(A.r, j, it, c0[u], c1[u]);
        const T *src = reinterpret_cast<const T *>(j.in.p) + (int64_t)(t0 + t) * j.in.ts + (int64_t)h * j.in.hs;
        dst[u] = reinterpret_cast<T *>(j.out.p) + (int64_t)(t0 + t) * j.out.ts + (int64_t)h * j.out.hs;
        x[u] = ld<T, V>(src + c0[u]);
        if (c1[u] >= 0) y[u] = ld<T, V>(src + c1[u]);
        pair[u] = turned ? t * A.r.half + V * it : -1;
    }
    fill_table(A, cs, t0, n);
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kItems; ++u) {
        if (pair[u] == -2) continue;
        if (pair[u] >= 0) {
            float a[V], b[V];
#pragma unroll
            for (int e = 0; e < V; ++e) { a[e] = tof(x[u].x[e]); b[e] = tof(y[u].x[e]); }
            turn<V>(a, b, cs, pair[u], A.r.inter, A.sgn);
#pragma unroll
            for (int e = 0; e < V; ++e) { x[u].x[e] = fromf<T>(a[e]); y[u].x[e] = fromf<T>(b[e]); }
        }
        st<T, V>(dst[u] + c0[u], x[u]);
        if (c1[u] >= 0) st<T, V>(dst[u] + c1[u], y[u]);
    }
}

// The gradient of a shared head: item i of the CTA's tokens is summed over the heads by kSplit
// threads (heads s, s + kSplit, ...), whose sums meet in shared memory.
template <typename T, int V> __device__ void shared_block(const RopeArgs &A, float2 *cs, float *part) {
    const int t0 = (int)(blockIdx.x - A.main_blocks) * A.shared_tokens, n = min(A.shared_tokens, A.T - t0);
    const RopeJob &j = A.b;
    fill_table(A, cs, t0, n);
    constexpr int kPer = kThreads / kSplit;               // items at a time
    const int slot = threadIdx.x % kPer, s = threadIdx.x / kPer;
    for (int base = 0; base < n * j.items; base += kPer) {
        const int i = base + slot;
        const bool live = i < n * j.items;
        const int t = live ? i / j.items : 0, it = live ? i - t * j.items : 0;
        int c0 = 0, c1 = -1;
        const bool turned = item_at<V>(A.r, j, it, c0, c1);
        float a[V], b[V];
#pragma unroll
        for (int e = 0; e < V; ++e) a[e] = b[e] = 0.f;
        if (live) {
            const T *src = reinterpret_cast<const T *>(j.in.p) + (int64_t)(t0 + t) * j.in.ts;
#pragma unroll 4
            for (int h = s; h < j.heads; h += kSplit) {
                const Piece<T, V> x = ld<T, V>(src + (int64_t)h * j.in.hs + c0);
                Piece<T, V> y = x;
                if (c1 >= 0) y = ld<T, V>(src + (int64_t)h * j.in.hs + c1);
#pragma unroll
                for (int e = 0; e < V; ++e) { a[e] += tof(x.x[e]); b[e] += tof(y.x[e]); }
            }
        }
        __syncthreads();                                  // the table is there; the last round's sums are read
#pragma unroll
        for (int e = 0; e < V; ++e) {
            part[(2 * e) * kThreads + threadIdx.x] = a[e];
            part[(2 * e + 1) * kThreads + threadIdx.x] = b[e];
        }
        __syncthreads();
        if (s != 0 || !live) continue;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            for (int k = 1; k < kSplit; ++k) {
                a[e] += part[(2 * e) * kThreads + k * kPer + slot];
                b[e] += part[(2 * e + 1) * kThreads + k * kPer + slot];
            }
        }
        if (turned) turn<V>(a, b, cs, t * A.r.half + V * it, A.r.inter, A.sgn);
        T *dst = reinterpret_cast<T *>(j.out.p) + (int64_t)(t0 + t) * j.out.ts;
        Piece<T, V> x, y;
#pragma unroll
        for (int e = 0; e < V; ++e) { x.x[e] = fromf<T>(a[e]); y.x[e] = fromf<T>(b[e]); }
        st<T, V>(dst + c0, x);
        if (c1 >= 0) st<T, V>(dst + c1, y);
    }
}

template <typename T, int V> __global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs A) {
    extern __shared__ float2 cs[];
    if (blockIdx.x < A.main_blocks) plain_block<T, V>(A, cs);
    else shared_block<T, V>(A, cs, reinterpret_cast<float *>(cs + A.table));
}

RopeJob make_job(const k3mla_view *in, const k3mla_view *out, int H, int d, const Rope &r, int V, bool in_place) {
    RopeJob j{};
    j.heads = H;
    if (H == 0) return j;
    j.in = make_view(in);
    j.out = make_view(out);
    j.pairs = r.half / V;
    j.copy = in_place ? 0 : (d - r.dim) / V;
    j.items = j.pairs + (j.copy + 1) / 2;
    return j;
}

bool same(const k3mla_view *a, const k3mla_view *b) {
    return a->data == b->data && a->token_stride == b->token_stride && a->head_stride == b->head_stride;
}

}  // namespace

cudaError_t launch_rope(const k3mla_view *q, const k3mla_view *q_out, int Hq, const k3mla_view *k, const k3mla_view *k_out,
                        int Hk, int shared, int bf16, const int32_t *pos, int T, int d, const k3mla_rope_args *rope,
                        float sgn, cudaStream_t s) {
    RopeArgs A;
    A.r = make_rope(rope);
    A.pos = pos;
    A.T = T;
    A.sgn = sgn;
    A.shared = shared;
    const int size = bf16 ? 2 : 4;
    int V = 16 / size;
    const Rope &r = A.r;
    bool vec = d % V == 0 && r.off % V == 0 && (r.inter ? r.dim % (2 * V) == 0 : r.half % V == 0);
    vec = vec && (Hq == 0 || (view_vec(q, size, T, Hq) && view_vec(q_out, size, T, Hq)));
    vec = vec && (Hk == 0 || (view_vec(k, size, T, Hk) && view_vec(k_out, size, T, shared ? 1 : Hk)));
    if (!vec) V = 1;
    A.a = make_job(q, q_out, Hq, d, r, V, Hq && same(q, q_out));
    A.b = make_job(k, k_out, Hk, d, r, V, Hk && !shared && same(k, k_out));
    A.per_token = A.a.heads * A.a.items + (shared ? 0 : A.b.heads * A.b.items);
    // a CTA's items, fewer where many tokens' tables would not fit
    const int fit = r.half > 0 ? kTable / r.half : 1 << 20;
    const long long most = (long long)(fit - 2) * A.per_token;
    A.block_items = (int)(most < kThreads * kItems ? most : kThreads * kItems);
    const long long main_blocks = A.per_token ? ((long long)T * A.per_token + A.block_items - 1) / A.block_items : 0;
    int spans = A.per_token ? A.block_items / A.per_token + 2 : 0;
    // shared sums: as many tokens as fill kThreads / kSplit items
    A.shared_tokens = 1;
    long long shared_blocks = 0;
    if (shared) {
        A.shared_tokens = kThreads / kSplit / A.b.items;
        A.shared_tokens = A.shared_tokens < 1 ? 1 : A.shared_tokens > fit ? fit : A.shared_tokens;
        shared_blocks = (T + A.shared_tokens - 1) / A.shared_tokens;
        spans = spans > A.shared_tokens ? spans : A.shared_tokens;
    }
    A.table = r.half * (spans < T ? spans : T);
    const size_t smem = (size_t)A.table * sizeof(float2) + (shared ? (size_t)2 * V * kThreads * sizeof(float) : 0);
    if (main_blocks + shared_blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    if (main_blocks + shared_blocks == 0) return cudaSuccess;      // everything in place and nothing to turn
    A.main_blocks = (unsigned)main_blocks;
    const unsigned grid = (unsigned)(main_blocks + shared_blocks);
    if (bf16 && V > 1) rope_kernel<__nv_bfloat16, 8><<<grid, kThreads, smem, s>>>(A);
    else if (bf16) rope_kernel<__nv_bfloat16, 1><<<grid, kThreads, smem, s>>>(A);
    else if (V > 1) rope_kernel<float, 4><<<grid, kThreads, smem, s>>>(A);
    else rope_kernel<float, 1><<<grid, kThreads, smem, s>>>(A);
    count_launch();
    return cudaGetLastError();
}

}  // namespace k3kda
