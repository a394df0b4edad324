// rope.cu -- rotary positions of the attention layers on sm_103a: forward and gradient.
//
//   (x, y) -> m (x cos - y sin, y cos + x sin),   angle = position * f_i            (forward)
//   (x, y) -> m (x cos + y sin, y cos - x sin)                                      (gradient: the transpose)
//
// Bound by HBM: each element is read and written once.  A thread's item is two 16-byte pieces of a
// head: the two halves' pieces i and i + dim/2 (HALF), two neighbouring pieces
// (INTERLEAVED), or two pieces that pass through.  A thread keeps its item of its head and goes through its CTA's tokens,
// so that its place is worked out once and the next token's pieces are on their way while one is turned; the
// tokens' cosines and sines are formed once a CTA, for all heads, under the first loads.
// Rows that are not 16-byte aligned go one element at a time (V = 1) through the same code.
// Measured: 805 MB of bf16 heads in 147 us, 5.5 TB/s (81 % of a copy's rate); their gradient, 407 MB, in 76 us.
//
// A key head that all heads shared gets the sum of their gradients: a thread adds an item's heads, or, with few
// tokens, kSplit threads divide them, add their sums in shared memory in a fixed order and turn the total.
#include <math.h>

#include "rope.cuh"

namespace k3kda {
namespace {

constexpr int kThreads = 256;
constexpr int kTable = 4096;              // most (cos, sin) pairs of a CTA's tokens (32 KB)
constexpr int kTokens = 16;               // most tokens a thread goes through
constexpr int kSplit = 8;                 // threads that divide a shared head's sum where there are few

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
    int parts;                            // CTAs that share a token's items
    int side;                             // tokens side by side in a CTA (1 when a token fills it)
    int tokens;                           // tokens of a CTA, a multiple of side
    unsigned main_blocks;                 // CTAs of the plain rotation; the rest form the shared sums
    int shared_side;                      // tokens of a CTA of the shared sums
    int split;                            // threads that share an item's sum
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
    const int part = (int)(blockIdx.x % A.parts);
    const int t0 = (int)(blockIdx.x / A.parts) * A.tokens, n = min(A.tokens, A.T - t0);
    // this thread's item: which token of those side by side, which array, head and pieces
    int e = part * kThreads + threadIdx.x;
    const int st0 = e / A.per_token;
    e -= st0 * A.per_token;
    const int na = A.a.heads * A.a.items;
    const bool second = e >= na;
    const RopeJob &j = second ? A.b : A.a;
    e -= second ? na : 0;
    const int h = e / j.items, it = e - h * j.items;
    int c0, c1;
    const bool turned = item_at<V>(A.r, j, it, c0, c1);
    const T *src = reinterpret_cast<const T *>(j.in.p) + (int64_t)t0 * j.in.ts + (int64_t)h * j.in.hs;
    T *dst = reinterpret_cast<T *>(j.out.p) + (int64_t)t0 * j.out.ts + (int64_t)h * j.out.hs;
    const bool live = st0 < A.side && (A.parts == 1 || part * kThreads + (int)threadIdx.x < A.per_token);
    Piece<T, V> x, y, nx, ny;
    auto fetch = [&](int t) {
        nx = ld<T, V>(src + (int64_t)t * j.in.ts + c0);
        if (c1 >= 0) ny = ld<T, V>(src + (int64_t)t * j.in.ts + c1);
    };
    int t = st0;
    if (live && t < n) fetch(t);
    fill_table(A, cs, t0, n);
    __syncthreads();
    if (!live) return;
#pragma unroll 1
    for (; t < n; t += A.side) {
        x = nx;
        y = ny;
        if (t + A.side < n) fetch(t + A.side);
        if (turned) {
            float a[V], b[V];
#pragma unroll
            for (int q = 0; q < V; ++q) { a[q] = tof(x.x[q]); b[q] = tof(y.x[q]); }
            turn<V>(a, b, cs + t * A.r.half, V * it, A.r.inter, A.sgn);
#pragma unroll
            for (int q = 0; q < V; ++q) { x.x[q] = fromf<T>(a[q]); y.x[q] = fromf<T>(b[q]); }
        }
        st<T, V>(dst + (int64_t)t * j.out.ts + c0, x);
        if (c1 >= 0) st<T, V>(dst + (int64_t)t * j.out.ts + c1, y);
    }
}

// The gradient of a shared head: an item of a token is summed over the heads by `split` threads (heads s, s + split, ...),
// whose sums meet in shared memory: one thread where there are items enough to fill the SMs, else kSplit.
template <typename T, int V> __device__ void shared_block(const RopeArgs &A, float2 *cs, float *part) {
    const RopeJob &j = A.b;
    const int per = kThreads / A.split;                   // items at a time
    const int rounds = (j.items + per - 1) / per;         // more than one: a token's items take several CTAs
    const int round = (int)((blockIdx.x - A.main_blocks) % rounds);
    const int t0 = (int)((blockIdx.x - A.main_blocks) / rounds) * A.shared_side, n = min(A.shared_side, A.T - t0);
    const int slot = threadIdx.x % per, s = threadIdx.x / per, e = round * per + slot;
    const int t = rounds > 1 ? 0 : e / j.items, it = rounds > 1 ? e : e - t * j.items;
    const bool live = t < n && it < j.items;
    int c0 = 0, c1 = -1;
    const bool turned = item_at<V>(A.r, j, live ? it : 0, c0, c1);
    float a[V], b[V];
#pragma unroll
    for (int q = 0; q < V; ++q) a[q] = b[q] = 0.f;
    if (live) {
        const T *src = reinterpret_cast<const T *>(j.in.p) + (int64_t)(t0 + t) * j.in.ts;
#pragma unroll 4
        for (int h = s; h < j.heads; h += A.split) {
            const Piece<T, V> x = ld<T, V>(src + (int64_t)h * j.in.hs + c0);
            Piece<T, V> y = x;
            if (c1 >= 0) y = ld<T, V>(src + (int64_t)h * j.in.hs + c1);
#pragma unroll
            for (int q = 0; q < V; ++q) {
                a[q] += tof(x.x[q]);
                b[q] += tof(y.x[q]);
            }
        }
    }
    fill_table(A, cs, t0, n);
    __syncthreads();
    if (A.split > 1) {
#pragma unroll
        for (int q = 0; q < V; ++q) {
            part[(2 * q) * kThreads + threadIdx.x] = a[q];
            part[(2 * q + 1) * kThreads + threadIdx.x] = b[q];
        }
        __syncthreads();
        if (s != 0) return;
        for (int k = 1; k < A.split; ++k) {
#pragma unroll
            for (int q = 0; q < V; ++q) {
                a[q] += part[(2 * q) * kThreads + k * per + slot];
                b[q] += part[(2 * q + 1) * kThreads + k * per + slot];
            }
        }
    }
    if (!live) return;
    if (turned) turn<V>(a, b, cs + t * A.r.half, V * it, A.r.inter, A.sgn);
    T *dst = reinterpret_cast<T *>(j.out.p) + (int64_t)(t0 + t) * j.out.ts;
    Piece<T, V> x, y;
#pragma unroll
    for (int q = 0; q < V; ++q) { x.x[q] = fromf<T>(a[q]); y.x[q] = fromf<T>(b[q]); }
    st<T, V>(dst + c0, x);
    if (c1 >= 0) st<T, V>(dst + c1, y);
}

// SHARED: the shared sums' CTAs follow the plain ones in one launch (a kernel of its own: the plain path alone takes half the registers)
template <typename T, int V, bool SHARED> __global__ void __launch_bounds__(kThreads, 4) rope_kernel(const __grid_constant__ RopeArgs A) {
    extern __shared__ float2 cs[];
    if (!SHARED || blockIdx.x < A.main_blocks) plain_block<T, V>(A, cs);
    else if constexpr (SHARED) shared_block<T, V>(A, cs, reinterpret_cast<float *>(cs + A.table));
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
    // Tokens a thread goes through: as many as leave several CTAs for each SM (up to kTokens), and fit the table.
    const int fit = r.half > 0 ? kTable / r.half : 1 << 20;
    auto depth = [&](long long ctas_at_one, int side) {
        long long d = ctas_at_one / (152 * 8);
        d = d < 1 ? 1 : d > kTokens ? kTokens : d;
        while (d > 1 && d * side > fit) --d;
        return (int)d;
    };
    long long main_blocks = 0, shared_blocks = 0;
    int table_tokens = 0;
    if (A.per_token) {
        A.parts = (A.per_token + kThreads - 1) / kThreads;
        A.side = A.parts > 1 ? 1 : kThreads / A.per_token;
        A.side = A.side > fit ? fit : A.side;
        const long long rows = ((long long)T + A.side - 1) / A.side;
        A.tokens = A.side * depth(rows * A.parts, A.side);
        main_blocks = ((long long)T + A.tokens - 1) / A.tokens * A.parts;
        table_tokens = A.tokens;
    }
    if (shared) {
        // one thread an item reads at 16-byte pieces in flight alone from 512 threads an SM on; below, kSplit of them share it
        A.split = (long long)T * A.b.items >= 152 * 512 ? 1 : kSplit;
        const int per = kThreads / A.split, rounds = (A.b.items + per - 1) / per;
        A.shared_side = rounds > 1 ? 1 : per / A.b.items;
        A.shared_side = A.shared_side > fit ? fit : A.shared_side;
        shared_blocks = ((long long)T + A.shared_side - 1) / A.shared_side * rounds;
        table_tokens = table_tokens > A.shared_side ? table_tokens : A.shared_side;
    }
    A.table = r.half * (table_tokens < T ? table_tokens : T);
    const size_t smem = (size_t)A.table * sizeof(float2) + (shared ? (size_t)2 * V * kThreads * sizeof(float) : 0);
    if (main_blocks + shared_blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    if (main_blocks + shared_blocks == 0) return cudaSuccess;      // everything in place and nothing to turn
    A.main_blocks = (unsigned)main_blocks;
    const unsigned grid = (unsigned)(main_blocks + shared_blocks);
    void (*fn)(const RopeArgs);
    if (bf16) fn = V > 1 ? (shared ? rope_kernel<__nv_bfloat16, 8, true> : rope_kernel<__nv_bfloat16, 8, false>)
                         : (shared ? rope_kernel<__nv_bfloat16, 1, true> : rope_kernel<__nv_bfloat16, 1, false>);
    else fn = V > 1 ? (shared ? rope_kernel<float, 4, true> : rope_kernel<float, 4, false>)
                    : (shared ? rope_kernel<float, 1, true> : rope_kernel<float, 1, false>);
    fn<<<grid, kThreads, smem, s>>>(A);
    count_launch();
    return cudaGetLastError();
}

}  // namespace k3kda
