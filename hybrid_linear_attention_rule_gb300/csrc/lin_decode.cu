// lin_decode.cu -- one token of linear attention with a decay a head for N sequences: S <- e^g S + k v^T in place, o = scale q S.
//
// Roofline: HBM, 8 dk dv bytes a head.  The columns of a state do not need one another, so a CTA takes a slice of them for one
// head: every thread loads all its 16-byte pieces (16 at most) before the first is used, adds its rows' part of the
// update, stores them, and the rows' sums for the output meet in shared memory.  Slices are narrow where heads are few, so
// that every SM has a CTA or two: one sequence of 16 heads is 128 CTAs instead of 16.  256 sequences of 32 heads of 128 x 128 take 171 us, 94 % of
// a plain copy's rate; one of 16 heads 6, a launch's latency.
#include "lin.cuh"

namespace k3kda {
namespace {

constexpr int THREADS = 256, MOST = 16;

struct Args {
    const void *q, *k, *v;
    int bf16;
    const float *g;
    int fixed;
    float *state;
    const int32_t *slot;
    int num_slots, H, group, dk, dv, width, parts;
    float scale;
    void *out;
    int out_bf16;
};

__global__ void __launch_bounds__(THREADS, 2) lin_decode_kernel(const Args A) {
    __shared__ float sq[128], sk[128];
    __shared__ float4 sums[THREADS];
    const int tid = threadIdx.x, part = blockIdx.x % A.parts;
    const long long item = blockIdx.x / A.parts;
    const int n = (int)(item / A.H), h = (int)(item % A.H), col0 = part * A.width;
    const int slot = seq_slot(A.slot, A.num_slots, n);
    if (slot < 0) {
        for (int c = tid; c < A.width; c += THREADS) store_elt(A.out, (size_t)item * A.dv + col0 + c, 0.f, A.out_bf16);
        return;
    }
    const int per = A.width / 4, rows = THREADS / per, r0 = tid / per, c = tid % per;
    float4 *S = reinterpret_cast<float4 *>(A.state + ((size_t)slot * A.H + h) * A.dk * A.dv + col0) + c;
    const int pitch = A.dv / 4;
    const bool on = r0 < rows;
    float4 s[MOST];
#pragma unroll
    for (int i = 0; i < MOST; ++i) {
        const int r = r0 + i * rows;
        if (on && r < A.dk) s[i] = __ldcs(S + (size_t)r * pitch);
    }
    const size_t kh = (size_t)n * (A.H / A.group) + h / A.group;
    for (int i = tid; i < A.dk; i += THREADS) {
        sq[i] = load_elt(A.q, kh * A.dk + i, A.bf16);
        sk[i] = load_elt(A.k, kh * A.dk + i, A.bf16);
    }
    const float e = expf(A.g[A.fixed ? h : item]);
    float v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = load_elt(A.v, (size_t)item * A.dv + col0 + 4 * c + u, A.bf16);
    __syncthreads();
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < MOST; ++i) {
        const int r = r0 + i * rows;
        if (on && r < A.dk) {
            const float k = sk[r], q = sq[r];
            s[i] = make_float4(fmaf(e, s[i].x, k * v[0]), fmaf(e, s[i].y, k * v[1]), fmaf(e, s[i].z, k * v[2]), fmaf(e, s[i].w, k * v[3]));
            __stcs(S + (size_t)r * pitch, s[i]);
            o = make_float4(fmaf(q, s[i].x, o.x), fmaf(q, s[i].y, o.y), fmaf(q, s[i].z, o.z), fmaf(q, s[i].w, o.w));
        }
    }
    sums[tid] = o;
    __syncthreads();
    if (tid < A.width) {
        float t = 0.f;
        for (int r = 0; r < rows; ++r) t += reinterpret_cast<float *>(&sums[r * per + tid / 4])[tid % 4];
        store_elt(A.out, (size_t)item * A.dv + col0 + tid, A.scale * t, A.out_bf16);
    }
}

}  // namespace

cudaError_t launch_lin_decode(const void *q, const void *k, const void *v, int bf16, const float *g, int fixed, float *state,
                              const int32_t *slot, int num_slots, int N, int Hk, int H, int dk, int dv, float scale, void *out,
                              int out_bf16, cudaStream_t s) {
    if (N == 0) return cudaSuccess;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    int parts = 1;
    while (parts < 8 && dv / (2 * parts) >= 16 && dv % (8 * parts) == 0 && (long long)N * H * parts < 2LL * sms) parts *= 2;
    const Args A{q, k, v, bf16, g, fixed, state, slot, num_slots, H, H / Hk, dk, dv, dv / parts, parts, scale, out, out_bf16};
    lin_decode_kernel<<<(unsigned)((long long)N * H * parts), THREADS, 0, s>>>(A);
    count_launch();
    return cudaGetLastError();
}

}  // namespace k3kda
