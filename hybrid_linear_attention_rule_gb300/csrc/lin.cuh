// lin.cuh -- linear attention with one decay a head: what its kernels share.
//
// Prefill and the three large gradients are one operator on different arrays, a "job".  For every sequence and value head,
// with S [a, b] the state, x, y rows of a channels and z rows of b channels,
//     forward in time    S_t = e^{g_t} S_{t-1} + y_t z_t^T          out_t = x_t S_t
//     backward in time   R_t = y_t z_t^T + e^{g_{t+1}} R_{t+1}      out_t = x_t R_t
// and, with state K^T V and its gradient R = sum_u e^{G_u - G_t} scale q_u do_u^T:
//     o  = job(x = q,  y = k, z = v)            dv = job(x = k, y = q,  z = do) backward in time
//     dq = job(x = do, y = v, z = k)            dk = job(x = v, y = do, z = q)  backward in time
// In chunks, G the sum of g from the chunk's first token on (that token's own included), G_end the whole chunk's:
//     out_i = c_i x_i S + sum_j D_ij (x_i . y_j) z_j,   S' = e^{G_end} S + sum_j w_j y_j z_j^T
// forward: D_ij = e^{G_i - G_j} for j <= i, c_i = e^{G_i}, w_j = e^{G_end - G_j}; backward in time: D_ij = e^{G_j - G_i} for
// j >= i, c_i = e^{G_end - G_i}, w_j = e^{G_j}.  No exponent is positive while g <= 0.
#pragma once

#include "common.cuh"

namespace k3kda {
namespace lin {

// Sums of g are kept as 64-bit integers in units of 2^-32 of a power of two: differences of any two are exact, whatever lies
// between, and the order of the sum does not matter.  One decay counts as at most 4096 powers of two (e^g = 0 in FP32 long
// before: minus infinity is a reset), so a chunk's sum stays within 2^50 units; sums of many chunks stop at 2^62 (`add_units`).
__device__ __forceinline__ long long decay_units(float g) {
    constexpr float kLog2e = 1.442695040888963f, kRest = 1.925963033500e-8f;       // log2(e) and what its FP32 value leaves
    const float p = g * kLog2e;
    if (!(fabsf(p) < 4096.f)) return p != p ? 0 : p < 0.f ? -(4096LL << 32) : 4096LL << 32;
    const float whole = rintf(p), rest = (p - whole) + (fmaf(g, kLog2e, -p) + g * kRest);        // |rest| < 0.51
    return ((long long)(int)whole << 32) + 2LL * __float2int_rn(rest * 2147483648.f);
}
// The sum of a piece's decays and of a chunk's.  It stops at 2^30 powers of two either way, where a plain sum of 2^19 resets would leave 64 bits.
__device__ __forceinline__ long long add_units(long long sum, long long chunk) {
    constexpr long long kMost = 1LL << 62;
    sum += chunk;
    return sum > kMost ? kMost : sum < -kMost ? -kMost : sum;
}
// The sum's whole and remaining powers of two, apart: differences of two such pairs keep an accuracy of 2^-24 however large the sums.
__device__ __forceinline__ float2 two_floats(long long v) {
    return make_float2((float)(int)(v >> 32), (float)(unsigned)v * 2.3283064365386963e-10f);
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float exp2_units(long long v) {
    const float2 f = two_floats(v);
    return ex2(f.x) * ex2(f.y);
}

// Tokens between the anchors at which the gradient of the decays starts its sums anew (see lin_grad.cu).
constexpr int kAnchor = 512;
// Slots of the anchors of sequence n from `first` on: slot + floor(tokens before its end / kAnchor) is never shared, as
// ceil(len / kAnchor) <= floor((start + len) / kAnchor) - floor(start / kAnchor) + 1.
__host__ __device__ inline long long anchor_slot(int start, int n) { return start / kAnchor + (long long)n; }
inline size_t anchor_slots(int N, int T) { return (size_t)(T / kAnchor) + N + 2; }

struct Rows {              // [T, H / share, d]
    const void *p;
    int share;             // value heads that share one head of it
};

struct Job {
    Rows x, y, z;
    int a, b;              // channels of x and y, of z
    int reverse;
    float sp, sc, sw;      // factors on D, on c and on w
    const float *first;    // [slots, H, ...] or null: element (a, b) of a state lies at a * first_sa + b * first_sb
    float *last;           // likewise, or null
    int sa, sb;
    void *out;             // [T, H, b]
    int out_bf16;
    int exact;             // operands of the tensor cores in three parts instead of two (of all jobs of a call if of one)
    // for the gradient of the decays: dots[t, h] = sum_c r[t, c] (out[t, c] without the term j = i), and the states at the anchors
    Rows r;
    float *dots;           // [slices][T, H], or null
    float *anchors;        // [anchor_slots, H] states laid out as first, or null; the state entering the anchor (forward) or leaving it (backward)
    int last_anchor;       // the last state is an anchor too, in its sequence's last slot
};

struct Call {
    Job job[3];
    int jobs;
    int bf16;              // type of x, y, z, r
    const float *g;        // [T, H], or [H] when fixed
    int fixed;
    const int32_t *cu;
    int N, T, H;
    const int32_t *slot;   // of first and last, or null
    int num_slots;
    unsigned *status;
    void *pieces;          // the path's own part of the workspace
};

// The slices of the output's channels that one CTA of the CUDA-core path takes, as wide for all jobs of a call; dots has one row of [T, H] for each.
// 64 channels read less of shared memory for the same products, 32 have shorter steps where the call cannot fill the GPU with pieces of two
// chunks.  (8 heads of 128 channels, with 32 and 64: 8,192 tokens 479 and 336 us, 1,024 tokens 79 and 65, 256 tokens 34 and 42; 32 heads of 2,048
// tokens 495 and 378; gradients of 8 heads of 8,192 tokens 1,515 and 1,097.)
inline int slice_width(int N, int T, int H, int jobs, int most_b) {
    const long long chunks = (long long)T / 32 / N, pieces = chunks < 4 ? 1 : chunks / 2;
    return most_b > 32 && pieces * N * H * jobs * ((most_b + 63) / 64) >= 152 ? 64 : 32;
}
inline int slices(int b, int width) { return (b + width - 1) / width; }

size_t f32_workspace();
cudaError_t launch_scan_f32(const Call &c, cudaStream_t s);
// The tensor-core path (lin_tc.cu): BF16, T > 0; dots has a row for each 32 channels (four, whatever the width).
size_t tc_workspace(int N, int T, int H, int directions);
// Jobs of at most two directions and scales.  `apart`: they are dq, dv and dk, and dk gets a launch of its own.
cudaError_t launch_scan_tc(const Call &c, bool apart, cudaStream_t s);

}  // namespace lin

cudaError_t launch_lin_decode(const void *q, const void *k, const void *v, int bf16, const float *g, int fixed, float *state,
                              const int32_t *slot, int num_slots, int N, int Hk, int H, int dk, int dv, float scale, void *out,
                              int out_bf16, cudaStream_t s);
size_t lin_workspace(int N, int T, int Hk, int H, int dk, int dv, int bf16, int backward);

struct LinArgs {
    const void *q, *k, *v;
    int bf16;
    const float *g;
    int fixed;
    const float *first;
    const int32_t *slot;
    int num_slots;
    const int32_t *cu;
    int N, T, Hk, H, dk, dv;
    float scale;
    void *ws;
};
cudaError_t launch_lin_prefill(const LinArgs &a, void *out, int out_bf16, float *last, cudaStream_t s);
cudaError_t launch_lin_backward(const LinArgs &a, const void *dO, const float *dlast, void *dq, void *dk, void *dv, float *dg,
                                float *dfirst, cudaStream_t s);

}  // namespace k3kda
