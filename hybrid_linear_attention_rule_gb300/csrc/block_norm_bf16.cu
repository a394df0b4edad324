// block_norm_bf16.cu -- the norms around a block, BF16 arrays; and the weights' gradients joined over the CTAs.
#include "block_norm.cuh"

namespace k3kda {
namespace blk {
namespace {

// dpost and dpre: the CTAs' partial sums, added in a fixed order.  32 columns a CTA, 16 warps each every 16th part.
__global__ void __launch_bounds__(512) join_kernel(const float *parts, int count, int D, float *dpost, float *dpre) {
    __shared__ float meet[16][33];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, c = blockIdx.x * 32 + lane;
    float *out = blockIdx.y ? dpre : dpost;
    if (!out) return;
    parts += (long long)blockIdx.y * count * D;
    float v = 0.f;
    if (c < D)
        for (int p = warp; p < count; p += 16) v += parts[(long long)p * D + c];
    meet[warp][lane] = v;
    __syncthreads();
    if (warp == 0 && c < D) {
        v = 0.f;
        for (int u = 0; u < 16; ++u) v += meet[u][lane];
        out[c] = v;
    }
}

}  // namespace

cudaError_t launch_bf16(const Args &a, bool grad, cudaStream_t s) { return launch_type<__nv_bfloat16>(a, grad, s); }

}  // namespace blk

using namespace blk;

size_t blk_norm_workspace(long long rows, int D) { return (size_t)2 * parts_of(rows, D) * D * sizeof(float); }

cudaError_t launch_blk_norm(const Args &a, int bf16, bool grad, cudaStream_t s) {
    if (a.rows > 0)
        if (cudaError_t e = bf16 ? launch_bf16(a, grad, s) : launch_f32(a, grad, s)) return e;
    if (!grad || (!a.dpost && !a.dpre)) return cudaSuccess;
    join_kernel<<<dim3((a.D + 31) / 32, 2), 512, 0, s>>>(a.parts, parts_of(a.rows, a.D), a.D, a.dpost, a.dpre);
    count_launch();
    return cudaGetLastError();
}

}  // namespace k3kda
