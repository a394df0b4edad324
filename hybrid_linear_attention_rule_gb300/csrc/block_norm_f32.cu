// block_norm_f32.cu -- the norms around a block, FP32 arrays.
#include "block_norm.cuh"

namespace k3kda {
namespace blk {

cudaError_t launch_f32(const Args &a, bool grad, cudaStream_t s) { return launch_type<float>(a, grad, s); }

}  // namespace blk
}  // namespace k3kda
