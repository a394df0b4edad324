// paged_attend_bf16_r8.cu -- the paged attention's kernels for bf16 pages, eight query rows at a time.
#include "paged_attend.cuh"

namespace k3kda {
namespace attend {
cudaError_t run_bf16_r8(int dqk, int dv, const Args &A, int max_new, cudaStream_t s) { return pick<false, 2>(dqk, dv, A, max_new, s); }
}  // namespace attend
}  // namespace k3kda
