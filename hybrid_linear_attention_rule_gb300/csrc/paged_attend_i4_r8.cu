// paged_attend_i4_r8.cu -- the paged attention's kernels for 4-bit pages, eight query rows at a time.
#include "paged_attend.cuh"

namespace k3kda {
namespace attend {
cudaError_t run_i4_r8(int dqk, int dv, const Args &A, int max_new, cudaStream_t s) { return pick<true, 2>(dqk, dv, A, max_new, s); }
}  // namespace attend
}  // namespace k3kda
