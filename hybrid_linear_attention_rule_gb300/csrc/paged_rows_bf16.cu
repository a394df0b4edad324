// paged_rows_bf16.cu -- the paged attention's kernels for bf16 pages, 128 query rows at a time.
#include "paged_rows.cuh"

namespace k3kda {
namespace attend {
cudaError_t run_bf16_rows(int dqk, int dv, const Args &A, cudaStream_t s) { return pick_rows<false>(dqk, dv, A, s); }
}  // namespace attend
}  // namespace k3kda
