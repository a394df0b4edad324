// paged_rows_i4.cu -- the paged attention's kernels for 4-bit pages, 128 query rows at a time.
#include "paged_rows.cuh"

namespace k3kda {
namespace attend {
cudaError_t run_i4_rows(int dqk, int dv, const Args &A, cudaStream_t s) { return pick_rows<true>(dqk, dv, A, s); }
}  // namespace attend
}  // namespace k3kda
