// Paged decode at head dim 256, bf16 caches (a file of its own: compiled in parallel).
#include "paged_decode_launch.cuh"

namespace fa {
cudaError_t launch_paged_decode_h256_bf16(const PagedDecodeArgs& a, int grid, cudaStream_t st) {
  return launch_decode_rows<256, false>(a, grid, st);
}
}  // namespace fa
