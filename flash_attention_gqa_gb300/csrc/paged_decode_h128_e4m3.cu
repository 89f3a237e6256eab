// Paged decode at head dim 128, e4m3 caches (a file of its own: compiled in parallel).
#include "paged_decode_launch.cuh"

namespace fa {
cudaError_t launch_paged_decode_h128_e4m3(const PagedDecodeArgs& a, int grid, cudaStream_t st) {
  return launch_decode_rows<128, true>(a, grid, st);
}
}  // namespace fa
