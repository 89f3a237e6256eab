// Attention over shared prefixes at head dim 256, e4m3 caches (a file of its own: compiled in parallel).
#include "paged_shared_launch.cuh"

namespace fa {
cudaError_t launch_paged_shared_h256_e4m3(const PagedSharedArgs& a, cudaStream_t st) {
  return launch_shared<256, true>(a, st);
}
}  // namespace fa
