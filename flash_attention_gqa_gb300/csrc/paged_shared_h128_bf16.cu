// Attention over shared prefixes at head dim 128, bf16 caches (a file of its own: compiled in parallel).
#include "paged_shared_launch.cuh"

namespace fa {
cudaError_t launch_paged_shared_h128_bf16(const PagedSharedArgs& a, cudaStream_t st) {
  return launch_shared<128, false>(a, st);
}
}  // namespace fa
