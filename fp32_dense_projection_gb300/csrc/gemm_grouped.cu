// Instantiations of the promoted GEMM for the BF16 products grouped by expert.
#include "promoted_gemm.cuh"

namespace dp {

cudaError_t launch_grouped(int kind, int bn, const PgLaunch& l, cudaStream_t stream) {
#define DP_GROUPED(KIND)                                       \
  case KIND:                                                   \
    if (bn == 64) return launch_pg<64, KIND>(l, stream);       \
    if (bn == 128) return launch_pg<128, KIND>(l, stream);     \
    if (bn == 256) return launch_pg<256, KIND>(l, stream);     \
    break;
  switch (kind) {
    DP_GROUPED(kGroupKK)
    DP_GROUPED(kGroupKM)
    DP_GROUPED(kGroupMM)
  }
#undef DP_GROUPED
  return cudaErrorInvalidValue;
}

cudaError_t set_attributes_grouped() {
  cudaError_t e = cudaSuccess;
#define DP_GROUPED(KIND)                                \
  if (e == cudaSuccess) e = set_attr_pg<64, KIND>();    \
  if (e == cudaSuccess) e = set_attr_pg<128, KIND>();   \
  if (e == cudaSuccess) e = set_attr_pg<256, KIND>();
  DP_GROUPED(kGroupKK)
  DP_GROUPED(kGroupKM)
  DP_GROUPED(kGroupMM)
#undef DP_GROUPED
  return e;
}

}  // namespace dp
