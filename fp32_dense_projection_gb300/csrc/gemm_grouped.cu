// Instantiations of the promoted GEMM for the BF16 products grouped by expert.
#include "promoted_gemm.cuh"

namespace dp {

// (tile width, kind, form) of every kernel of this file
#define DP_GROUPED_KERNELS(X) \
  X(64, kGroupKK, kPlain)     \
  X(128, kGroupKK, kPlain)    \
  X(256, kGroupKK, kPlain)    \
  X(256, kGroupKK, kPair)     \
  X(64, kGroupKM, kPlain)     \
  X(128, kGroupKM, kPlain)    \
  X(256, kGroupKM, kPlain)    \
  X(256, kGroupKM, kPair)     \
  X(64, kGroupMM, kPlain)     \
  X(128, kGroupMM, kPlain)    \
  X(256, kGroupMM, kPlain)

cudaError_t launch_grouped(int kind, int bn, int form, const PgLaunch& l, cudaStream_t stream) {
#define DP_LAUNCH(BN, KIND, FORM) \
  if (bn == BN && kind == KIND && form == FORM) return launch_pg<BN, KIND, FORM>(l, stream);
  DP_GROUPED_KERNELS(DP_LAUNCH)
#undef DP_LAUNCH
  return cudaErrorInvalidValue;
}

cudaError_t set_attributes_grouped() {
  cudaError_t e = cudaSuccess;
#define DP_SET(BN, KIND, FORM) \
  if (e == cudaSuccess) e = set_attr_pg<BN, KIND, FORM>();
  DP_GROUPED_KERNELS(DP_SET)
#undef DP_SET
  return e;
}

}  // namespace dp
