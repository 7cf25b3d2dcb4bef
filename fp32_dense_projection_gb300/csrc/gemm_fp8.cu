// Instantiations of the promoted GEMM for the 8-bit products with a scale per 128
// contraction elements.
#include "promoted_gemm.cuh"

namespace dp {

// (tile width, kind, form) of every kernel of this file
#define DP_FP8_KERNELS(X) \
  X(128, kFp8KK, kPlain)  \
  X(256, kFp8KK, kPlain)  \
  X(256, kFp8KK, kPair)   \
  X(128, kFp8KK, kSplit)  \
  X(256, kFp8KK, kSplit)  \
  X(128, kFp8KM, kPlain)  \
  X(256, kFp8KM, kPlain)  \
  X(256, kFp8KM, kPair)   \
  X(128, kFp8KM, kSplit)  \
  X(256, kFp8KM, kSplit)  \
  X(128, kFp8MM, kPlain)  \
  X(256, kFp8MM, kPlain)  \
  X(256, kFp8MM, kPair)   \
  X(128, kFp8MM, kSplit)  \
  X(256, kFp8MM, kSplit)

cudaError_t launch_fp8(int kind, int bn, int form, const PgLaunch& l, cudaStream_t stream) {
#define DP_LAUNCH(BN, KIND, FORM) \
  if (bn == BN && kind == KIND && form == FORM) return launch_pg<BN, KIND, FORM>(l, stream);
  DP_FP8_KERNELS(DP_LAUNCH)
#undef DP_LAUNCH
  return cudaErrorInvalidValue;
}

cudaError_t set_attributes_fp8() {
  cudaError_t e = cudaSuccess;
#define DP_SET(BN, KIND, FORM) \
  if (e == cudaSuccess) e = set_attr_pg<BN, KIND, FORM>();
  DP_FP8_KERNELS(DP_SET)
#undef DP_SET
  return e;
}

// Clusters of `split` CTAs of this kernel that run at one time (0 if the query fails).
int max_clusters_fp8(int kind, int bn, int split) {
#define DP_MAX(BN, KIND, FORM) \
  if (FORM == kSplit && bn == BN && kind == KIND) return max_clusters_pg<BN, KIND, FORM>(split);
  DP_FP8_KERNELS(DP_MAX)
#undef DP_MAX
  return 0;
}

}  // namespace dp
