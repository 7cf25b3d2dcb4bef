// Instantiations of the promoted GEMM for the 8-bit products with a scale per 128
// contraction elements.
#include "promoted_gemm.cuh"

namespace dp {

cudaError_t launch_fp8(int kind, int bn, bool pair, const PgLaunch& l, cudaStream_t stream) {
  if (pair) {
    if (bn != 256) return cudaErrorInvalidValue;
    if (kind == kFp8KK) return launch_pg<256, kFp8KK, true>(l, stream);
    if (kind == kFp8KM) return launch_pg<256, kFp8KM, true>(l, stream);
    if (kind == kFp8MM) return launch_pg<256, kFp8MM, true>(l, stream);
    return cudaErrorInvalidValue;
  }
  switch (kind) {
    case kFp8KK:
      if (bn == 64) return launch_pg<64, kFp8KK>(l, stream);
      if (bn == 128) return launch_pg<128, kFp8KK>(l, stream);
      if (bn == 256) return launch_pg<256, kFp8KK>(l, stream);
      break;
    case kFp8KM:
      if (bn == 128) return launch_pg<128, kFp8KM>(l, stream);
      if (bn == 256) return launch_pg<256, kFp8KM>(l, stream);
      break;
    case kFp8MM:
      if (bn == 128) return launch_pg<128, kFp8MM>(l, stream);
      if (bn == 256) return launch_pg<256, kFp8MM>(l, stream);
      break;
  }
  return cudaErrorInvalidValue;
}

cudaError_t set_attributes_fp8() {
  cudaError_t e = set_attr_pg<64, kFp8KK>();
  if (e == cudaSuccess) e = set_attr_pg<128, kFp8KK>();
  if (e == cudaSuccess) e = set_attr_pg<256, kFp8KK>();
  if (e == cudaSuccess) e = set_attr_pg<128, kFp8KM>();
  if (e == cudaSuccess) e = set_attr_pg<256, kFp8KM>();
  if (e == cudaSuccess) e = set_attr_pg<128, kFp8MM>();
  if (e == cudaSuccess) e = set_attr_pg<256, kFp8MM>();
  if (e == cudaSuccess) e = set_attr_pg<256, kFp8KK, true>();
  if (e == cudaSuccess) e = set_attr_pg<256, kFp8KM, true>();
  if (e == cudaSuccess) e = set_attr_pg<256, kFp8MM, true>();
  return e;
}

}  // namespace dp
