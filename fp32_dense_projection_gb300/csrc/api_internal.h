// What the translation units of the C ABI share: the current device's state, argument
// checks and tensor-map encoding (defined in dp_api.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "dp_gemm.h"

namespace dp {

constexpr int kMaxDevices = 64;

struct DeviceContext {
  int device = 0;  // below kMaxDevices
  int sm_count = 0;
  uint32_t* fault = nullptr;  // device status word
};

// The current device's context; initialises the device on its first call.
dp_status device_context(DeviceContext* ctx);

// A tuning override's value: `unset` if the variable is absent or the process has no DP_TUNING.
int tuning_override(const char* name, int unset);

bool is_aligned16(const void* p);

// A row-major rows x cols operand with leading dimension *ld (0 = cols).
dp_status check_operand(const void* p, int64_t rows, int64_t cols, int64_t* ld, int esize);

// Tiled tensor map over a matrix [batch][rows][cols] (rank 3) or [rows][cols] (rank 2;
// batch 0): strides in elements, boxes of box_cols x box_rows (x 1), 128-byte swizzle,
// zero fill outside.
bool encode_operand(CUtensorMap* map, const void* ptr, CUtensorMapDataType type, int esize, int64_t rows, int64_t cols,
                    int64_t ld, int64_t batch, int64_t bstride, uint32_t box_cols, uint32_t box_rows);

// Tiled tensor map over rows of row_bytes bytes (packed; a multiple of 16), boxes of 128 bytes x box_rows with 128-byte
// swizzle and zero fill outside; depth > 1 (rows of whole 128 bytes): of that many neighbouring 128-byte
// pieces, [piece][row][128].
bool encode_bytes(CUtensorMap* map, const void* ptr, int64_t rows, int64_t row_bytes, uint32_t box_rows, uint32_t depth);

// Shared memory of the products with 4-bit weights, of layer norm and of the sort by expert (for the current device).
cudaError_t set_attributes_int4();
cudaError_t set_attributes_layer_norm();
cudaError_t set_attributes_experts();

// A launch that may begin while the grid before it on the stream ends (the kernel waits for it by itself).
template <typename... P, typename... A>
dp_status launch_dependent(void (*kernel)(P...), unsigned grid, unsigned block, size_t smem, dp_stream stream, A&&... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid), cfg.blockDim = dim3(block), cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream), cfg.attrs = attr, cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, static_cast<A&&>(args)...) == cudaSuccess) return DP_OK;
  cudaGetLastError();  // (reported here: not once more by the next call that asks)
  return DP_ERR_LAUNCH;
}

}  // namespace dp
