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

}  // namespace dp
