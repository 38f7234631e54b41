// ops_block.cuh -- what the operators of 8-bit layers with block scales share.
#pragma once
#include "ops_common.cuh"

#include <cuda_fp8.h>

namespace emu_ops {

constexpr int kBlock = 128;                              // values that share a scale

// one code's value; every FP8 value is exact in fp16
__device__ __forceinline__ float code_value(uint8_t code, int fmt) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(code, fmt == EMU_E4M3FN ? __NV_E4M3 : __NV_E5M2)));
}

}  // namespace emu_ops
