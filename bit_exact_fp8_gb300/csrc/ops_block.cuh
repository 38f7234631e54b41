// ops_block.cuh -- what the operators of 8-bit layers with block scales share.
#pragma once
#include "ops_common.cuh"

#include <cuda_fp8.h>

namespace emu_ops {

constexpr int kBlock = 128;                              // values that share a scale

template <class T> __device__ __forceinline__ void put(void* out, int64_t i, float v) { static_cast<T*>(out)[i] = from_f<T>(v); }
__device__ __forceinline__ void put(void* out, int type, int64_t i, float v) {
  if (type == EMU_OUT_F32) put<float>(out, i, v);
  else if (type == EMU_OUT_BF16) put<__nv_bfloat16>(out, i, v);
  else put<__half>(out, i, v);
}
// zeros over the elements [from, to) of the output, by `count` threads
__device__ __forceinline__ void put_zeros(void* out, int type, int64_t from, int64_t to, int64_t who, int64_t count) {
  for (int64_t i = from + who; i < to; i += count) put(out, type, i, 0.0f);
}

}  // namespace emu_ops
