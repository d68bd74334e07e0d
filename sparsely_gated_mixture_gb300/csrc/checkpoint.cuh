// Reading the 8-bit checkpoint's values on the device. Internal to libmoe.so.
#pragma once

#include "moe_internal.cuh"

#include <cuda_fp8.h>

namespace moe {

// Two e4m3 bytes as floats.
__device__ __forceinline__ float2 ckpt_e4m3x2(uint32_t v) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)v, __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}
// What a scale byte multiplies by: 2^(byte - 127), NaN for 255.
__device__ __forceinline__ float ckpt_scale(uint32_t byte) {
  return __uint_as_float(byte == 255u ? 0x7fc00000u : byte << 23);
}

}  // namespace moe
