// Element access by mm_dtype for the operator kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "../common.h"

namespace mm {

__device__ __forceinline__ float load_value(const void *p, int t, int64_t i) {
  if (t == MM_F32) return static_cast<const float *>(p)[i];
  if (t == MM_BF16) return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
  return __half2float(static_cast<const __half *>(p)[i]);
}

// e4m3, nearest even, saturating at +-448; NaN stays NaN.
__device__ __forceinline__ uint8_t to_e4m3(float v) {
  return (uint8_t)__nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float from_e4m3(uint8_t v) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)v, __NV_E4M3)));
}

__device__ __forceinline__ void store_value(void *p, int t, int64_t i, float v) {
  if (t == MM_F32)
    static_cast<float *>(p)[i] = v;
  else if (t == MM_BF16)
    static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
  else if (t == MM_F16)
    static_cast<__half *>(p)[i] = __float2half_rn(v);
  else
    static_cast<uint8_t *>(p)[i] = to_e4m3(v);
}

// Four values of a row from element i on, `step` apart, those below `left`
// elements from i: one store where step is 1 (a 16-byte aligned row).
template <int STEP>
__device__ __forceinline__ void store_four(void *p, int t, int64_t i, float4 v, int left) {
  if (STEP == 1 && left >= 4) {
    if (t == MM_F32) {
      *reinterpret_cast<float4 *>(static_cast<float *>(p) + i) = v;
    } else if (t == MM_BF16) {
      const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
      *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p) + i) =
          make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    } else {
      const __half2 a = __floats2half2_rn(v.x, v.y), b = __floats2half2_rn(v.z, v.w);
      *reinterpret_cast<uint2 *>(static_cast<__half *>(p) + i) =
          make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    }
    return;
  }
  const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (k * STEP < left) store_value(p, t, i + k * STEP, x[k]);
}

}  // namespace mm
