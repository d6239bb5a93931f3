// What the kernels of products with 4-bit weights share.
#pragma once

#include "../operators.h"
#include "values.cuh"

namespace mm {

struct W4Scales {
  const void *s;
  const uint8_t *z;  // null: 8
  int64_t lds;
  int N, K, ts, group_shift, groups;
};
inline W4Scales w4_scales(const W4Args &a) {
  return W4Scales{a.scales, a.zeros, a.lds, a.N, a.K, a.ts, a.group == 32 ? 5 : a.group == 64 ? 6 : 7,
                  (a.K + a.group - 1) / a.group};
}

// A's 16-bit type, two to a register.
template <int TA>
struct Pair16 {
  using T = __nv_bfloat162;
  static __device__ __forceinline__ T both(float v) { return __float2bfloat162_rn(v); }
};
template <>
struct Pair16<MM_F16> {
  using T = __half2;
  static __device__ __forceinline__ T both(float v) { return __float2half2_rn(v); }
};
template <typename T>
__device__ __forceinline__ T bits_as(uint32_t v) {
  return *reinterpret_cast<const T *>(&v);
}
template <typename T>
__device__ __forceinline__ uint32_t as_bits(const T &v) {
  return *reinterpret_cast<const uint32_t *>(&v);
}

// A row's scales and zero points: where they start, and how many there are (0
// past the last row).
struct ScaleRow {
  const char *s;
  const uint8_t *z;
  int groups;
};
__device__ __forceinline__ ScaleRow scale_row(const W4Scales &p, int n) {
  const bool in = n < p.N;
  const int64_t at = in ? (int64_t)n * p.lds : 0;
  return ScaleRow{static_cast<const char *>(p.s) + at * (p.ts == MM_F32 ? 4 : 2),
                  p.z ? p.z + at : nullptr, in ? p.groups : 0};
}
// A scale and a zero point as they lie in memory, loaded a stage of codes ahead.
struct RawScale {
  uint32_t s, z;
};
__device__ __forceinline__ RawScale load_raw_scale(const W4Scales &p, const ScaleRow &row, int k) {
  RawScale r{0u, 8u};
  const int g = k >> p.group_shift;
  if (g < row.groups) {
    r.s = p.ts == MM_F32 ? reinterpret_cast<const uint32_t *>(row.s)[g]
                         : (uint32_t)reinterpret_cast<const uint16_t *>(row.s)[g];
    if (row.z) r.z = row.z[g];
  }
  return r;
}

__device__ __forceinline__ float raw_scale_value(const W4Scales &p, const RawScale &r) {
  return p.ts == MM_F32    ? __uint_as_float(r.s)
         : p.ts == MM_BF16 ? __uint_as_float(r.s << 16)
                           : __half2float(__ushort_as_half((unsigned short)r.s));
}

}  // namespace mm
