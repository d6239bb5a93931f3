// Product with weights held in 4 bits and group scales:
//   out[m, n] = sum_k A[m, k] s[n, k / group] (q[n, k] - z[n, k / group])
//
// Simple form: a warp an output row of W and kRows rows of A; each lane sums
// its k's in fp32.
#include "../operators.h"
#include "values.cuh"

namespace mm {

namespace {

constexpr int kThreads = 256;
constexpr int kRows = 8;

__global__ void __launch_bounds__(kThreads) w4_simple_kernel(const W4Args a) {
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t n = (int64_t)blockIdx.x * (kThreads / 32) + warp;
  if (n >= a.N) return;
  for (int64_t m0 = (int64_t)blockIdx.y * kRows; m0 < a.M; m0 += (int64_t)gridDim.y * kRows) {
    float acc[kRows] = {};
    for (int k = lane; k < a.K; k += 32) {
      const int g = k / a.group;
      const uint8_t b = a.codes[(n * a.ldw + k) / 2];
      const int q = k & 1 ? b >> 4 : b & 15;
      const int z = a.zeros ? a.zeros[n * a.lds + g] & 15 : 8;
      const float w = load_value(a.scales, a.ts, n * a.lds + g) * (float)(q - z);
#pragma unroll
      for (int i = 0; i < kRows; ++i)
        if (m0 + i < a.M) acc[i] += w * load_value(a.A, a.ta, (m0 + i) * a.lda + k);
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      float v = acc[i];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (lane == 0 && m0 + i < a.M) store_value(a.out, a.tc, (m0 + i) * a.ldc + n, v);
    }
  }
}

}  // namespace

mm_status launch_gemm_w4(const W4Args &a, LaunchCtx &ctx) {
  if (a.M > 16 && a.K > 0) return launch_gemm_w4_tiles(a, ctx);
  const int64_t gx = ((int64_t)a.N + kThreads / 32 - 1) / (kThreads / 32);
  const int64_t gy = std::min<int64_t>(((int64_t)a.M + kRows - 1) / kRows, 1024);
  cudaError_t e = launch_pdl(w4_simple_kernel, dim3((unsigned)gx, (unsigned)gy), dim3(kThreads), 0,
                             ctx.stream, dim3(1), a);
  if (e != cudaSuccess) return cuda_error(e, "gemm_w4 launch");
  count_operator_launch();
  return MM_OK;
}

}  // namespace mm
