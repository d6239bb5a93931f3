// Product of e4m3 operands with row scales:
//   out[m, n] = scale_a[m] scale_b[n] sum_k A[m, k] B[n, k]
//
// Simple form: a warp a row of B and kRows rows of A; each lane sums its k's
// in fp32.
#include "../operators.h"
#include "values.cuh"

namespace mm {

namespace {

constexpr int kThreads = 256;
constexpr int kRows = 8;

__global__ void __launch_bounds__(kThreads) q8_simple_kernel(const Q8Args a) {
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t n = (int64_t)blockIdx.x * (kThreads / 32) + warp;
  if (n >= a.N) return;
  const float sb = a.scale_b && a.K ? a.scale_b[n] : 1.f;
  for (int64_t m0 = (int64_t)blockIdx.y * kRows; m0 < a.M; m0 += (int64_t)gridDim.y * kRows) {
    float acc[kRows] = {};
    for (int k = lane; k < a.K; k += 32) {
      const float w = from_e4m3(a.B[n * a.ldb + k]);
#pragma unroll
      for (int i = 0; i < kRows; ++i)
        if (m0 + i < a.M) acc[i] += w * from_e4m3(a.A[(m0 + i) * a.lda + k]);
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      float v = acc[i];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (lane == 0 && m0 + i < a.M) {
        const float sa = a.scale_a && a.K ? a.scale_a[m0 + i] : 1.f;
        store_value(a.out, a.tc, (m0 + i) * a.ldc + n, v * sa * sb);
      }
    }
  }
}

}  // namespace

mm_status launch_gemm_q8(const Q8Args &a, LaunchCtx &ctx) {
  const int64_t gx = ((int64_t)a.N + kThreads / 32 - 1) / (kThreads / 32);
  const int64_t gy = std::min<int64_t>(((int64_t)a.M + kRows - 1) / kRows, 1024);
  cudaError_t e = launch_pdl(q8_simple_kernel, dim3((unsigned)gx, (unsigned)gy), dim3(kThreads), 0,
                             ctx.stream, dim3(1), a);
  if (e != cudaSuccess) return cuda_error(e, "gemm_q8 launch");
  count_operator_launch();
  return MM_OK;
}

}  // namespace mm
