// Root-mean-square norm with the residual's addition, and its gradients.
//
//   h = x + residual, rstd = 1 / sqrt(mean(h^2) + eps), y = h rstd w
//   8-bit output: scale = max|y| / 448, q = e4m3(y / scale)
//   g = dy w, dx = dh + rstd (g - h rstd^2 mean(g h)), dw = sum_rows dy h rstd
//
// Simple forms: a block a row, two passes over it, sums in fp32.
#include "../operators.h"
#include "values.cuh"

namespace mm {

namespace {

constexpr int kThreads = 256;
constexpr float kE4m3Max = 448.f;

// Sum over the block, in every thread.
__device__ float block_sum(float v, float *sh) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) s += sh[w];
  return s;
}

// Largest over the block of the bits of non-negative floats (a NaN's bits are
// above every number's, so a NaN anywhere is the largest).
__device__ uint32_t block_max(uint32_t v, uint32_t *sh) {
  v = __reduce_max_sync(0xffffffffu, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  uint32_t m = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) m = max(m, sh[w]);
  return m;
}

// The scale of an 8-bit row: max|y| / 448, 1 for a row of zeros, and no
// smaller than the least normal float, so that its reciprocal is finite.  A
// NaN stays one.
__device__ __forceinline__ float row_scale(float amax) {
  const float s = amax / kE4m3Max;
  return amax == 0.f ? 1.f : s < 0x1p-126f ? 0x1p-126f : s;
}

__global__ void __launch_bounds__(kThreads) rmsnorm_kernel(const NormArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ float sh[kThreads / 32];
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    float ss = 0.f;
    uint32_t big = 0;  // of |h w|: y is this times rstd
    for (int j = threadIdx.x; j < a.cols; j += kThreads) {
      float h = load_value(a.x, a.tx, r * a.ldx + j);
      if (a.residual) h += load_value(a.residual, a.tx, r * a.ldr + j);
      ss += h * h;
      if (a.scale) big = max(big, __float_as_uint(fabsf(h * load_value(a.weight, a.tw, j))));
    }
    ss = block_sum(ss, sh);
    const float rstd = 1.f / sqrtf(ss / (float)a.cols + a.eps);
    float inv = 1.f;
    if (a.scale) {
      const float amax = __uint_as_float(block_max(big, reinterpret_cast<uint32_t *>(sh))) * rstd;
      const float scale = row_scale(amax);
      inv = 1.f / scale;
      if (threadIdx.x == 0) a.scale[r] = scale;
    }
    if (a.rstd && threadIdx.x == 0) a.rstd[r] = rstd;
    for (int j = threadIdx.x; j < a.cols; j += kThreads) {
      float h = load_value(a.x, a.tx, r * a.ldx + j);
      if (a.residual) h += load_value(a.residual, a.tx, r * a.ldr + j);
      if (a.h) store_value(a.h, a.tx, r * a.ldh + j, h);
      float y = h * rstd * load_value(a.weight, a.tw, j);
      if (a.scale) y *= inv;
      store_value(a.y, a.ty, r * a.ldy + j, y);
    }
  }
}

// 1 / sqrt(mean(h^2) + eps) of each row, where the caller did not keep it.
__global__ void __launch_bounds__(kThreads) rstd_kernel(const NormBwdArgs a, float *rstd) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ float sh[kThreads / 32];
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    float ss = 0.f;
    for (int j = threadIdx.x; j < a.cols; j += kThreads) {
      const float h = load_value(a.h, a.tx, r * a.ldh + j);
      ss += h * h;
    }
    ss = block_sum(ss, sh);
    if (threadIdx.x == 0) rstd[r] = 1.f / sqrtf(ss / (float)a.cols + a.eps);
  }
}

__global__ void __launch_bounds__(kThreads) dweight_kernel(const NormBwdArgs a, const float *rstd) {
  pdl_launch_dependents();
  pdl_wait();
  const int j = blockIdx.x * kThreads + threadIdx.x;
  if (j >= a.cols) return;
  float s = 0.f;
  for (int64_t r = 0; r < a.rows; ++r)
    s += load_value(a.dy, a.ty, r * a.lddy + j) * load_value(a.h, a.tx, r * a.ldh + j) * rstd[r];
  store_value(a.dweight, a.tw, j, s);
}

__global__ void __launch_bounds__(kThreads) dx_kernel(const NormBwdArgs a, const float *rstd) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ float sh[kThreads / 32];
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    float dot = 0.f;
    for (int j = threadIdx.x; j < a.cols; j += kThreads)
      dot += load_value(a.dy, a.ty, r * a.lddy + j) * load_value(a.weight, a.tw, j) *
             load_value(a.h, a.tx, r * a.ldh + j);
    dot = block_sum(dot, sh);
    const float rs = rstd[r], c = dot / (float)a.cols * rs * rs;
    for (int j = threadIdx.x; j < a.cols; j += kThreads) {
      const float g = load_value(a.dy, a.ty, r * a.lddy + j) * load_value(a.weight, a.tw, j);
      float dx = rs * (g - load_value(a.h, a.tx, r * a.ldh + j) * c);
      if (a.dh) dx += load_value(a.dh, a.tx, r * a.lddh + j);
      store_value(a.dx, a.tx, r * a.lddx + j, dx);
    }
  }
}

template <typename K, typename... Args>
mm_status launch(K kern, int64_t blocks, cudaStream_t s, const char *what, Args... args) {
  cudaError_t e = launch_pdl(kern, dim3((unsigned)blocks), dim3(kThreads), 0, s, dim3(1), args...);
  if (e != cudaSuccess) return cuda_error(e, what);
  count_operator_launch();
  return MM_OK;
}

}  // namespace

mm_status launch_rmsnorm(const NormArgs &a, LaunchCtx &ctx) {
  return launch(rmsnorm_kernel, std::min<int64_t>(a.rows, 8 * ctx.dev->info.sms), ctx.stream,
                "rmsnorm launch", a);
}

mm_status launch_rmsnorm_backward(const NormBwdArgs &a, LaunchCtx &ctx) {
  const int64_t blocks = std::max<int64_t>(1, std::min<int64_t>(a.rows, 8 * ctx.dev->info.sms));
  const float *rstd = a.rstd;
  if (!rstd && a.rows > 0) {
    void *w = nullptr;
    mm_status st = get_scratch(*ctx.dev, ctx.stream, SCRATCH_WORKSPACE, a.rows * sizeof(float), &w);
    if (st != MM_OK) return st;
    rstd = static_cast<float *>(w);
    st = launch(rstd_kernel, blocks, ctx.stream, "rmsnorm_backward launch (rstd)", a,
                static_cast<float *>(w));
    if (st != MM_OK) return st;
  }
  if (a.dweight) {
    mm_status st = launch(dweight_kernel, ((int64_t)a.cols + kThreads - 1) / kThreads, ctx.stream,
                          "rmsnorm_backward launch (dweight)", a, rstd);
    if (st != MM_OK) return st;
  }
  if (a.rows == 0) return MM_OK;
  return launch(dx_kernel, blocks, ctx.stream, "rmsnorm_backward launch (dx)", a, rstd);
}

}  // namespace mm
