// extern "C" entry points of the operators around a quantised linear layer:
// argument checks, then one launch function each (kernels/rmsnorm.cu,
// kernels/gemm_w4.cu, kernels/gemm_q8.cu).
#include "operators.h"

#include <cmath>
#include <exception>

using namespace mm;

namespace {

constexpr int64_t kMaxDim = 1LL << 30;

bool is_float_type(int t) { return t == MM_BF16 || t == MM_F16 || t == MM_F32; }
int type_bytes(int t) { return t == MM_E4M3 ? 1 : dtype_bytes(t); }

// A rows x cols operand with leading dimension ld: ld covers a row, the
// pointer is there and on a multiple of the element size.
mm_status check_rows(const char *name, const void *p, int64_t rows, int64_t cols, int64_t ld, int t) {
  if (!p) return set_error(MM_ERR_INVALID_ARG, "null %s", name);
  if ((uintptr_t)p % type_bytes(t))
    return set_error(MM_ERR_INVALID_ARG, "%s not aligned to its element size", name);
  if (ld < cols)
    return set_error(MM_ERR_INVALID_ARG, "leading dimension of %s too small (%lld for rows of %lld)",
                     name, (long long)ld, (long long)cols);
  if (rows > 1 && ld > (INT64_MAX / 8 - cols) / (rows - 1))
    return set_error(MM_ERR_INVALID_ARG, "%s spans more than the address space", name);
  return MM_OK;
}

mm_status check_vector(const char *name, const void *p, int t) {
  if (!p) return set_error(MM_ERR_INVALID_ARG, "null %s", name);
  if ((uintptr_t)p % type_bytes(t))
    return set_error(MM_ERR_INVALID_ARG, "%s not aligned to its element size", name);
  return MM_OK;
}

mm_status check_eps(float eps) {
  if (!(eps >= 0.f) || std::isinf(eps)) return set_error(MM_ERR_INVALID_ARG, "eps must be finite and >= 0");
  return MM_OK;
}

// The current device's state, refused where the kernels were not built for it.
mm_status operator_context(void *stream, LaunchCtx *ctx) {
  DeviceState *ds = nullptr;
  mm_status st = current_device(&ds);
  if (st != MM_OK) return st;
  if (ds->info.cc_major != 10) return set_error(MM_ERR_UNSUPPORTED, "needs an sm_10x device");
  *ctx = LaunchCtx{static_cast<cudaStream_t>(stream), ds, false};
  return MM_OK;
}

// No C++ exception leaves an entry point (host allocations are the only
// thing here that throws).
template <typename F>
mm_status guarded(F &&f) {
  try {
    return f();
  } catch (const std::exception &e) {
    return set_error(MM_ERR_CUDA, "host exception: %s", e.what());
  } catch (...) {
    return set_error(MM_ERR_CUDA, "host exception");
  }
}

#define MM_TRY(expr)               \
  do {                             \
    mm_status st__ = (expr);       \
    if (st__ != MM_OK) return st__; \
  } while (0)

}  // namespace

extern "C" {

mm_status mm_rmsnorm(const void *x, const void *residual, const void *weight, void *h, void *y,
                     float *scale, float *rstd, int64_t rows, int64_t cols, int64_t ldx,
                     int64_t ldr, int64_t ldh, int64_t ldy, mm_dtypes dt, float eps, void *stream) {
  return guarded([&]() -> mm_status {
    if (rows < 0 || cols < 0) return set_error(MM_ERR_INVALID_ARG, "negative size");
    if (!is_float_type(dt.a) || !is_float_type(dt.b) || !(is_float_type(dt.c) || dt.c == MM_E4M3))
      return set_error(MM_ERR_INVALID_ARG, "types (%d, %d, %d): x and weight bf16, f16 or f32, y also e4m3",
                       dt.a, dt.b, dt.c);
    MM_TRY(check_eps(eps));
    if ((dt.c == MM_E4M3) != (scale != nullptr) && rows > 0 && cols > 0)
      return set_error(MM_ERR_INVALID_ARG, "scale goes with an e4m3 output, and only with it");
    if (rows == 0 || cols == 0) return MM_OK;
    if (cols >= kMaxDim) return set_error(MM_ERR_UNSUPPORTED, "cols too large");
    MM_TRY(check_rows("x", x, rows, cols, ldx, dt.a));
    if (residual) MM_TRY(check_rows("residual", residual, rows, cols, ldr, dt.a));
    MM_TRY(check_vector("weight", weight, dt.b));
    if (h) MM_TRY(check_rows("h", h, rows, cols, ldh, dt.a));
    MM_TRY(check_rows("y", y, rows, cols, ldy, dt.c));
    if (h && h == y) return set_error(MM_ERR_INVALID_ARG, "h and y are the same buffer");
    if (scale) MM_TRY(check_vector("scale", scale, MM_F32));
    if (rstd) MM_TRY(check_vector("rstd", rstd, MM_F32));
    LaunchCtx ctx;
    MM_TRY(operator_context(stream, &ctx));
    NormArgs a{x, residual, weight, h, y, scale, rstd, rows, (int)cols, ldx, ldr, ldh, ldy,
               dt.a, dt.b, dt.c, eps};
    return launch_rmsnorm(a, ctx);
  });
}

mm_status mm_rmsnorm_backward(const void *dy, const void *dh, const void *h, const void *weight,
                              const float *rstd, void *dx, void *dweight, int64_t rows,
                              int64_t cols, int64_t lddy, int64_t lddh, int64_t ldh, int64_t lddx,
                              mm_dtypes dt, float eps, void *stream) {
  return guarded([&]() -> mm_status {
    if (rows < 0 || cols < 0) return set_error(MM_ERR_INVALID_ARG, "negative size");
    if (!is_float_type(dt.a) || !is_float_type(dt.b) || !is_float_type(dt.c))
      return set_error(MM_ERR_INVALID_ARG, "types (%d, %d, %d): bf16, f16 or f32", dt.a, dt.b, dt.c);
    MM_TRY(check_eps(eps));
    if (cols == 0) return MM_OK;
    if (cols >= kMaxDim) return set_error(MM_ERR_UNSUPPORTED, "cols too large");
    if (dweight) MM_TRY(check_vector("dweight", dweight, dt.b));
    if (rows > 0) {
      MM_TRY(check_rows("dy", dy, rows, cols, lddy, dt.c));
      if (dh) MM_TRY(check_rows("dh", dh, rows, cols, lddh, dt.a));
      MM_TRY(check_rows("h", h, rows, cols, ldh, dt.a));
      MM_TRY(check_vector("weight", weight, dt.b));
      MM_TRY(check_rows("dx", dx, rows, cols, lddx, dt.a));
      if (dx == h) return set_error(MM_ERR_INVALID_ARG, "dx may not be h in place");
      if (rstd) MM_TRY(check_vector("rstd", rstd, MM_F32));
    } else if (!dweight) {
      return MM_OK;
    }
    LaunchCtx ctx;
    MM_TRY(operator_context(stream, &ctx));
    NormBwdArgs a{dy, dh, h, weight, rstd, dx, dweight, rows, (int)cols, lddy, lddh, ldh, lddx,
                  dt.a, dt.b, dt.c, eps};
    return launch_rmsnorm_backward(a, ctx);
  });
}

mm_status mm_gemm_w4(const void *A, const void *codes, const void *scales, const void *zeros,
                     void *out, int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldw,
                     int64_t lds, int64_t ldc, int32_t group, mm_dtypes dt, void *stream) {
  return guarded([&]() -> mm_status {
    if (M < 0 || N < 0 || K < 0) return set_error(MM_ERR_INVALID_ARG, "negative size");
    if (dt.a != MM_BF16 && dt.a != MM_F16)
      return set_error(MM_ERR_INVALID_ARG, "A's type %d: bf16 or f16", dt.a);
    if (!is_float_type(dt.b) || !is_float_type(dt.c))
      return set_error(MM_ERR_INVALID_ARG, "types of scales and out (%d, %d): bf16, f16 or f32", dt.b, dt.c);
    if (group != 32 && group != 64 && group != 128)
      return set_error(MM_ERR_INVALID_ARG, "group %d: 32, 64 or 128", (int)group);
    if (ldw % 2) return set_error(MM_ERR_INVALID_ARG, "ldw %lld: rows of codes start on whole bytes", (long long)ldw);
    if (M == 0 || N == 0) return MM_OK;
    if (M >= kMaxDim || N >= kMaxDim || K >= kMaxDim) return set_error(MM_ERR_UNSUPPORTED, "size too large");
    MM_TRY(check_rows("out", out, M, N, ldc, dt.c));
    if (K > 0) {
      MM_TRY(check_rows("A", A, M, K, lda, dt.a));
      MM_TRY(check_rows("codes", codes, N, K, ldw, MM_E4M3));
      MM_TRY(check_rows("scales", scales, N, (K + group - 1) / group, lds, dt.b));
    }
    LaunchCtx ctx;
    MM_TRY(operator_context(stream, &ctx));
    W4Args a{A, static_cast<const uint8_t *>(codes), scales, static_cast<const uint8_t *>(zeros), out,
             (int)M, (int)N, (int)K, lda, ldw, lds, ldc, group, dt.a, dt.b, dt.c};
    return launch_gemm_w4(a, ctx);
  });
}

mm_status mm_gemm_q8(const void *A, const void *B, const float *scale_a, const float *scale_b,
                     void *out, int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldb,
                     int64_t ldc, mm_dtypes dt, void *stream) {
  return guarded([&]() -> mm_status {
    if (M < 0 || N < 0 || K < 0) return set_error(MM_ERR_INVALID_ARG, "negative size");
    if (dt.a != MM_E4M3 || dt.b != MM_E4M3 || !is_float_type(dt.c))
      return set_error(MM_ERR_INVALID_ARG, "types (%d, %d, %d): A and B e4m3, out bf16, f16 or f32", dt.a,
                       dt.b, dt.c);
    if (M == 0 || N == 0) return MM_OK;
    if (M >= kMaxDim || N >= kMaxDim || K >= kMaxDim) return set_error(MM_ERR_UNSUPPORTED, "size too large");
    MM_TRY(check_rows("out", out, M, N, ldc, dt.c));
    if (K > 0) {
      MM_TRY(check_rows("A", A, M, K, lda, MM_E4M3));
      MM_TRY(check_rows("B", B, N, K, ldb, MM_E4M3));
    }
    if (scale_a) MM_TRY(check_vector("scale_a", scale_a, MM_F32));
    if (scale_b) MM_TRY(check_vector("scale_b", scale_b, MM_F32));
    LaunchCtx ctx;
    MM_TRY(operator_context(stream, &ctx));
    Q8Args a{static_cast<const uint8_t *>(A), static_cast<const uint8_t *>(B), scale_a, scale_b, out,
             (int)M, (int)N, (int)K, lda, ldb, ldc, dt.c};
    return launch_gemm_q8(a, ctx);
  });
}

mm_status mm_operator_status(void *stream) {
  return guarded([&]() -> mm_status {
    LaunchCtx ctx;
    MM_TRY(operator_context(stream, &ctx));
    MM_CUDA_TRY(cudaStreamSynchronize(ctx.stream));
    int code = 0, *word = ctx.dev->d_err + kOperatorErrorWord;
    MM_CUDA_TRY(cudaMemcpy(&code, word, sizeof code, cudaMemcpyDeviceToHost));
    if (code == 0) return MM_OK;
    MM_CUDA_TRY(cudaMemset(word, 0, sizeof code));
    return set_error(MM_ERR_TIMEOUT,
                     "an operator kernel's bounded wait gave up (code 0x%x); results of the calls "
                     "since the previous status query may be wrong", code);
  });
}

}  // extern "C"
