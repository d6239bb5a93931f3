// Internal declarations of the operators around a quantised linear layer:
// what operators.cpp has checked and the kernels take.
#pragma once

#include "common.h"

namespace mm {

// These kernels start while the one before them on the stream still runs (see
// launch_pdl), and that one may write what they read: one's output is the next
// one's operand or scale.  So they read global memory after pdl_wait(), by plain
// loads and TMA; __ldg and ld.global.nc want memory that nothing writes while the
// kernel runs.

struct NormArgs {
  const void *x, *residual, *weight;
  void *h, *y;
  float *scale, *rstd;
  int64_t rows;
  int cols;
  int64_t ldx, ldr, ldh, ldy;  // elements
  int tx, tw, ty;              // mm_dtype, ty also MM_E4M3
  float eps;
};
mm_status launch_rmsnorm(const NormArgs &a, LaunchCtx &ctx);

struct NormBwdArgs {
  const void *dy, *dh, *h, *weight;
  const float *rstd;
  void *dx, *dweight;
  int64_t rows;
  int cols;
  int64_t lddy, lddh, ldh, lddx;  // elements
  int tx, tw, ty;                 // h, dh, dx; weight, dweight; dy
  float eps;
};
mm_status launch_rmsnorm_backward(const NormBwdArgs &a, LaunchCtx &ctx);

struct W4Args {
  const void *A;
  const uint8_t *codes;
  const void *scales;
  const uint8_t *zeros;  // null: 8
  void *out;
  int M, N, K;
  int64_t lda, ldw, lds, ldc;  // elements (codes for ldw)
  int group;
  int ta, ts, tc;
};
mm_status launch_gemm_w4(const W4Args &a, LaunchCtx &ctx);

struct Q8Args {
  const uint8_t *A, *B;
  const float *scale_a, *scale_b;  // null: 1
  void *out;
  int M, N, K;
  int64_t lda, ldb, ldc;
  int tc;
};
mm_status launch_gemm_q8(const Q8Args &a, LaunchCtx &ctx);

// Their forms for at most 16 and at most 8 rows of A (K > 0).
mm_status launch_gemv_w4(const W4Args &a, LaunchCtx &ctx);
mm_status launch_gemv_q8(const Q8Args &a, LaunchCtx &ctx);

// The product over no k.
mm_status write_zeros(void *out, int64_t ldc, int M, int N, int tc, LaunchCtx &ctx);

// Rows that TMA is to read: `rows` rows of `bytes` bytes, ld bytes apart.
struct TmaRows {
  const void *p;
  int64_t ld, rows, bytes;
};
// Operands whose base or distance between rows is not a multiple of 16 bytes
// are copied into the stream's scratch and pointed there.
mm_status align_rows(TmaRows &a, TmaRows &b, LaunchCtx &ctx);

// The operators' error word among the 16 of DeviceState::d_err (the first is
// the GEMM candidates').  A kernel whose bounded wait gives up leaves a code
// there; mm_operator_status reports and clears it.
constexpr int kOperatorErrorWord = 8;

// A kernel's bounded waits: the error word, the limit of a main-loop wait (option
// wait_limit_us), and the test hook (option wait_stall) that makes a kernel first
// wait on a barrier that nothing arrives on.
struct Waits {
  int *err;
  uint64_t limit_ns;
  int stall;
};
inline Waits operator_waits(const LaunchCtx &ctx) {
  const Options &o = get_options();
  return Waits{ctx.dev->d_err + kOperatorErrorWord, (uint64_t)(o.wait_limit_us * 1000.0), o.wait_stall};
}

// A kernel launch of the library outside the candidates, for the counters.
inline void count_operator_launch() { stats().launches.fetch_add(1, std::memory_order_relaxed); }

}  // namespace mm
