// Internal declarations of the operators (those around a quantised linear layer
// and those at the ends of a language model): what operators.cpp has checked and
// the kernels take.
#pragma once

#include "common.h"
#include "embed_chunks.h"

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

struct EmbedArgs {
  const void *weight, *tokens;
  void *out;
  int64_t rows;
  int cols;
  int64_t vocab, ldw, ldo;
  int tw, ti, to;  // ti: MM_I32 or MM_I64
  float scale;
};
mm_status launch_embedding(const EmbedArgs &a, LaunchCtx &ctx);

struct EmbedBwdArgs {
  const void *dout, *tokens, *base;  // base null: none
  void *dweight;
  int64_t rows;
  int cols;
  int64_t vocab, lddo, ldb, lddw;
  int tw, ti, to;  // dweight and base; tokens; dout
  float scale;
};
mm_status launch_embedding_backward(const EmbedBwdArgs &a, LaunchCtx &ctx);

// The places 0 .. rows - 1 of tokens in the order of their keys, equal ones in their own:
// (key, place) as two 32-bit numbers each to `to`; `other`: room for as many.  A key is a
// token without its `drop` low bits; no token has the key keys_of(vocab, drop).
MM_HOST_DEVICE int64_t keys_of(int64_t vocab, int drop) { return (vocab + (1 << drop) - 1) >> drop; }
struct SortArgs {
  const void *tokens;
  int ti;
  int64_t vocab;
  int rows, drop;
  void *to, *other;
};
mm_status sort_ready(LaunchCtx &ctx);  // what a launch needs set up, which may fail
mm_status sort_tokens(const SortArgs &a, LaunchCtx &ctx);

// The loss over a vocabulary and its gradients (those: dloss or null for 1, dx
// and dweight, either null).
struct LossArgs {
  const void *x, *weight, *targets;
  float *loss, *lse;
  int rows, cols, vocab;
  int64_t ldx, ldw;
  int tx, ti;
  const float *dloss;
  void *dx, *dweight;
  int64_t lddx, lddw;
};
mm_status launch_cross_entropy(const LossArgs &a, LaunchCtx &ctx);
mm_status launch_cross_entropy_backward(const LossArgs &a, LaunchCtx &ctx);

// The product over no k.
mm_status write_zeros(void *out, int64_t ldc, int M, int N, int tc, LaunchCtx &ctx);

// Rows that TMA is to read: `rows` rows of `bytes` bytes, ld bytes apart.
struct TmaRows {
  const void *p;
  int64_t ld, rows, bytes;
};
// Whether TMA reads them as they lie.
bool addressable(const TmaRows &r);
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
