// Rows of bytes copied to rows that start on 16 bytes, the last 16 bytes of a
// row filled up with zeros: for operands that TMA cannot address in place.
#include <algorithm>

#include "../operators.h"
#include "row_copy.cuh"

namespace mm {

namespace {

__global__ void __launch_bounds__(256) pack_rows_kernel(const PackRows p) {
  pdl_launch_dependents();
  pdl_wait();
  pack_rows(p, (int64_t)blockIdx.x * 256 + threadIdx.x, (int64_t)gridDim.x * 256);
}

mm_status pack(TmaRows &r, uint8_t *dst, int64_t ld16, LaunchCtx &ctx) {
  const PackShape shape = pack_shape(r.rows, ld16, 256, 16 * ctx.dev->info.sms);
  const PackRows p = pack_job(r.p, r.ld, r.rows, r.bytes, dst, ld16, shape.log_threads);
  cudaError_t e = launch_pdl(pack_rows_kernel, dim3((unsigned)shape.blocks), dim3(256), 0, ctx.stream, dim3(1), p);
  if (e != cudaSuccess) return cuda_error(e, "row copy launch");
  count_operator_launch();
  r.p = dst;
  r.ld = ld16;
  return MM_OK;
}

}  // namespace

bool addressable(const TmaRows &r) {
  return (uintptr_t)r.p % 16 == 0 && (r.rows == 1 || (r.ld % 16 == 0 && r.ld < (1LL << 40)));
}

mm_status align_rows(TmaRows &a, TmaRows &b, LaunchCtx &ctx) {
  TmaRows *op[2] = {&a, &b};
  int64_t ld16[2];
  size_t need = 0, at[2];
  for (int i = 0; i < 2; ++i) {
    ld16[i] = (op[i]->bytes + 15) / 16 * 16;
    at[i] = need;
    if (!addressable(*op[i])) need += (size_t)ld16[i] * op[i]->rows;
    else if (op[i]->rows == 1) op[i]->ld = ld16[i];  // a distance that is never used, as maps want it
  }
  if (!need) return MM_OK;
  void *w = nullptr;
  mm_status st = get_scratch(ctx, SCRATCH_REPACK, need, &w);
  if (st != MM_OK) return st;
  for (int i = 0; i < 2; ++i)
    if (!addressable(*op[i]) &&
        (st = pack(*op[i], static_cast<uint8_t *>(w) + at[i], ld16[i], ctx)) != MM_OK)
      return st;
  return MM_OK;
}

mm_status write_zeros(void *out, int64_t ldc, int M, int N, int tc, LaunchCtx &ctx) {
  const size_t es = (size_t)dtype_bytes(tc);
  MM_CUDA_TRY(cudaMemset2DAsync(out, (size_t)ldc * es, 0, (size_t)N * es, (size_t)M, ctx.stream));
  return MM_OK;
}

}  // namespace mm
