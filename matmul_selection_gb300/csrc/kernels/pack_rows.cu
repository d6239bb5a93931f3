// Rows of bytes copied to rows that start on 16 bytes, the last 16 bytes of a
// row filled up with zeros: for operands that TMA cannot address in place.
#include <algorithm>

#include "../operators.h"

namespace mm {

namespace {

// A thread 16 bytes of the copy; a source on any address, read byte by byte
// (neighbouring threads share its sectors).
__global__ void __launch_bounds__(256) pack_rows_kernel(const uint8_t *src, int64_t ld, int64_t rows,
                                                        int64_t bytes, uint8_t *dst, int64_t ld16) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t per = ld16 / 16, total = per * rows;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / per, c = (i - r * per) * 16;
    const uint8_t *s = src + r * ld + c;
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      w[k] = 0;
#pragma unroll
      for (int b = 0; b < 4; ++b)
        if (c + 4 * k + b < bytes) w[k] |= (uint32_t)s[4 * k + b] << (8 * b);
    }
    *reinterpret_cast<uint4 *>(dst + r * ld16 + c) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

mm_status pack(TmaRows &r, uint8_t *dst, int64_t ld16, LaunchCtx &ctx) {
  const int64_t blocks = std::min<int64_t>((ld16 / 16 * r.rows + 255) / 256, 16 * ctx.dev->info.sms);
  cudaError_t e = launch_pdl(pack_rows_kernel, dim3((unsigned)blocks), dim3(256), 0, ctx.stream, dim3(1),
                             static_cast<const uint8_t *>(r.p), r.ld, r.rows, r.bytes, dst, ld16);
  if (e != cudaSuccess) return cuda_error(e, "row copy launch");
  count_operator_launch();
  r.p = dst;
  r.ld = ld16;
  return MM_OK;
}

bool addressable(const TmaRows &r) {
  return (uintptr_t)r.p % 16 == 0 && (r.rows == 1 || (r.ld % 16 == 0 && r.ld < (1LL << 40)));
}

}  // namespace

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
