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

}  // namespace

mm_status launch_pack_rows(const void *src, int64_t ld, int64_t rows, int64_t bytes, void *dst, int64_t ld16,
                           LaunchCtx &ctx) {
  const int64_t blocks = std::min<int64_t>((ld16 / 16 * rows + 255) / 256, 16 * ctx.dev->info.sms);
  cudaError_t e = launch_pdl(pack_rows_kernel, dim3((unsigned)blocks), dim3(256), 0, ctx.stream, dim3(1),
                             static_cast<const uint8_t *>(src), ld, rows, bytes, static_cast<uint8_t *>(dst), ld16);
  if (e != cudaSuccess) return cuda_error(e, "row copy launch");
  count_operator_launch();
  return MM_OK;
}

}  // namespace mm
