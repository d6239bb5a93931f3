// Rows of a matrix by token number, and the gradient to the matrix.
//
//   out[t] = scale W[token[t]]
//   dW[v]  = base[v] + scale sum over {t : token[t] = v} of dout[t]
//
// Forward: memory traffic, the rows read and written once.  A power of two of
// threads has a row, each thread up to four 16-byte pieces in flight.
//
// Backward: the places t are sorted by token (stable), so that the rows of one
// token stand together and are added in the order of t, in registers, without
// atomics.  Threads take equal chunks of the sorted places, however often a token
// occurs; a token whose places go past a chunk's end leaves fp32 parts, which a
// second kernel adds in order.
#include <algorithm>

#include "../operators.h"
#include "indices.cuh"
#include "pieces.cuh"

namespace mm {

namespace {

constexpr int kE = 8;  // elements of a piece: 16 bytes of the 16-bit types

// ---------------------------------------------------------------- forward
template <int TW, int TO, bool EDGES>
__global__ void __launch_bounds__(256) embed_kernel(const EmbedArgs a, int log_threads) {
  constexpr int E = EDGES ? 1 : kE;
  pdl_launch_dependents();
  pdl_wait();
  const int threads = 1 << log_threads, t = threadIdx.x & (threads - 1);
  const int64_t r = (int64_t)blockIdx.x * (256 >> log_threads) + (threadIdx.x >> log_threads);
  if (r >= a.rows) return;
  const int64_t token = load_token(a.tokens, a.ti, r, a.vocab);
  const float scale = token < a.vocab ? a.scale : 0.f;  // (zeros, whatever the scale)
  const int step = threads * E;
  for (int j0 = t * E; j0 < a.cols; j0 += 4 * step) {
    float v[4][E];
    const int n = token < a.vocab ? pieces_below<4>(j0, step, a.cols) : 0;
    load_pieces<TW>(a.weight, token * a.ldw + j0, step, n, v);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (j0 + k * step >= a.cols) break;
#pragma unroll
      for (int e = 0; e < E; ++e) v[k][e] *= scale;
      store_piece<TO>(a.out, r * a.ldo + j0 + k * step, v[k]);
    }
  }
}

template <int TW, int TO>
cudaError_t embed_launch(const EmbedArgs &a, LaunchCtx &ctx) {
  const int bw = bytes_of(TW), bo = bytes_of(TO);
  const bool whole = a.cols % kE == 0 && (uintptr_t)a.weight % 16 == 0 && (uintptr_t)a.out % 16 == 0 &&
                     (a.ldw * bw % 16 == 0 || a.vocab <= 1) && (a.ldo * bo % 16 == 0 || a.rows == 1);
  const int64_t pieces = whole ? a.cols / kE : a.cols;
  int log_threads = 0;
  while (log_threads < 8 && (4ll << log_threads) < pieces) ++log_threads;
  const int64_t rows = 256 >> log_threads;
  const dim3 grid((unsigned)((a.rows + rows - 1) / rows));
  return whole ? launch_pdl(embed_kernel<TW, TO, false>, grid, dim3(256), 0, ctx.stream, dim3(1), a, log_threads)
               : launch_pdl(embed_kernel<TW, TO, true>, grid, dim3(256), 0, ctx.stream, dim3(1), a, log_threads);
}

// ---------------------------------------------------------------- sort
// Least significant digit first, 8 bits a pass, by one block: tiles of a key a
// thread; a key's rank among the equal digits of its tile is its warp's, by
// matching, behind those of the warps before.
constexpr int kSortThreads = 1024, kBins = 256;

__global__ void __launch_bounds__(kSortThreads) sort_kernel(const void *tokens, int ti, int64_t vocab, int rows,
                                                            uint2 *to, uint2 *other, int passes) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ uint32_t base[kBins];
  __shared__ uint16_t count[kSortThreads / 32][kBins];
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  uint2 *src = nullptr, *dst = passes & 1 ? to : other;  // the last pass ends in `to`
  for (int pass = 0; pass < passes; ++pass) {
    const auto pair_at = [&](int i) {
      return pass ? src[i] : make_uint2((uint32_t)load_token(tokens, ti, i, vocab), (uint32_t)i);
    };
    const int shift = pass * 8;
    if (t < kBins) base[t] = 0;
    __syncthreads();
    for (int i = t; i < rows; i += kSortThreads) atomicAdd(&base[(pair_at(i).x >> shift) & 255], 1u);
    __syncthreads();
    if (warp == 0) {
      uint32_t before = 0;
      for (int b = lane; b < kBins; b += 32) {
        const uint32_t n = base[b];
        uint32_t sum = n;
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t u = __shfl_up_sync(0xffffffffu, sum, o);
          if (lane >= o) sum += u;
        }
        base[b] = before + sum - n;
        before += __shfl_sync(0xffffffffu, sum, 31);
      }
    }
    for (int i0 = 0; i0 < rows; i0 += kSortThreads) {
      for (int b = lane; b < kBins; b += 32) count[warp][b] = 0;
      __syncthreads();
      const bool have = i0 + t < rows;
      const uint2 p = have ? pair_at(i0 + t) : make_uint2(0, 0);
      const uint32_t d = have ? (p.x >> shift) & 255 : kBins;
      const uint32_t same = __match_any_sync(0xffffffffu, d);
      const int rank = __popc(same & ((1u << lane) - 1));
      if (have && rank == 0) count[warp][d] = (uint16_t)__popc(same);
      __syncthreads();
      if (t < kBins) {
        uint32_t at = 0;
        for (int w = 0; w < kSortThreads / 32; ++w) {
          const uint32_t n = count[w][t];
          count[w][t] = (uint16_t)at;
          at += n;
        }
      }
      __syncthreads();
      if (have) dst[base[d] + count[warp][d] + rank] = p;
      __syncthreads();
      if (have) atomicAdd(&base[d], 1u);
      __syncthreads();
    }
    src = dst;
    dst = dst == to ? other : to;
    __syncthreads();
  }
}

// ---------------------------------------------------------------- sums
struct SumParams {
  EmbedBwdArgs a;
  const uint2 *sorted;  // (token, place)
  float *parts;         // [chunk][2][cols]: a token from the chunk before; one that goes on
  int chunk, chunks;
  int log_threads;
};

template <int TW, int TO, int E>
__device__ __forceinline__ void write_sum(const EmbedBwdArgs &a, int64_t token, int j, float (&sum)[E]) {
  float b[E];
#pragma unroll
  for (int e = 0; e < E; ++e) b[e] = 0.f;
  if (a.base) load_piece<TW>(a.base, token * a.ldb + j, b);
#pragma unroll
  for (int e = 0; e < E; ++e) b[e] = fmaf(a.scale, sum[e], b[e]);
  store_piece<TW>(a.dweight, token * a.lddw + j, b);
}

template <int TW, int TO, int E>
__global__ void __launch_bounds__(256) embed_sum_kernel(const SumParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const EmbedBwdArgs &a = p.a;
  const int threads = 1 << p.log_threads, t = threadIdx.x & (threads - 1);
  const int chunk = (int)blockIdx.x * (256 >> p.log_threads) + (threadIdx.x >> p.log_threads);
  const int j = ((int)blockIdx.y * threads + t) * E;
  if (chunk >= p.chunks || j >= a.cols) return;
  const int rows = (int)a.rows, i0 = chunk * p.chunk, i1 = min(rows, i0 + p.chunk);
  const uint32_t none = (uint32_t)a.vocab;
  float sum[E];
  uint32_t token = p.sorted[i0].x;
  bool from_before = i0 > 0 && p.sorted[i0 - 1].x == token;
  for (int i = i0; i < i1;) {
    if (token == none) return;
    int n = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) sum[e] = 0.f;
    uint32_t next = token;
    for (; i < i1; ++i, ++n) {
      const uint2 s = p.sorted[i];
      next = s.x;
      if (next != token) break;
      float v[E];
      load_piece<TO>(a.dout, (int64_t)s.y * a.lddo + j, v);
#pragma unroll
      for (int e = 0; e < E; ++e) sum[e] += v[e];
    }
    const bool goes_on = i == i1 && i1 < rows && p.sorted[i1].x == token;
    if (from_before || goes_on) {
      float *part = p.parts + ((int64_t)chunk * 2 + (from_before ? 0 : 1)) * a.cols + j;
#pragma unroll
      for (int e = 0; e < E; ++e) part[e] = sum[e];
    } else {
      write_sum<TW, TO, E>(a, token, j, sum);
    }
    from_before = false;
    token = next;
  }
}

// Tokens whose places go past a chunk's end: the chunk where one begins adds the
// parts of the chunks after it, a column a thread.
template <int TW, int TO>
__global__ void __launch_bounds__(256) embed_join_kernel(const SumParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const EmbedBwdArgs &a = p.a;
  const int j = (int)blockIdx.y * 256 + threadIdx.x;
  if (j >= a.cols) return;
  const int rows = (int)a.rows;
  for (int c = (int)blockIdx.x; c + 1 < p.chunks; c += (int)gridDim.x) {
    const int i0 = c * p.chunk, i1 = i0 + p.chunk;
    const uint32_t token = p.sorted[i1].x;
    if (token == (uint32_t)a.vocab) return;
    if (p.sorted[i1 - 1].x != token) continue;                             // none goes past this end
    if (p.sorted[i0].x == token && i0 > 0 && p.sorted[i0 - 1].x == token) continue;  // it began before
    float sum[1] = {p.parts[((int64_t)c * 2 + 1) * a.cols + j]};
    for (int k = c + 1; k < p.chunks && p.sorted[k * p.chunk].x == token; ++k) {
      sum[0] += p.parts[(int64_t)k * 2 * a.cols + j];
      if (p.sorted[min(rows, (k + 1) * p.chunk) - 1].x != token) break;
    }
    write_sum<TW, TO, 1>(a, token, j, sum);
  }
}

template <int TW, int TO>
mm_status embed_sums(const EmbedBwdArgs &a, SumParams p, LaunchCtx &ctx) {
  const int bw = bytes_of(TW), bo = bytes_of(TO);
  const bool whole = a.cols % kE == 0 && (uintptr_t)a.dout % 16 == 0 && (uintptr_t)a.dweight % 16 == 0 &&
                     (uintptr_t)a.base % 16 == 0 && (a.lddo * bo % 16 == 0 || a.rows == 1) &&
                     (a.vocab == 1 || (a.lddw * bw % 16 == 0 && a.ldb * bw % 16 == 0));
  const int64_t pieces = whole ? a.cols / kE : a.cols;
  p.log_threads = 0;
  while (p.log_threads < 8 && (1ll << p.log_threads) < pieces) ++p.log_threads;
  const int64_t groups = 256 >> p.log_threads;
  const dim3 grid((unsigned)((p.chunks + groups - 1) / groups),
                  (unsigned)((pieces + (1 << p.log_threads) - 1) >> p.log_threads));
  cudaError_t e = whole ? launch_pdl(embed_sum_kernel<TW, TO, kE>, grid, dim3(256), 0, ctx.stream, dim3(1), p)
                        : launch_pdl(embed_sum_kernel<TW, TO, 1>, grid, dim3(256), 0, ctx.stream, dim3(1), p);
  if (e != cudaSuccess) return cuda_error(e, "embedding_backward launch");
  count_operator_launch();
  if (p.chunks == 1) return MM_OK;
  const dim3 join((unsigned)std::min(p.chunks, 64), (unsigned)((a.cols + 255) / 256));
  e = launch_pdl(embed_join_kernel<TW, TO>, join, dim3(256), 0, ctx.stream, dim3(1), p);
  if (e != cudaSuccess) return cuda_error(e, "embedding_backward launch (join)");
  count_operator_launch();
  return MM_OK;
}

// f(type of one, type of the other) as constants.
template <typename F>
auto with_type(int t, F &&f) {
  if (t == MM_BF16) return f(std::integral_constant<int, MM_BF16>());
  if (t == MM_F16) return f(std::integral_constant<int, MM_F16>());
  return f(std::integral_constant<int, MM_F32>());
}

}  // namespace

mm_status launch_embedding(const EmbedArgs &a, LaunchCtx &ctx) {
  const cudaError_t e = with_type(a.tw, [&](auto tw) {
    return with_type(a.to, [&](auto to) { return embed_launch<decltype(tw)::value, decltype(to)::value>(a, ctx); });
  });
  if (e != cudaSuccess) return cuda_error(e, "embedding launch");
  count_operator_launch();
  return MM_OK;
}

mm_status launch_embedding_backward(const EmbedBwdArgs &a, LaunchCtx &ctx) {
  const size_t es = (size_t)dtype_bytes(a.tw);
  SumParams p;
  std::memset(&p, 0, sizeof p);
  p.a = a;
  p.chunk = a.rows >= 4096 ? 32 : 8;
  p.chunks = (int)((a.rows + p.chunk - 1) / p.chunk);
  const size_t pairs = ((size_t)a.rows * sizeof(uint2) + 255) / 256 * 256;
  char *w = nullptr;
  if (a.rows > 0) {
    void *s = nullptr;
    mm_status st = get_scratch(ctx, SCRATCH_WORKSPACE, 2 * pairs + (size_t)p.chunks * 2 * a.cols * sizeof(float), &s);
    if (st != MM_OK) return st;
    w = static_cast<char *>(s);
  }
  if (!a.base)
    MM_CUDA_TRY(cudaMemset2DAsync(a.dweight, (size_t)a.lddw * es, 0, (size_t)a.cols * es, (size_t)a.vocab, ctx.stream));
  else if (a.base != a.dweight)
    MM_CUDA_TRY(cudaMemcpy2DAsync(a.dweight, (size_t)a.lddw * es, a.base, (size_t)a.ldb * es, (size_t)a.cols * es,
                                  (size_t)a.vocab, cudaMemcpyDeviceToDevice, ctx.stream));
  if (a.rows == 0) return MM_OK;
  uint2 *sorted = reinterpret_cast<uint2 *>(w), *other = reinterpret_cast<uint2 *>(w + pairs);
  p.sorted = sorted;
  p.parts = reinterpret_cast<float *>(w + 2 * pairs);
  int passes = 1;
  while (passes < 4 && a.vocab >> (8 * passes)) ++passes;
  cudaError_t e = launch_pdl(sort_kernel, dim3(1), dim3(kSortThreads), 0, ctx.stream, dim3(1), a.tokens, a.ti, a.vocab,
                             (int)a.rows, sorted, other, passes);
  if (e != cudaSuccess) return cuda_error(e, "embedding_backward launch (sort)");
  count_operator_launch();
  return with_type(a.tw, [&](auto tw) {
    return with_type(a.to, [&](auto to) { return embed_sums<decltype(tw)::value, decltype(to)::value>(a, p, ctx); });
  });
}

}  // namespace mm
