// Softmax cross entropy of x projected on a vocabulary, and its gradients.
//
//   l[t, v] = sum_c x[t, c] W[v, c];  lse[t] = log sum_v exp l[t, v]
//   loss[t] = lse[t] - l[t, y[t]]
//   g[t, v] = dloss[t] (exp(l[t, v] - lse[t]) - [v = y[t]]);  dx = g W, dW = g^T x
//
// Forward: a product whose tiles never leave the SM: a tile's rows leave their
// maximum and sum of exponentials, and the target's logit.  The sums are kept as
// s 2^r, r a whole number not below the logits times log2(e): the powers of two
// that bring two sums together are exact.
// Backward: the vocabulary in pieces, each the product again with g as the
// epilogue's output in 16 bits, then its two products.
// Rows without a target are left out: the others' x is gathered first, so the
// products run over whole tiles of rows that count, and what a padded row holds
// is never read.
#include <algorithm>

#include "../operators.h"
#include "indices.cuh"
#include "tcgen05.cuh"
#include "values.cuh"

namespace mm {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kRowTile = 256;
// g in f16 lies in [-1, 1] times this: f16's smallest normal number is 2^-14, and
// most probabilities over a large vocabulary are below it.
constexpr float kF16Gain = 16384.f;

__device__ __forceinline__ float exp2_fast(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// ---------------------------------------------------------------- the rows that count
// Where each call's scratch holds what; i: a row among those that count, of
// `rows_pad`, a multiple of 256.
struct Rows {
  int *count;       // [0] the rows that count
  float *gain;      // largest |dloss|
  int *slot;        // [rows] i of a row, or -1
  int *target;      // [rows_pad], -1 past the count
  float *ratio;     // [rows_pad] dloss / gain (f16: times kF16Gain), 0 past the count
  float *lse2;      // [rows_pad] lse log2(e)
  uint16_t *x;      // [rows_pad][ldx], zeros from cols to ldx and for rows up to a multiple of 64
  int64_t ldx;
  int rows_pad;
};

struct GatherParams {
  LossArgs a;
  Rows r;
  int backward;
};

__device__ __forceinline__ int valid_target(const LossArgs &a, int64_t t) {
  const int64_t v = load_token(a.targets, a.ti, t, a.vocab);
  return v < a.vocab ? (int)v : -1;
}

// Each block has an equal share of the rows and counts the rows that count
// before its own.
constexpr int kGatherThreads = 256;
__global__ void __launch_bounds__(kGatherThreads) gather_kernel(const GatherParams p) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ int warp_count[kGatherThreads / 32];
  __shared__ float warp_max[kGatherThreads / 32];
  __shared__ int at_row[kGatherThreads];  // the source row of slot first + k
  const LossArgs &a = p.a;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int r0 = (int)((int64_t)a.rows * blockIdx.x / gridDim.x);
  const int r1 = (int)((int64_t)a.rows * (blockIdx.x + 1) / gridDim.x);
  int before = 0;
  float top = 0.f;  // of the finite ones
  const int look = p.backward ? a.rows : r0;
  for (int i = t; i < look; i += kGatherThreads)
    if (valid_target(a, i) >= 0) {
      before += i < r0;
      if (p.backward) {
        const float d = a.dloss ? fabsf(a.dloss[i]) : 1.f;
        if (d <= 3.402823466e38f) top = fmaxf(top, d);
      }
    }
  before = __reduce_add_sync(0xffffffffu, before);
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) warp_count[warp] = before, warp_max[warp] = top;
  __syncthreads();
  before = 0;
  for (int w = 0; w < kGatherThreads / 32; ++w) before += warp_count[w], top = fmaxf(top, warp_max[w]);
  if (top == 0.f) top = 1.f;
  __syncthreads();

  const int pieces = (int)(p.r.ldx / 8);
  const uint16_t *x = static_cast<const uint16_t *>(a.x);
  const bool whole = (uintptr_t)x % 16 == 0 && a.ldx % 8 == 0;
  for (int g0 = r0; g0 < r1; g0 += kGatherThreads) {
    const int i = g0 + t, target = i < r1 ? valid_target(a, i) : -1;
    const uint32_t mask = __ballot_sync(0xffffffffu, target >= 0);
    if (lane == 0) warp_count[warp] = __popc(mask);
    __syncthreads();
    int at = __popc(mask & ((1u << lane) - 1)), total = 0;
    for (int w = 0; w < kGatherThreads / 32; ++w) {
      if (w < warp) at += warp_count[w];
      total += warp_count[w];
    }
    if (i < r1) p.r.slot[i] = target >= 0 ? before + at : -1;
    if (target >= 0) {
      at_row[at] = i;
      p.r.target[before + at] = target;
      if (p.backward) {
        const float d = a.dloss ? a.dloss[i] : 1.f;
        p.r.ratio[before + at] = d / top * (a.tx == MM_F16 ? kF16Gain : 1.f);
        p.r.lse2[before + at] = a.lse[i] * kLog2e;
      }
    }
    __syncthreads();
    for (int k = warp; k < total; k += kGatherThreads / 32) {
      const uint16_t *from = x + (int64_t)at_row[k] * a.ldx;
      uint16_t *to = p.r.x + (int64_t)(before + k) * p.r.ldx;
      for (int c = lane; c < pieces; c += 32) {
        uint4 v;
        if (whole && c * 8 + 8 <= a.cols) {
          v = reinterpret_cast<const uint4 *>(from)[c];
        } else {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = c * 8 + 2 * e;
            w[e] = (j < a.cols ? from[j] : 0u) | (j + 1 < a.cols ? (uint32_t)from[j + 1] << 16 : 0u);
          }
          v = make_uint4(w[0], w[1], w[2], w[3]);
        }
        reinterpret_cast<uint4 *>(to)[c] = v;
      }
    }
    before += total;
    __syncthreads();
  }
  if (blockIdx.x == gridDim.x - 1) {
    if (t == 0) *p.r.count = before, *p.r.gain = top;
    const int end = max(1, (before + kRowTile - 1) / kRowTile) * kRowTile;
    for (int i = before + t; i < end; i += kGatherThreads) {
      p.r.target[i] = -1;
      if (p.backward) p.r.ratio[i] = p.r.lse2[i] = 0.f;
    }
    const int64_t z0 = (int64_t)before * pieces, z1 = (int64_t)max(1, (before + 63) / 64) * 64 * pieces;
    for (int64_t i = z0 + t; i < z1; i += kGatherThreads)
      reinterpret_cast<uint4 *>(p.r.x)[i] = make_uint4(0, 0, 0, 0);
  }
}

// ---------------------------------------------------------------- the products
enum Mode { MODE_LSE, MODE_G, MODE_DX, MODE_DW };

struct TileParams {
  Rows r;
  const uint16_t *W;
  int64_t ldw;
  int cols, vocab;
  int v0, width;     // the piece of the vocabulary: its first token, how many (G: padded to 64)
  int tx;
  float2 *part;      // LSE: [tile of the vocabulary][rows_pad] (r, s)
  float *hit;        // LSE: [rows_pad] the target's logit
  uint16_t *g;       // [rows_pad][ldg]
  int64_t ldg;
  float *acc;        // DX: [rows_pad][ldacc]
  int64_t ldacc;
  int first;         // DX: the first piece
  uint16_t *dw;
  int64_t lddw;
};

__device__ __forceinline__ float value16(const uint16_t *p, int t, int64_t i) {
  return t == MM_BF16 ? __bfloat162float(__ushort_as_bfloat16(p[i])) : __half2float(__ushort_as_half(p[i]));
}
__device__ __forceinline__ uint16_t bits16(int t, float v) {
  return t == MM_BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v)) : __half_as_ushort(__float2half_rn(v));
}

// 64 x 64 of a product, 4 x 4 a thread.
template <int MODE>
__global__ void __launch_bounds__(256) tile_kernel(const TileParams p) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ float sa[16][65], sb[16][65];
  const int count = *p.r.count, rows = max(1, (count + 63) / 64) * 64;
  const int m0 = (int)blockIdx.y * 64, n0 = (int)blockIdx.x * 64, t = threadIdx.x;
  const int tm = t >> 4, tn = t & 15;
  constexpr bool kLogits = MODE == MODE_LSE || MODE == MODE_G;
  const int M = MODE == MODE_DW ? p.width : rows;
  const int K = kLogits ? p.cols : MODE == MODE_DX ? p.width : rows;
  if (m0 >= M) return;
  const auto A = [&](int m, int k) -> float {
    if (m >= M || k >= K) return 0.f;
    if (kLogits) return value16(p.r.x, p.tx, (int64_t)m * p.r.ldx + k);
    if (MODE == MODE_DX) return value16(p.g, p.tx, (int64_t)m * p.ldg + k);
    return value16(p.g, p.tx, (int64_t)k * p.ldg + m);
  };
  const auto B = [&](int n, int k) -> float {
    if (k >= K) return 0.f;
    if (kLogits) return p.v0 + n < p.vocab ? value16(p.W, p.tx, (int64_t)(p.v0 + n) * p.ldw + k) : 0.f;
    if (n >= p.cols) return 0.f;
    if (MODE == MODE_DX) return p.v0 + k < p.vocab ? value16(p.W, p.tx, (int64_t)(p.v0 + k) * p.ldw + n) : 0.f;
    return value16(p.r.x, p.tx, (int64_t)k * p.r.ldx + n);
  };
  float acc[4][4] = {};
  for (int k0 = 0; k0 < K; k0 += 16) {
    for (int i = t; i < 1024; i += 256) {
      // neighbouring threads along what is contiguous in memory
      const int am = MODE == MODE_DW ? i & 63 : i >> 4, ak = MODE == MODE_DW ? i >> 6 : i & 15;
      sa[ak][am] = A(m0 + am, k0 + ak);
      const int bn = kLogits ? i >> 4 : i & 63, bk = kLogits ? i & 15 : i >> 6;
      sb[bk][bn] = B(n0 + bn, k0 + bk);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 16; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] += sa[k][tm * 4 + i] * sb[k][tn * 4 + j];
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int m = m0 + tm * 4 + i;
    if constexpr (kLogits) {
      const int target = p.r.target[m];
      if constexpr (MODE == MODE_LSE) {
        float top = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (n0 + tn * 4 + j < p.vocab) top = fmaxf(top, acc[i][j]);
        for (int o = 1; o < 16; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float r = top == -INFINITY ? 0.f : ceilf(top * kLog2e);
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int n = n0 + tn * 4 + j;
          if (n < p.vocab) s += exp2_fast(fmaf(acc[i][j], kLog2e, -r));
          if (n == target) p.hit[m] = acc[i][j];
        }
        for (int o = 1; o < 16; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (tn == 0) p.part[(int64_t)blockIdx.x * p.r.rows_pad + m] = make_float2(r, s);
      } else {
        const float ratio = p.r.ratio[m], lse2 = p.r.lse2[m];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int n = n0 + tn * 4 + j;
          if (n >= p.width) continue;
          float g = 0.f;
          if (target >= 0 && p.v0 + n < p.vocab)
            g = ratio * (exp2_fast(fmaf(acc[i][j], kLog2e, -lse2)) - (p.v0 + n == target ? 1.f : 0.f));
          p.g[(int64_t)m * p.ldg + n] = bits16(p.tx, g);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = n0 + tn * 4 + j;
        if (n >= p.cols) continue;
        if constexpr (MODE == MODE_DX) {
          float *to = p.acc + (int64_t)m * p.ldacc + n;
          *to = p.first ? acc[i][j] : *to + acc[i][j];
        } else {
          if (p.v0 + m >= p.vocab || m >= M) continue;
          const float gain = *p.r.gain * (p.tx == MM_F16 ? 1.f / kF16Gain : 1.f);
          p.dw[(int64_t)(p.v0 + m) * p.lddw + n] = bits16(p.tx, acc[i][j] * gain);
        }
      }
    }
  }
}

// ---------------------------------------------------------------- loss and dx by row
struct LossParams {
  LossArgs a;
  Rows r;
  const float2 *part;
  const float *hit;
  int tiles;
};

// 32 rows a block, 8 threads a row over the tiles of the vocabulary; the last
// steps in fp64, so that a loss is no less exact than its sums.
__global__ void __launch_bounds__(256) loss_kernel(const LossParams p) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ float2 sh[8][32];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int64_t row = (int64_t)blockIdx.x * 32 + x;
  const int slot = row < p.a.rows ? p.r.slot[row] : -1;
  float r = -INFINITY, s = 0.f;
  if (slot >= 0)
    for (int i = y; i < p.tiles; i += 8) {
      const float2 v = p.part[(int64_t)i * p.r.rows_pad + slot];
      const float top = fmaxf(r, v.x);
      s = s * exp2_fast(r - top) + v.y * exp2_fast(v.x - top);
      r = top;
    }
  sh[y][x] = make_float2(r, s);
  __syncthreads();
  if (y > 0 || row >= p.a.rows) return;
  for (int k = 1; k < 8; ++k) {
    const float2 v = sh[k][x];
    const float top = fmaxf(r, v.x);
    if (v.x == -INFINITY) continue;  // (no tile)
    s = s * exp2_fast(r - top) + v.y * exp2_fast(v.x - top);
    r = top;
  }
  const double lse = slot < 0 ? 0.0 : (double)r * 0.693147180559945309 + log((double)s);
  p.a.loss[row] = slot < 0 ? 0.f : (float)(lse - (double)p.hit[slot]);
  if (p.a.lse) p.a.lse[row] = (float)lse;
}

struct DxParams {
  LossArgs a;
  Rows r;
  const float *acc;
  int64_t ldacc;
};
__global__ void __launch_bounds__(256) dx_kernel(const DxParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const float gain = *p.r.gain * (p.a.tx == MM_F16 ? 1.f / kF16Gain : 1.f);
  for (int64_t row = blockIdx.x; row < p.a.rows; row += gridDim.x) {
    const int slot = p.r.slot[row];
    for (int c = threadIdx.x; c < p.a.cols; c += 256)
      static_cast<uint16_t *>(p.a.dx)[row * p.a.lddx + c] =
          slot < 0 ? (uint16_t)0 : bits16(p.a.tx, p.acc[(int64_t)slot * p.ldacc + c] * gain);
  }
}

// A call's scratch, cut up.
struct Cut {
  char *base = nullptr;
  size_t used = 0;
  template <typename T>
  T *take(int64_t n) {
    T *p = base ? reinterpret_cast<T *>(base + used) : nullptr;
    used += ((size_t)n * sizeof(T) + 255) / 256 * 256;
    return p;
  }
};

Rows cut_rows(Cut &cut, const LossArgs &a, bool backward) {
  Rows r;
  std::memset(&r, 0, sizeof r);
  r.rows_pad = (a.rows + kRowTile - 1) / kRowTile * kRowTile;
  r.ldx = ((int64_t)a.cols + 7) / 8 * 8;
  r.count = cut.take<int>(1);
  r.gain = cut.take<float>(1);
  r.slot = cut.take<int>(a.rows);
  r.target = cut.take<int>(r.rows_pad);
  if (backward) {
    r.ratio = cut.take<float>(r.rows_pad);
    r.lse2 = cut.take<float>(r.rows_pad);
  }
  r.x = cut.take<uint16_t>((int64_t)r.rows_pad * r.ldx);
  return r;
}

mm_status launch_gather(const LossArgs &a, const Rows &r, bool backward, LaunchCtx &ctx) {
  GatherParams p{a, r, backward};
  const int blocks = std::min(a.rows, 2 * ctx.dev->info.sms);
  cudaError_t e = launch_pdl(gather_kernel, dim3((unsigned)blocks), dim3(kGatherThreads), 0, ctx.stream, dim3(1), p);
  if (e != cudaSuccess) return cuda_error(e, "cross_entropy launch (gather)");
  count_operator_launch();
  return MM_OK;
}

template <int MODE>
mm_status launch_tiles(const TileParams &p, int M, int N, LaunchCtx &ctx) {
  cudaError_t e = launch_pdl(tile_kernel<MODE>, dim3((unsigned)((N + 63) / 64), (unsigned)((M + 63) / 64)), dim3(256), 0,
                             ctx.stream, dim3(1), p);
  if (e != cudaSuccess) return cuda_error(e, "cross_entropy launch");
  count_operator_launch();
  return MM_OK;
}

}  // namespace

mm_status launch_cross_entropy(const LossArgs &a, LaunchCtx &ctx) {
  TileParams p;
  std::memset(&p, 0, sizeof p);
  const int tiles = (a.vocab + 63) / 64;
  Cut cut;
  for (int pass = 0; pass < 2; ++pass) {
    cut.used = 0;
    p.r = cut_rows(cut, a, false);
    p.hit = cut.take<float>(p.r.rows_pad);
    p.part = cut.take<float2>((int64_t)tiles * p.r.rows_pad);
    if (pass == 0) {
      void *w = nullptr;
      mm_status st = get_scratch(ctx, SCRATCH_WORKSPACE, cut.used, &w);
      if (st != MM_OK) return st;
      cut.base = static_cast<char *>(w);
    }
  }
  p.W = static_cast<const uint16_t *>(a.weight);
  p.ldw = a.ldw;
  p.cols = a.cols;
  p.vocab = p.width = a.vocab;
  p.tx = a.tx;
  mm_status st = launch_gather(a, p.r, false, ctx);
  if (st != MM_OK) return st;
  if (tiles > 0 && (st = launch_tiles<MODE_LSE>(p, a.rows, a.vocab, ctx)) != MM_OK) return st;
  LossParams l{a, p.r, p.part, p.hit, tiles};
  cudaError_t e = launch_pdl(loss_kernel, dim3((unsigned)((a.rows + 31) / 32)), dim3(256), 0, ctx.stream, dim3(1), l);
  if (e != cudaSuccess) return cuda_error(e, "cross_entropy launch (loss)");
  count_operator_launch();
  return MM_OK;
}

mm_status launch_cross_entropy_backward(const LossArgs &a, LaunchCtx &ctx) {
  if (a.rows == 0) return write_zeros(a.dweight, a.lddw, a.vocab, a.cols, a.tx, ctx);
  if (a.vocab == 0) return write_zeros(a.dx, a.lddx, a.rows, a.cols, a.tx, ctx);
  TileParams p;
  std::memset(&p, 0, sizeof p);
  const int piece = std::min((a.vocab + 63) / 64 * 64, 4096);
  Cut cut;
  for (int pass = 0; pass < 2; ++pass) {
    cut.used = 0;
    p.r = cut_rows(cut, a, true);
    p.ldg = piece;
    p.g = cut.take<uint16_t>((int64_t)p.r.rows_pad * piece);
    p.ldacc = ((int64_t)a.cols + 63) / 64 * 64;
    if (a.dx) p.acc = cut.take<float>((int64_t)p.r.rows_pad * p.ldacc);
    if (pass == 0) {
      void *w = nullptr;
      mm_status st = get_scratch(ctx, SCRATCH_WORKSPACE, cut.used, &w);
      if (st != MM_OK) return st;
      cut.base = static_cast<char *>(w);
    }
  }
  p.W = static_cast<const uint16_t *>(a.weight);
  p.ldw = a.ldw;
  p.cols = a.cols;
  p.vocab = a.vocab;
  p.tx = a.tx;
  p.dw = static_cast<uint16_t *>(a.dweight);
  p.lddw = a.lddw;
  mm_status st = launch_gather(a, p.r, true, ctx);
  if (st != MM_OK) return st;
  for (p.v0 = 0; p.v0 < a.vocab; p.v0 += piece) {
    p.first = p.v0 == 0;
    p.width = std::min(piece, (a.vocab - p.v0 + 63) / 64 * 64);
    if ((st = launch_tiles<MODE_G>(p, a.rows, p.width, ctx)) != MM_OK) return st;
    if (a.dx && (st = launch_tiles<MODE_DX>(p, a.rows, a.cols, ctx)) != MM_OK) return st;
    if (a.dweight && (st = launch_tiles<MODE_DW>(p, p.width, a.cols, ctx)) != MM_OK) return st;
  }
  if (!a.dx) return MM_OK;
  DxParams d{a, p.r, p.acc, p.ldacc};
  cudaError_t e = launch_pdl(dx_kernel, dim3((unsigned)std::min(a.rows, 8 * ctx.dev->info.sms)), dim3(256), 0,
                             ctx.stream, dim3(1), d);
  if (e != cudaSuccess) return cuda_error(e, "cross_entropy_backward launch (dx)");
  count_operator_launch();
  return MM_OK;
}

}  // namespace mm
