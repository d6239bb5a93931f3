// Softmax cross entropy of x projected on a vocabulary, and its gradients.
//
//   l[t, v] = sum_c x[t, c] W[v, c];  lse[t] = log sum_v exp l[t, v]
//   loss[t] = lse[t] - l[t, y[t]]
//   g[t, v] = dloss[t] (exp(l[t, v] - lse[t]) - [v = y[t]]);  dx = g W, dW = g^T x
//
// Forward: a product whose tiles never leave the SM: a tile's rows leave their
// maximum m and s = sum exp(l - m), and the target's logit; loss = (m - l[y]) + log s.
// The maximum is subtracted before the factor log2(e): the difference is exact where the
// share is not small, whatever the logits' size, and the largest one's share is exactly 1.
// Backward: the vocabulary in pieces, each the product again with g as the
// epilogue's output in 16 bits, then its two products; what g's rounding loses at the
// targets, whose terms are the large ones, is kept and added.
// Rows without a target are left out: the others' x is gathered first, so the
// products run over whole tiles of rows that count, and what a padded row holds
// is never read.
// What bounds it: above a few hundred rows the tensor cores, under the power cap
// (8192 x 4096 x 131072 5.2-5.3 ms, 1.66-1.70 PFLOP/s; backward 8192 x 4096 x 32000, a
// quarter without a target, 3.0 ms); below, W's bytes (16 x 4096 x 32000 46-47 us, 5.6 TB/s
// over the whole call; backward, W twice and dW, 164 us).
#include <algorithm>

#include "../operators.h"
#include "../per_device.h"
#include "indices.cuh"
#include "row_copy.cuh"
#include "tcgen05.cuh"
#include "tile_out.cuh"
#include "values.cuh"

namespace mm {

namespace {

using namespace tc;

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
// exp of a logit less another, or less the logarithm of a row's sum, not above it.  (2^(l log2(e) - r) in one FMA, r a
// rounded multiple, is off by half a step of r: it passed 2^x's range from logits of 3e9 on,
// and log2(e)'s rounding put a loss off by 1.5e-8 of its largest logit.)
__device__ __forceinline__ float exp_fast(float d) { return exp2_fast(d * kLog2e); }
// Below every logit but -infinity, and what a sum of none has for its maximum.
constexpr float kLeast = -3.402823466e38f;

// ---------------------------------------------------------------- the rows that count
// Where each call's scratch holds what; i: a row among those that count, of
// `rows_pad`, a multiple of 256.
// Few rows that TMA reads as they lie are not gathered (they are one row tile whether or
// not all count): count is null then, i is the row itself, and there are only gain and x.
struct Rows {
  int *count;       // [0] the rows that count, or null
  float *gain;      // largest |dloss|
  int *slot;        // [rows] i of a row, or -1
  int *row;         // [rows] the row of an i
  int *target;      // [rows_pad], -1 past the count
  float *ratio;     // [rows_pad] dloss / gain (f16: times kF16Gain), 0 past the count
  float *lse;       // [rows_pad]
  uint16_t *x;      // [rows_pad][ldx], zeros from cols to ldx and for rows up to a multiple of 64
  // Backward of many rows: the rows in the order of their targets' tiles of 256 tokens, and
  // what the rounding of g leaves at the targets (see leave_rest).
  float *rest;      // [rows_pad] as g is scaled; 0 where nothing was left
  int *first;       // [tiles + 1] the first i of a tile's targets
  uint16_t *cells;  // [cell][64 rows][256 tokens]
  int64_t ldx;
  int rows_pad;
};

__device__ __forceinline__ float abs_weight(const float *dloss, int64_t i) { return dloss ? fabsf(dloss[i]) : 1.f; }
constexpr float kLargestFinite = 3.402823466e38f;
// What g's rows are multiplied by.
__device__ __forceinline__ float ratio_of(const float *dloss, int64_t i, float gain, int tx) {
  return (dloss ? dloss[i] : 1.f) / gain * (tx == MM_F16 ? kF16Gain : 1.f);
}

struct GatherParams {
  LossArgs a;
  Rows r;
  int backward;
  int log_threads;  // threads a row
  int blocks;       // that gather; those after them copy
  PackRows pack;    // W, where TMA cannot read it as it lies
};

__device__ __forceinline__ int valid_target(const LossArgs &a, int64_t t) {
  const int64_t v = load_token(a.targets, a.ti, t, a.vocab);
  return v < a.vocab ? (int)v : -1;
}

// Each block has an equal share of the rows and counts the rows that count before its
// own (and, backward, finds the largest |dloss| of all) for itself: a few KB from L2
// instead of another kernel.  Rows move in 16-byte pieces, wherever they start.  W is
// copied by the same launch where it has to be.  (8192 x 4096: 29 us; 50257 x 1001 of W
// 41 us, 5 TB/s.)
constexpr int kGatherThreads = 512, kGatherWarps = kGatherThreads / 32;
__global__ void __launch_bounds__(kGatherThreads, 2) gather_kernel(const GatherParams p) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ int warp_count[kGatherWarps];
  __shared__ float warp_max[kGatherWarps];
  __shared__ int at_row[kGatherThreads];  // the source row of the k-th that counts
  const LossArgs &a = p.a;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  if ((int)blockIdx.x >= p.blocks) {
    pack_rows(p.pack, ((int64_t)blockIdx.x - p.blocks) * kGatherThreads + t, ((int64_t)gridDim.x - p.blocks) * kGatherThreads);
    return;
  }
  const int r0 = (int)((int64_t)a.rows * blockIdx.x / p.blocks);
  const int r1 = (int)((int64_t)a.rows * (blockIdx.x + 1) / p.blocks);
  int before = 0;
  float top = 0.f;  // of the finite ones
  const int look = p.backward ? a.rows : r0;
#pragma unroll 4
  for (int i = t; i < look; i += kGatherThreads) {
    const int target = valid_target(a, i);
    const float d = abs_weight(p.backward ? a.dloss : nullptr, i);
    before += target >= 0 && i < r0;
    if (target >= 0 && d <= kLargestFinite) top = fmaxf(top, d);
  }
  before = __reduce_add_sync(0xffffffffu, before);
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) warp_count[warp] = before, warp_max[warp] = top;
  __syncthreads();
  before = 0;
  for (int w = 0; w < kGatherWarps; ++w) before += warp_count[w], top = fmaxf(top, warp_max[w]);
  if (top == 0.f) top = 1.f;
  __syncthreads();

  const int pieces = (int)(p.r.ldx / 8);
  const uint8_t *x = static_cast<const uint8_t *>(a.x);
  for (int g0 = r0; g0 < r1; g0 += kGatherThreads) {
    const int i = g0 + t, target = i < r1 ? valid_target(a, i) : -1;
    const uint32_t mask = __ballot_sync(0xffffffffu, target >= 0);
    if (lane == 0) warp_count[warp] = __popc(mask);
    __syncthreads();
    int at = __popc(mask & ((1u << lane) - 1)), total = 0;
    for (int w = 0; w < kGatherWarps; ++w) {
      if (w < warp) at += warp_count[w];
      total += warp_count[w];
    }
    if (i < r1) p.r.slot[i] = target >= 0 ? before + at : -1;
    if (target >= 0) {
      at_row[at] = i;
      p.r.row[before + at] = i;
      p.r.target[before + at] = target;
      if (p.backward) {
        p.r.ratio[before + at] = ratio_of(a.dloss, i, top, a.tx);
        p.r.lse[before + at] = a.lse[i];
      }
    }
    __syncthreads();
    constexpr int U = 4;  // pieces read before the first is stored
    const int threads = 1 << p.log_threads, t0 = t & (threads - 1);
    for (int k = t >> p.log_threads; k < total; k += kGatherThreads >> p.log_threads) {
      const uint8_t *from = x + (int64_t)at_row[k] * a.ldx * 2;
      uint4 *to = reinterpret_cast<uint4 *>(p.r.x + (int64_t)(before + k) * p.r.ldx);
      for (int c = t0; c < pieces; c += threads * U) {
        RowPiece<2> v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (c + u * threads < pieces) v[u].load(from, (int64_t)a.cols * 2, (int64_t)(c + u * threads) * 16);
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (c + u * threads < pieces)
            to[c + u * threads] = v[u].value(from, (int64_t)a.cols * 2, (int64_t)(c + u * threads) * 16);
      }
    }
    before += total;
    __syncthreads();
  }
  if ((int)blockIdx.x == p.blocks - 1) {
    if (t == 0) *p.r.count = before, *p.r.gain = top;
    const int end = max(1, (before + kRowTile - 1) / kRowTile) * kRowTile;
    for (int i = before + t; i < end; i += kGatherThreads) {
      p.r.target[i] = -1;
      if (p.backward) p.r.ratio[i] = p.r.lse[i] = 0.f;
    }
    const int64_t z0 = (int64_t)before * pieces, z1 = (int64_t)max(1, (before + 63) / 64) * 64 * pieces;
    for (int64_t i = z0 + t; i < z1; i += kGatherThreads)
      reinterpret_cast<uint4 *>(p.r.x)[i] = make_uint4(0, 0, 0, 0);
  }
}

// The same for the backward pass of many rows, in the order in which the targets were sorted.
constexpr int kTileTokens = 256, kLogTileTokens = 8, kCellRows = 64;
struct SortedParams {
  GatherParams g;
  const uint2 *sorted;  // (tile of the target, row), or null: to be counted
  int tiles;            // the key of a row without a target
  int64_t cell_pieces;  // all cells', of 16 bytes
};
__global__ void __launch_bounds__(kGatherThreads, 2) gather_sorted_kernel(const SortedParams q) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ float warp_max[kGatherWarps];
  __shared__ int at_row[kGatherThreads];  // the source row of a place, -1: zeros, -2: left as it is
  const GatherParams &p = q.g;
  const LossArgs &a = p.a;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  if ((int)blockIdx.x >= p.blocks) {
    pack_rows(p.pack, ((int64_t)blockIdx.x - p.blocks) * kGatherThreads + t, ((int64_t)gridDim.x - p.blocks) * kGatherThreads);
    return;
  }
  for (int64_t i = (int64_t)blockIdx.x * kGatherThreads + t; i < q.cell_pieces; i += (int64_t)p.blocks * kGatherThreads)
    reinterpret_cast<uint4 *>(p.r.cells)[i] = make_uint4(0, 0, 0, 0);
  float top = 0.f;  // of the finite ones
#pragma unroll 4
  for (int i = t; i < a.rows; i += kGatherThreads) {
    const float d = abs_weight(a.dloss, i);
    if (valid_target(a, i) >= 0 && d <= kLargestFinite) top = fmaxf(top, d);
  }
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) warp_max[warp] = top;
  __syncthreads();
  for (int w = 0; w < kGatherWarps; ++w) top = fmaxf(top, warp_max[w]);
  if (top == 0.f) top = 1.f;
  if (blockIdx.x == 0 && t == 0) *p.r.gain = top;

  const int none = q.tiles, pieces = (int)(p.r.ldx / 8);
  const auto key_at = [&](int i) { return i < 0 ? -1 : i < a.rows ? (int)q.sorted[i].x : none; };
  const int r0 = (int)((int64_t)p.r.rows_pad * blockIdx.x / p.blocks);
  const int r1 = (int)((int64_t)p.r.rows_pad * (blockIdx.x + 1) / p.blocks);
  const uint8_t *x = static_cast<const uint8_t *>(a.x);
  for (int g0 = r0; g0 < r1; g0 += kGatherThreads) {
    const int i = g0 + t;
    if (i < r1) {
      const int key = key_at(i), row = i < a.rows ? (int)q.sorted[i].y : -1;
      const bool live = key < none;
      at_row[t] = live ? row : i < kCellRows || key_at(i & ~(kCellRows - 1)) < none ? -1 : -2;
      if (row >= 0) p.r.slot[row] = live ? i : -1;
      if (live) p.r.row[i] = row;
      p.r.target[i] = live ? valid_target(a, row) : -1;
      p.r.ratio[i] = live ? ratio_of(a.dloss, row, top, a.tx) : 0.f;
      p.r.lse[i] = live ? a.lse[row] : 0.f;
      p.r.rest[i] = 0.f;
      // (rows_pad is past the rows or the last of them is the last place: both ends are seen)
      for (int k = key_at(i - 1) + 1; k <= key; ++k) p.r.first[k] = i;
      if (i + 1 == p.r.rows_pad && live)
        for (int k = key + 1; k <= none; ++k) p.r.first[k] = i + 1;
      if (live && key_at(i + 1) >= none) *p.r.count = i + 1;
      if (i == 0 && !live) *p.r.count = 0;
    }
    __syncthreads();
    constexpr int U = 4;  // pieces read before the first is stored
    const int threads = 1 << p.log_threads, t0 = t & (threads - 1), total = min(kGatherThreads, r1 - g0);
    for (int k = t >> p.log_threads; k < total; k += kGatherThreads >> p.log_threads) {
      const int source = at_row[k];
      if (source == -2) continue;
      const uint8_t *from = x + (int64_t)source * a.ldx * 2;
      uint4 *to = reinterpret_cast<uint4 *>(p.r.x + (int64_t)(g0 + k) * p.r.ldx);
      for (int c = t0; c < pieces; c += threads * U) {
        RowPiece<2> v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (source >= 0 && c + u * threads < pieces) v[u].load(from, (int64_t)a.cols * 2, (int64_t)(c + u * threads) * 16);
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (c + u * threads < pieces)
            to[c + u * threads] = source >= 0 ? v[u].value(from, (int64_t)a.cols * 2, (int64_t)(c + u * threads) * 16)
                                              : make_uint4(0, 0, 0, 0);
      }
    }
    __syncthreads();
  }
}

// The same of fewer rows, by counting: a row's place is how many come before it, one by a
// smaller key or by the same and a smaller number, counted by a warp over all keys in shared
// memory.  (A sort and its launch are 5-8 us: gradients of 129 x 256 x 512 36 -> 32 us, 300 x 1024
// x 32000 114 -> 108; 4096 x 1024 x 32000 sorted 572, counted 575.)
constexpr int kCountedRows = 2048;
__global__ void __launch_bounds__(kGatherThreads, 2) gather_counted_kernel(const SortedParams q) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ float warp_max[kGatherWarps];
  __shared__ int keys[kCountedRows], at_place[kGatherThreads];
  const GatherParams &p = q.g;
  const LossArgs &a = p.a;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31, none = q.tiles;
  if ((int)blockIdx.x >= p.blocks) {
    pack_rows(p.pack, ((int64_t)blockIdx.x - p.blocks) * kGatherThreads + t, ((int64_t)gridDim.x - p.blocks) * kGatherThreads);
    return;
  }
  const int64_t thread = (int64_t)blockIdx.x * kGatherThreads + t, threads = (int64_t)p.blocks * kGatherThreads;
  for (int64_t i = thread; i < q.cell_pieces; i += threads) reinterpret_cast<uint4 *>(p.r.cells)[i] = make_uint4(0, 0, 0, 0);
  float top = 0.f;  // of the finite ones
  for (int i = t; i < a.rows; i += kGatherThreads) {
    const int target = valid_target(a, i);
    const float d = abs_weight(a.dloss, i);
    keys[i] = target >= 0 ? target >> kLogTileTokens : none;
    if (target >= 0 && d <= kLargestFinite) top = fmaxf(top, d);
  }
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) warp_max[warp] = top;
  __syncthreads();
  for (int w = 0; w < kGatherWarps; ++w) top = fmaxf(top, warp_max[w]);
  if (top == 0.f) top = 1.f;
  // how many rows have a smaller key, or this one and a number below `row`
  const auto before = [&](int key, int row) {
    int n = 0;
    for (int j = lane; j < a.rows; j += 32) n += keys[j] < key || (keys[j] == key && j < row);
    return __reduce_add_sync(0xffffffffu, n);
  };
  const int count = before(none, 0);
  if (thread == 0) *p.r.gain = top, *p.r.count = count;
  for (int64_t k = (int64_t)blockIdx.x * kGatherWarps + warp; k <= none; k += (int64_t)p.blocks * kGatherWarps) {
    const int n = before((int)k, 0);
    if (lane == 0) p.r.first[k] = n;
  }
  const int pieces = (int)(p.r.ldx / 8);
  for (int64_t i = count + thread; i < p.r.rows_pad; i += threads) {
    p.r.target[i] = -1;
    p.r.ratio[i] = p.r.lse[i] = p.r.rest[i] = 0.f;
  }
  const int64_t z1 = (int64_t)max(1, (count + 63) / 64) * 64 * pieces;
  for (int64_t i = (int64_t)count * pieces + thread; i < z1; i += threads) reinterpret_cast<uint4 *>(p.r.x)[i] = make_uint4(0, 0, 0, 0);

  const int r0 = (int)((int64_t)a.rows * blockIdx.x / p.blocks), n = (int)((int64_t)a.rows * (blockIdx.x + 1) / p.blocks) - r0;
  for (int k = warp; k < n; k += kGatherWarps) {
    const int row = r0 + k, key = keys[row], place = before(key, row);
    if (lane != 0) continue;
    at_place[k] = key < none ? place : -1;
    p.r.slot[row] = at_place[k];
    if (key < none) {
      p.r.row[place] = row;
      p.r.target[place] = valid_target(a, row);
      p.r.ratio[place] = ratio_of(a.dloss, row, top, a.tx);
      p.r.lse[place] = a.lse[row];
      p.r.rest[place] = 0.f;
    }
  }
  __syncthreads();
  constexpr int U = 4;  // pieces read before the first is stored
  const int row_threads = 1 << p.log_threads, t0 = t & (row_threads - 1);
  for (int k = t >> p.log_threads; k < n; k += kGatherThreads >> p.log_threads) {
    if (at_place[k] < 0) continue;
    const uint8_t *from = static_cast<const uint8_t *>(a.x) + (int64_t)(r0 + k) * a.ldx * 2;
    uint4 *to = reinterpret_cast<uint4 *>(p.r.x + (int64_t)at_place[k] * p.r.ldx);
    for (int c = t0; c < pieces; c += row_threads * U) {
      RowPiece<2> v[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (c + u * row_threads < pieces) v[u].load(from, (int64_t)a.cols * 2, (int64_t)(c + u * row_threads) * 16);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (c + u * row_threads < pieces)
          to[c + u * row_threads] = v[u].value(from, (int64_t)a.cols * 2, (int64_t)(c + u * row_threads) * 16);
    }
  }
}

// ---------------------------------------------------------------- the products
// Products on tcgen05 (kind::f16), one after another:
//   LSE, G   x W^T, both K-major: the sums of a tile's rows, or g in 16 bits
//   G_ONE    G over no more of K than one chunk (see kChunkKb), on pairs
//   DX       g W, W MN-major as it lies, K the piece of the vocabulary; added to
//            fp32 sums over the pieces
//   DW       g^T x, both MN-major as they lie, K the rows
//   DW_LONG  DW over more rows than kLongRows, in chunks of kLongChunkKb
// 256 x 256 tiles on pairs of SMs, or 128 x 256 on single ones where there are few
// rows; persistent, two accumulators in TMEM, so that a tile's epilogue runs under
// the next tile's main loop.  Neither the rows that count nor the tiles are known
// to the host: each kernel reads the count and lays out its own tiles.
enum Mode { MODE_LSE, MODE_G, MODE_G_ONE, MODE_DX, MODE_DW, MODE_DW_LONG };
constexpr __host__ __device__ bool is_dw(int mode) { return mode == MODE_DW || mode == MODE_DW_LONG; }

// Warp 0 copies, warp 1 issues MMAs, the others take tiles out, eight a tile.  Where a
// tile leaves in 16 bits from one sum over K there are 16, eight for each accumulator:
// products over few of K are all epilogue, and what writes to memory in one half overlaps with
// what is converted in the other (all 16 on one tile: converted, then written).  G holds its
// sums over chunks of K in registers, so it has eight (16 with half of the columns each:
// gradients of 2048 x 4096 x 32000 1025 -> 1098 us).
constexpr int out_warps(int mode, int cg) { return cg == 2 && (mode == MODE_G_ONE || mode == MODE_DW) ? 16 : 8; }
constexpr int tile_threads(int mode, int cg) { return 64 + 32 * out_warps(mode, cg); }
constexpr int kErrCopy = 0xa01, kErrMma = 0xa02, kErrStore = 0xa03, kErrDrain = 0xa04;
constexpr int kGroupRows = 8;  // row tiles walked together, so that their operands stay in L2

// How the tiles of a product are walked: grouped by row tiles.  Those of a last wave that
// does not fill the places are cut: in two halves where they fill at most half of them
// (or there are no more), or, in DX, whose K is long, in as many parts of K as fit.
struct Tiles {
  int tiles_m, tiles_n, full, parts, total;
  bool cut_k;
};
__device__ __forceinline__ Tiles tiles_of(int M, int tile_m, int tiles_n, int bn, int places, int max_parts = 0) {
  Tiles s;
  s.tiles_m = (M + tile_m - 1) / tile_m;
  s.tiles_n = tiles_n;
  s.cut_k = max_parts > 0;
  const int tiles = s.tiles_m * tiles_n, rem = tiles % places;
  s.parts = rem == 0 ? 1 : s.cut_k ? max(1, min(places / rem, max_parts)) : bn == 256 && 2 * rem <= places ? 2 : 1;
  s.full = s.parts > 1 ? tiles - rem : tiles;
  s.total = s.full + (tiles - s.full) * s.parts;
  return s;
}
struct Unit {
  int tm, n0, w, part;
};
__device__ __forceinline__ Unit unit_at(const Tiles &s, int bn, int u) {
  Unit x;
  int t = u;
  x.part = 0;
  const bool cut = u >= s.full;
  if (cut) t = s.full + (u - s.full) / s.parts, x.part = (u - s.full) % s.parts;
  const int per = kGroupRows * s.tiles_n, g = t / per, rows = min(kGroupRows, s.tiles_m - g * kGroupRows);
  const int r = t - g * per;
  x.tm = g * kGroupRows + r % rows;
  x.n0 = (r / rows) * bn;
  x.w = bn;
  if (cut && !s.cut_k) x.w = bn / 2, x.n0 += x.part * x.w;
  return x;
}
// The place of tile (tm, tn) in the walk.
__device__ __forceinline__ int tile_at(const Tiles &s, int tm, int tn) {
  const int g = tm / kGroupRows, rows = min(kGroupRows, s.tiles_m - g * kGroupRows);
  return g * kGroupRows * s.tiles_n + tn * rows + tm - g * kGroupRows;
}
// DX: parts of at least eight blocks of K.
__device__ __forceinline__ int max_parts_of(int piece_kb) { return max(1, piece_kb / 8); }

struct TileParams {
  Rows r;
  const void *x, *targets;  // where r.count is null: x as it lies, `rows` of it ...
  const float *lse, *dloss;
  int64_t ldx;
  int ti, rows;
  int cols, vocab;
  int v0, width;     // the piece of the vocabulary: its first token, how many (G: padded to 64)
  int tx;
  int bn, tiles_n, places;
  int a_rows;        // CG = 1: the rows of A that are loaded
  int boxes;         // DW: boxes a warp
  int low;           // few rows: g is two values, the second in the rows from here on (else 0)
  int num_kb;        // 64-element blocks of K (DW: of the rows that count)
  int piece_kb;      // DX: those of a whole piece
  float2 *part;      // LSE: [128 of the vocabulary][rows_pad] (m, s)
  float *hit;        // LSE: [rows_pad] the target's logit
  // DX: blocks of 32 rows by 32 columns, each [4 columns][row][column]: the whole tiles'
  // [row block][acc_cols], then, from acc_cut on, [unit][row block][column block] of those
  // that are cut in parts
  float *acc, *acc_cut;
  int acc_cols;
  int first;         // DX: the first piece
  uint16_t *g;       // G of few rows: its rows, ldg apart
  int64_t ldg;
  uint16_t *dw;
  int64_t lddw;
  int vec;           // DW: its rows are whole 16-byte pieces
  Waits wait;
};

// Stages of 64 of K: 128 rows of A, and of B 128 (its half of a pair's tile) or 256.
// Few rows (CG = 1) wait for W, so their A has room for no more rows than there are (a
// multiple of 16): the MMA's other rows read what lies behind, and nobody reads theirs.
// That leaves more of the ring to W in flight.  A pair's tiles in 16 bits leave through
// boxes in shared memory, one for each warp that takes them out, or two where K is a few
// stages and the ring need not be long.
constexpr uint32_t kSmemBytes = 227 * 1024, kBarBytes = 1024;
template <int MODE, int CG>
struct Ring {
  static constexpr int kOut = out_warps(MODE, CG), kTeams = kOut / 8;
  static constexpr bool kHasBoxes = CG == 2 && (MODE == MODE_G || MODE == MODE_G_ONE || is_dw(MODE));
  static constexpr uint32_t kB = (CG == 2 ? 128 : 256) * 128;
  static constexpr int kMaxStages = 6;
  static constexpr size_t kSmem = kSmemBytes;
  // bytes before the ring's: boxes, or (LSE) sums
  static __host__ __device__ constexpr uint32_t front(int boxes) { return kHasBoxes ? kOut * boxes * kBoxB : 2 * 128 * 8; }
  static __host__ __device__ constexpr int stages(int a_rows, int boxes) {
    const int n = (int)((kSmemBytes - 1024 /* alignment */ - kBarBytes - front(boxes)) / (a_rows * 128 + kB));
    return n < kMaxStages ? n : kMaxStages;
  }
};
static_assert(Ring<MODE_G, 2>::stages(128, 1) == 6 && Ring<MODE_G_ONE, 2>::stages(128, 1) == 5 && Ring<MODE_DW, 2>::stages(128, 2) == 3 &&
                  Ring<MODE_LSE, 2>::stages(128, 1) == 6 && Ring<MODE_LSE, 1>::stages(128, 1) == 4 &&
                  Ring<MODE_G, 1>::stages(16, 1) == 6,
              "what the measurements were taken with");

// The rows that count, and how many a product has: one at least (a tile of zeros where
// none counts, so that dW is written), which then has no row of x behind it.
__device__ __forceinline__ int live_rows(const Rows &r, int rows) { return r.count ? *r.count : rows; }
__device__ __forceinline__ int row_count(const Rows &r, int rows) { return max(1, live_rows(r, rows)); }
__device__ __forceinline__ int target_of(const TileParams &p, int row) {
  if (p.r.count) return p.r.target[row];
  const int64_t v = row < p.rows ? load_token(p.targets, p.ti, row, p.vocab) : p.vocab;
  return v < p.vocab ? (int)v : -1;
}

template <int CG>
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap *map, uint32_t bar, int x, int y) {
  if constexpr (CG == 2) tma_load_2d_pair(dst, map, bar, x, y);
  else tma_load_2d(dst, map, bar, x, y);
}

// Whether `ok` holds in all of the warps that take tiles out (barrier 1).
__device__ __forceinline__ bool all_take(bool ok) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.and.aligned.pred q, 1, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(all)
      : "r"((uint32_t)ok)
      : "memory");
  return all != 0;
}

// What a tile leaves, by eight warps: two for each quarter of the 128 rows, a half of
// the columns each.

// LSE, G: the logits are fp32 sums over K that the tensor core truncates at each step of
// 16, towards zero, so that their error grows with K and the sum itself.  A sum over
// kChunkKb blocks at a time, added up here in registers, rounded, keeps it at that of
// an fp32 loop (8192 x 4096 x 131072: the loss off by 2.9e-6 of itself in one chain, by
// 7e-7 in chunks of 1024 of K, by 3e-7 of 512, for 2 % of the time).  Backward, the same sums
// in the same order give the same logits, bit for bit, so that a share is the exponential of
// what lse was made from.  (In one chain the share of a token that holds a row's whole mass
// was off by -2.4e-4 at K = 4096 and a logit of 30, by -0.8 % at 1000, by -6 % at K = 16384 and
// 1000, which is a gradient where there is none.  The chunks take 2-4 % of the gradients' time.)
constexpr int kChunkKb = 8;
// DW: a sum over the rows falls short by up to 2^-24 of itself a step of 16 rows, in one chain
// by 6e-5 at 65536 rows, a third of an f16 rounding, 3e-4 at 262144 and 1.1e-3 at 1048576 (an
// error of 1.2e-3 where rounding alone leaves 2e-4).  Sums over 8192 rows at a time leave 1e-5.
// They take a longer ring and half of the warps, which is faster besides, from about 1000 rows
// on: us of this product, two teams / one with chunks: 800 x 1000 x 50264 67 / 67, 2048 x 4096 x
// 32000 305 / 292, 8192 x 256 x 32000 104 / 97, 8192 x 4096 x 16000 607 / 588; chunks of 1024 rows
// 597; 16 x 4096 x 32000, all epilogue, two teams 51, one 64.
constexpr int kLongChunkKb = 128, kLongRows = 1024;

// A chunk of w columns, added to a thread's sums (the first: the sums themselves).
__device__ __forceinline__ void add_chunk(float (&sum)[128], uint32_t tmem, int w, bool first) {
#pragma unroll
  for (int b = 0; b < 4; ++b)
    if (b * 32 < w) {
      uint32_t v[32];
      tmem_ld_32cols(tmem + (uint32_t)(b * 32), v);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 32; ++i) sum[b * 32 + i] = first ? __uint_as_float(v[i]) : sum[b * 32 + i] + __uint_as_float(v[i]);
    }
}
// A row's maximum m and sum of exp(l - m) over w logits, the first of which is token n0.
__device__ __forceinline__ float2 sum_exp(const TileParams &p, float (&l)[128], int n0, int w, int target, float *hit) {
  float m = kLeast, s = 0.f;
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const int left = p.vocab - n0 - b * 32, at = target - n0 - b * 32;
    if (b * 32 >= w || left <= 0) break;
    if (__any_sync(0xffffffffu, (unsigned)at < 32u)) {
      float h = 0.f;
#pragma unroll
      for (int i = 0; i < 32; ++i) h = at == i ? l[b * 32 + i] : h;
      if ((unsigned)at < 32u) *hit = h;
    }
    if (left < 32) {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (i >= left) l[b * 32 + i] = -INFINITY;
    }
    float top[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      top[k] = l[b * 32 + k];
#pragma unroll
      for (int i = k + 4; i < 32; i += 4) top[k] = fmaxf(top[k], l[b * 32 + i]);
    }
    const float next = fmaxf(m, fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])));
    float sum[4] = {s * exp_fast(m - next), 0.f, 0.f, 0.f};
    m = next;
#pragma unroll
    for (int i = 0; i < 32; ++i) sum[i & 3] += exp_fast(l[b * 32 + i] - m);
    s = (sum[0] + sum[1]) + (sum[2] + sum[3]);
  }
  return make_float2(m, s);
}
// Two such sums as one.
__device__ __forceinline__ float2 join_sums(float2 a, float2 b) {
  const float m = fmaxf(a.x, b.x);
  return make_float2(m, a.y * exp_fast(a.x - m) + b.y * exp_fast(b.x - m));
}

// A warp's boxes, filled in turn.
struct Boxes {
  uint8_t *first;
  int n, turn;
  // the next one, free: its store has read it
  __device__ __forceinline__ uint8_t *next() {
    if ((threadIdx.x & 31) == 0) {
      if (n == 2) tma_store_wait_read<1>();
      else tma_store_wait_read<0>();
    }
    __syncwarp();
    uint8_t *box = first + turn * kBoxB;
    if (++turn == n) turn = 0;
    return box;
  }
};
// Columns 32 h .. of 32 rows in 16 bits to half a box.
__device__ __forceinline__ void fill_box(uint8_t *box, int tx, int h, const uint32_t (&v)[32]) {
  const int lane = threadIdx.x & 31;
  const auto f = [&](int i) { return __uint_as_float(v[i]); };
#pragma unroll
  for (int j = 0; j < 4; ++j)
    *reinterpret_cast<uint4 *>(box + lane * 128 + (((4 * h + j) ^ (lane & 7)) << 4)) =
        make_uint4(pack2(tx, f(8 * j), f(8 * j + 1)), pack2(tx, f(8 * j + 2), f(8 * j + 3)),
                   pack2(tx, f(8 * j + 4), f(8 * j + 5)), pack2(tx, f(8 * j + 6), f(8 * j + 7)));
}
__device__ __forceinline__ void store_box_tma(const CUtensorMap *map, uint8_t *box, int x, int y) {
  fence_proxy_async_smem();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) tma_store_2d(map, smem_u32(box), x, y);
}

// g of 32 columns, token `first` the first of them, in place of the logits: a thread's row.
struct GRow {
  int target;
  float ratio, lse;
};
__device__ __forceinline__ GRow g_row(const TileParams &p, int row, float gain) {
  GRow r{target_of(p, row), 0.f, 0.f};
  if (p.r.count) r.ratio = p.r.ratio[row], r.lse = p.r.lse[row];
  else if (r.target >= 0) r.ratio = ratio_of(p.dloss, row, gain, p.tx), r.lse = p.lse[row];
  return r;
}
__device__ __forceinline__ float unpack(int tx, uint32_t w, int odd) {
  if (tx == MM_BF16) return __uint_as_float(odd ? w & 0xffff0000u : w << 16);
  const __half2 v = *reinterpret_cast<const __half2 *>(&w);
  return odd ? __high2float(v) : __low2float(v);
}
// g of many rows is one 16-bit value.  Where a result has few large terms, which are those of the
// targets, their rounding would be in it as its own is: errors 1.2 to 1.5 times those of the
// results' rounding alone.  So what a target's g has lost is kept: dx adds it in fp32, times W's
// row (dx_kernel), and dW as 64 more of K for each 64 rows and tile of 256 tokens in which
// there are targets, which are few, since the rows are sorted by those tiles: cell b + j holds
// rows 64 b .. and tile j, along a path on which one of the two grows at a time.  That takes
// 1-4 % of the gradients' time over 4096 columns, 6 % at 300 x 1024 x 32000 (their order, 4 %
// more of dW's K, W's rows in the last step), more where a few tiles are all the tokens (dW's K
// grows by half over 512); a second value of all g would double dx's and dW's products.
__device__ __noinline__ void leave_rest(float *rests, uint16_t *cells, int tx, int row, int target, float g) {
  const float rest = g - unpack(tx, pack2(tx, g, 0.f), 0);
  rests[row] = rest;
  const int64_t cell = (row >> 6) + (target >> kLogTileTokens);
  cells[(cell * kCellRows + (row & (kCellRows - 1))) * kTileTokens + (target & (kTileTokens - 1))] =
      (uint16_t)pack2(tx, rest, 0.f);
}
// (row: of many, where what g's rounding leaves is kept; else -1)
__device__ __forceinline__ void make_g(const TileParams &p, const GRow &r, uint32_t (&v)[32], int first, int row) {
  const bool live = r.ratio != 0.f;  // (a weight of 0 takes its row out, whatever its logits)
#pragma unroll
  for (int i = 0; i < 32; ++i)
    v[i] = __float_as_uint(exp_fast(__uint_as_float(v[i]) - r.lse) * r.ratio);
  const int at = r.target - first, left = p.vocab - first;
  if (__any_sync(0xffffffffu, (unsigned)at < 32u)) {
    float g = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      g = at == i ? __uint_as_float(v[i]) - r.ratio : g;
      v[i] = at == i ? __float_as_uint(g) : v[i];
    }
    if (row >= 0 && live && (unsigned)at < 32u) leave_rest(p.r.rest, p.r.cells, p.tx, row, r.target, g);
  }
  if (left < 32 || __any_sync(0xffffffffu, !live)) {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = live && i < left ? v[i] : 0u;
  }
}
// G: columns n .. n + 63 of the product's rows row0 .. row0 + 31.
__device__ __forceinline__ void leave_g(const TileParams &p, const CUtensorMap *map, const GRow &r, uint32_t (&v)[2][32], int n,
                                        int row0, Boxes &boxes) {
  uint8_t *box = boxes.next();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    make_g(p, r, v[h], p.v0 + n + 32 * h, row0 + (int)(threadIdx.x & 31));
    fill_box(box, p.tx, h, v[h]);
  }
  store_box_tma(map, box, n, row0);
}
// Few rows: 32 columns from registers, 64 bytes a lane, as two 16-bit values whose sum is
// g to twice the bits, the second some rows behind the first (p.low).  Their products wait for
// memory, so the second costs no time, and a dx or dW of few terms does not show the
// rounding of one g (off by up to half a step, as its own rounding).
// Up to 32 rows the two fill the 64 rows of one block of dW's K, with x twice.
constexpr int kFewestRows = 32;
__device__ __forceinline__ void leave_g_few(const TileParams &p, const GRow &r, uint32_t (&v)[32], int n, int row) {
  make_g(p, r, v, p.v0 + n, -1);
  uint4 *high = reinterpret_cast<uint4 *>(p.g + (int64_t)row * p.ldg + n);
  uint4 *low = reinterpret_cast<uint4 *>(p.g + (int64_t)(row + p.low) * p.ldg + n);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float a = __uint_as_float(v[8 * j + 2 * k]), b = __uint_as_float(v[8 * j + 2 * k + 1]);
      h[k] = pack2(p.tx, a, b);
      l[k] = pack2(p.tx, a - unpack(p.tx, h[k], 0), b - unpack(p.tx, h[k], 1));
    }
    high[j] = make_uint4(h[0], h[1], h[2], h[3]);
    low[j] = make_uint4(l[0], l[1], l[2], l[3]);
  }
}

__device__ __forceinline__ void leave_dw(const TileParams &p, const CUtensorMap *map, uint32_t (&v)[2][32], int n, int v0,
                                         Boxes &boxes, float gain) {
  uint8_t *box = boxes.next();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[h][i] = __float_as_uint(__uint_as_float(v[h][i]) * gain);
    fill_box(box, p.tx, h, v[h]);
  }
  if (p.vec) {
    store_box_tma(map, box, n, v0);
  } else {  // rows that TMA cannot address, or would clip behind their end
    __syncwarp();
    store_box<2>(box, p.dw, (int64_t)v0 * p.lddw + n, p.lddw, min(32, p.vocab - v0), min(64, p.cols - n));
    __syncwarp();
  }
}

// Added to the pieces before: w columns of 32 rows, blocks of 32 x 32 from `acc` on, laid
// out so that a lane's 16 bytes lie beside the next one's.
__device__ __forceinline__ void take_dx(const TileParams &p, uint32_t tmem, float *acc, int w, bool empty) {
  const int lane = threadIdx.x & 31;
  if (empty && !p.first) return;
#pragma unroll 1
  for (int c = 0; c < w; c += 32) {
    float4 *to = reinterpret_cast<float4 *>(acc + c * 32) + lane;
    float4 sum[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) sum[k] = p.first ? make_float4(0.f, 0.f, 0.f, 0.f) : to[k * 32];
    uint32_t v[32];
    tmem_ld_32cols(tmem + (uint32_t)c, v);
    tmem_ld_wait();
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (!empty) {
        sum[k].x += __uint_as_float(v[4 * k]), sum[k].y += __uint_as_float(v[4 * k + 1]);
        sum[k].z += __uint_as_float(v[4 * k + 2]), sum[k].w += __uint_as_float(v[4 * k + 3]);
      }
      to[k * 32] = sum[k];
    }
  }
}

// What the gather does, for few rows that stay where they lie, by the warps that take
// tiles out: the largest |dloss| (for each warp by itself), and this CTA's share of x with zeros
// for the rows that do not count, which dW's product adds up times g's zeros (they may hold
// anything).
__device__ __forceinline__ float gain_of_few(const TileParams &p) {
  float top = 0.f;
  for (int i = threadIdx.x & 31; i < p.rows; i += 32)
    if (target_of(p, i) >= 0) {
      const float d = abs_weight(p.dloss, i);
      if (d <= kLargestFinite) top = fmaxf(top, d);
    }
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  return top == 0.f ? 1.f : top;
}
__device__ __forceinline__ void copy_few(const TileParams &p, int cta, int ctas, int t) {
  const int64_t pieces = p.r.ldx / 8, all = (p.rows + 63) / 64 * 64 * pieces;
  for (int64_t i = cta * 256 + t; i < all; i += ctas * 256) {
    const int row = (int)(i / pieces);
    const int64_t c = i - row * pieces;
    RowPiece<2> v;
    const int source = row & (p.low - 1);  // (where p.low is 32 the rows stand twice)
    const uint8_t *from = static_cast<const uint8_t *>(p.x) + (int64_t)source * p.ldx * 2;
    const bool live = target_of(p, source) >= 0;
    if (live) v.load(from, (int64_t)p.cols * 2, c * 16);
    reinterpret_cast<uint4 *>(p.r.x)[i] = live ? v.value(from, (int64_t)p.cols * 2, c * 16) : make_uint4(0, 0, 0, 0);
  }
}

template <int MODE, int CG>
__global__ void __launch_bounds__(tile_threads(MODE, CG), 1)
    tile_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                const __grid_constant__ CUtensorMap tmBh, const __grid_constant__ CUtensorMap tmO,
                const TileParams p) {
  using R = Ring<MODE, CG>;
  // (DX of few rows: both of g's values)
  constexpr int kAParts = MODE == MODE_DX && CG == 1 ? 2 : 1;
  const int a_rows = CG == 1 ? p.a_rows : 128;
  const uint32_t a_bytes = (uint32_t)(kAParts * a_rows) * 128, stage_bytes = a_bytes + R::kB;
  const int S = CG == 1 ? R::stages(kAParts * a_rows, 1) : MODE == MODE_DW ? R::stages(128, p.boxes) : R::stages(128, 1);
  constexpr bool kMnA = is_dw(MODE), kMnB = MODE == MODE_DX || is_dw(MODE);
  // blocks of K that an accumulator holds (0: all)
  constexpr int kChunk = MODE == MODE_LSE || MODE == MODE_G ? kChunkKb : MODE == MODE_DW_LONG ? kLongChunkKb : 0;
  pdl_launch_dependents();
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  uint8_t *boxes = smem + kBarBytes, *ring = boxes + R::front(MODE == MODE_DW ? p.boxes : 1);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem);
  const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * R::kMaxStages;
  const uint32_t tfull0 = empty0 + 8 * R::kMaxStages, tempty0 = tfull0 + 16, drain = tempty0 + 16, stall = drain + 8;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 2 * R::kMaxStages + 6);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pos = CG == 2 ? (int)cluster_ctarank() : 0;
  const bool leader = pos == 0;
  const int cid = (int)blockIdx.x / CG, ncl = (int)gridDim.x / CG;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull0 + 8 * a, 1);
      mbar_init(tempty0 + 8 * a, 8 * CG);
    }
    mbar_init(drain, 1);
    mbar_init(stall, 1);
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmB);
    prefetch_tmap(&tmBh);
    if (R::kHasBoxes && (!is_dw(MODE) || p.vec)) prefetch_tmap(&tmO);
  }
  // the blocks of K of a unit
  const auto k_of = [&](const Tiles &tiles, int num_kb, const Unit &u, int i, int &kb0) {
    kb0 = 0;
    if (MODE != MODE_DX || i < tiles.full) return num_kb;
    const int per = (num_kb + tiles.parts - 1) / tiles.parts;
    kb0 = u.part * per;
    return max(0, min(per, num_kb - kb0));
  };
  if (MODE == MODE_LSE && CG == 1 && warp == 0 && lane == 0) {
    // few rows: the first blocks of W into L2 while the kernel before still runs (one row
    // tile, so the first unit does not depend on the rows that count).  16 x 4096 x 32000:
    // none 48.5 us, 8 blocks 47.4, 16 46.7.  Backward, where products of W follow one another,
    // it gains nothing there (164.4 us without, 164.6 with) and loses where W stays in L2: 64 x
    // 1024 x 32000 82.4 and 88.5.
    const Tiles tiles = tiles_of(1, 128, p.tiles_n, p.bn, p.places);
    if (cid < tiles.total) {
      const Unit u = unit_at(tiles, p.bn, cid);
      for (int kb = 0; kb < min(p.num_kb, 16); ++kb) tma_prefetch_2d(u.w == p.bn ? &tmB : &tmBh, kb * 64, u.n0);
    }
  }
  if (warp == 1) tmem_alloc<CG>(smem_u32(tmem_slot), 512);
  fence_before();
  if (CG == 2) cluster_sync_all();
  else __syncthreads();
  fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const uint32_t leader_full0 = CG == 2 ? map_to_rank(full0, 0) : full0;
  const uint32_t leader_tempty0 = CG == 2 ? map_to_rank(tempty0, 0) : tempty0;
  pdl_wait();
  const int rows = row_count(p.r, p.rows);
  const Tiles tiles = tiles_of(is_dw(MODE) ? p.width : rows, 128 * CG, p.tiles_n, p.bn, p.places,
                               MODE == MODE_DX ? max_parts_of(p.piece_kb) : 0);
  const int num_kb = is_dw(MODE) ? (rows + 63) / 64 * (p.low > 64 ? 2 : 1) : p.num_kb;
  // DW of many rows: where the targets of a unit's tile of tokens are, whose cells are more
  // blocks of K (see leave_rest); read a unit ahead
  const auto targets_of = [&](int i) {
    if (!is_dw(MODE) || !p.r.first || i >= tiles.total) return make_int2(0, 0);
    const int *first = p.r.first + (p.v0 >> kLogTileTokens) + unit_at(tiles, p.bn, i).tm;
    return make_int2(first[0], first[1]);
  };
  const auto cells_of = [](int2 at) { return at.y > at.x ? ((at.y - 1) >> 6) - (at.x >> 6) + 1 : 0; };
  if (warp == 0) {
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    int2 next = targets_of(cid);
    for (int i = cid; i < tiles.total && ok; i += ncl) {
      const Unit u = unit_at(tiles, p.bn, i);
      const int2 at = next;
      next = targets_of(i + ncl);
      int kb0;
      const int nk = k_of(tiles, num_kb, u, i, kb0), nh = u.w / CG, m0 = u.tm * 128 * CG + pos * 128, n0 = u.n0 + pos * nh;
      const int end = kb0 + nk + cells_of(at), to_cells = (at.x >> 6) - nk, tile = (p.v0 >> kLogTileTokens) + u.tm;
      for (int kb = kb0; kb < end; ++kb) {
        if (!warp_wait(empty0 + 8 * stage, phase ^ 1, abort_flag, p.wait, kErrCopy)) {
          ok = false;
          break;
        }
        const uint32_t sa = smem_u32(ring + stage * stage_bytes), sb = sa + a_bytes, bar = leader_full0 + 8 * stage;
        if (leader) mbar_expect_tx(full0 + 8 * stage, (uint32_t)(CG * (kAParts * a_rows + nh)) * 128);
        // (dW of few rows: both of g's values, one after the other along K)
        const bool low = MODE == MODE_DW && p.low > 64 && 2 * kb >= num_kb;
        const bool rest = is_dw(MODE) && kb >= nk;  // (of a cell)
        const int xb = low ? kb - num_kb / 2 : rest ? kb + to_cells : kb;
        if (kMnA) {
          const CUtensorMap *ma = rest ? &tmBh : &tmA;
          const int xa = rest ? pos * 128 : m0, ya = (low ? p.low : 0) + (rest ? xb + tile : xb) * 64;
          for (int j = 0; j < 2; ++j) load_box<CG>(sa + j * 8192, ma, bar, xa + j * 64, ya);
        } else {
          load_box<CG>(sa, &tmA, bar, kb * 64, m0);
          if (kAParts == 2) load_box<CG>(sa + a_rows * 128, &tmA, bar, kb * 64, p.low);
        }
        if (!kMnB) load_box<CG>(sb, u.w == p.bn ? &tmB : &tmBh, bar, kb * 64, n0);
        else
          for (int j = 0; j < nh / 64; ++j) load_box<CG>(sb + j * 8192, &tmB, bar, n0 + j * 64, xb * 64);
        if (++stage == S) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    if (leader)  // the copies (of both CTAs) have landed
      for (int s = 0; s < S; ++s) {
        const int st = (stage + s) % S;
        wait_drain(full0 + 8 * st, st < stage ? phase : phase ^ 1, p.wait, kErrCopy);
      }
    __syncwarp();
  } else if (warp == 1) {
    if (leader) {
      constexpr uint64_t kDescA = kMnA ? kDescMnMajor128 : kDescKMajor128;
      constexpr uint64_t kDescB = kMnB ? kDescMnMajor128 : kDescKMajor128;
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = !p.wait.stall || warp_wait(stall, 0, abort_flag, p.wait, kErrMma);  // (test hook)
      const auto finish = [&] {  // the accumulator is handed on when the MMAs so far are done
        if (CG == 2) mma_commit_pair(tfull0 + 8 * acc);
        else mma_commit<1>(tfull0 + 8 * acc);
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1;
        }
      };
      int2 next = targets_of(cid);
      for (int i = cid; i < tiles.total && ok; i += ncl) {
        const Unit u = unit_at(tiles, p.bn, i);
        const int2 at = next;
        next = targets_of(i + ncl);
        int kb0;
        const int nk = k_of(tiles, num_kb, u, i, kb0) + cells_of(at);
        const uint32_t idesc = instr_desc(p.tx == MM_BF16, 128 * CG, (uint32_t)u.w) | (kMnA ? kMnMajorA : 0u) |
                               (kMnB ? kMnMajorB : 0u);
        uint32_t d = 0;
        for (int k = 0; k < max(nk, 1); ++k) {
          // an accumulator for the tile, or for each chunk of K
          const bool start = k == 0 || (kChunk && k % max(kChunk, 1) == 0);
          if (start) {
            if (!warp_wait(tempty0 + 8 * acc, acc_phase ^ 1, abort_flag, p.wait, kErrMma)) {
              ok = false;
              break;
            }
            fence_after();
            d = tmem_base + (uint32_t)(acc * 256);
          }
          if (nk == 0) {
            finish();
            break;
          }
          if (!warp_wait(full0 + 8 * stage, phase, abort_flag, p.wait, kErrMma)) {
            ok = false;
            break;
          }
          fence_after();
          const uint32_t sa = smem_u32(ring + stage * stage_bytes);
          const uint64_t ad = kDescA | (uint64_t)((sa >> 4) & 0x3FFFu);
          const uint64_t bd = kDescB | (uint64_t)(((sa + a_bytes) >> 4) & 0x3FFFu);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_f16<CG>(d, ad + (kMnA ? 128 : 2) * kk, bd + (kMnB ? 128 : 2) * kk, idesc, (!start || kk > 0) ? 1u : 0u);
          if constexpr (kAParts == 2) {
            const uint64_t al = ad + (uint64_t)(a_rows * 128 >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) mma_f16<CG>(d, al + 2 * kk, bd + 128 * kk, idesc, 1u);
          }
          if (CG == 2) mma_commit_pair(empty0 + 8 * stage);
          else mma_commit<1>(empty0 + 8 * stage);
          if (++stage == S) {
            stage = 0;
            phase ^= 1;
          }
          if (k + 1 == nk || (kChunk && (k + 1) % max(kChunk, 1) == 0)) finish();
        }
      }
      mma_commit<CG>(drain);
      wait_drain(drain, 0, p.wait, kErrDrain);
    }
    __syncwarp();
  } else {
    // q: the TMEM lanes this warp may read; half: its half of a tile's columns; team: of the
    // two that take turns, each with an accumulator of its own
    constexpr int kTeams = R::kTeams;
    const int q = warp & 3, half = (warp - 2) >> 2 & 1, team = (warp - 2) >> 3;
    const int box_count = MODE == MODE_DW ? p.boxes : 1;
    Boxes mine{boxes + (warp - 2) * box_count * (int)kBoxB, box_count, 0};
    float gain = 0.f;
    if (is_dw(MODE)) gain = *p.r.gain * (p.tx == MM_F16 ? 1.f / kF16Gain : 1.f);
    bool copy = MODE == MODE_G && CG == 1 && !p.r.count;
    if (copy) {
      gain = gain_of_few(p);
      if (cid == 0 && threadIdx.x == 64) *p.r.gain = gain;
    }
    int acc = team;
    uint32_t acc_phase = 0;
    const auto release = [&] {  // the accumulator has been read
      fence_before();
      __syncwarp();
      if (lane == 0) {
        if (CG == 2) mbar_arrive_cluster(leader_tempty0 + 8 * acc);
        else mbar_arrive(tempty0 + 8 * acc);
      }
      if (kTeams == 2 || ++acc == 2) {
        acc = team;
        acc_phase ^= 1;
      }
    };
    bool ok = true;
    int turn = 0;
    for (int i = cid + team * ncl; i < tiles.total && ok; i += kTeams * ncl, turn ^= 1) {
      const Unit u = unit_at(tiles, p.bn, i);
      const int row0 = u.tm * 128 * CG + pos * 128 + q * 32;
      const int lower = u.w > 128 ? 128 : u.w / 2, c0 = half ? lower : 0, wide = half ? u.w - lower : lower, n = u.n0 + c0;
      const uint32_t lanes = tmem_base + ((uint32_t)(q * 32) << 16);
      if constexpr (kChunk > 0) {
        const int left = min(wide, (MODE == MODE_G ? p.width : p.v0 + row0 < p.vocab ? p.cols : 0) - n);  // (G, DW)
        const bool live = MODE == MODE_LSE ? row0 < rows && u.n0 < p.vocab  // (else a half tile past the end)
                                           : left > 0 && (CG == 2 || row0 < p.low);
        float l[128];
        GRow r{};
        if (MODE == MODE_G) r = g_row(p, row0 + lane, gain);  // (read while the tile is waited for)
        bool good = true;
        int nk = num_kb;
        if (MODE == MODE_DW_LONG) nk += cells_of(targets_of(i));
        for (int k = 0; k < nk; k += kChunk) {
          if (!(good = warp_wait(tfull0 + 8 * acc, acc_phase, abort_flag, p.wait, kErrStore))) break;
          fence_after();
          if (live) add_chunk(l, lanes + (uint32_t)(acc * 256 + c0), wide, k == 0);
          release();
          if (copy && (k > 0 || nk <= kChunk)) {  // (the first two chunks come from L2)
            copy_few(p, cid, ncl, (int)threadIdx.x - 64);
            copy = false;
          }
        }
        if constexpr (MODE != MODE_LSE) {
          if (!good) break;
          if (!live) continue;
          // the sums move down as columns are taken, so that the code for those is there once
          // (800 x 1000 x 50264 118 -> 100 us of this kernel)
          constexpr int W = CG == 1 ? 32 : 64;
#pragma unroll 1
          for (int c = 0; c < left; c += W) {
            uint32_t v[W / 32][32];
#pragma unroll
            for (int k = 0; k < W; ++k) v[k / 32][k % 32] = __float_as_uint(l[k]);
            if constexpr (MODE == MODE_DW_LONG) leave_dw(p, &tmO, v, n + c, p.v0 + row0, mine, gain);
            else if constexpr (CG == 1) leave_g_few(p, r, v[0], n + c, row0 + lane);  // (rows from p.low on are the second values')
            else leave_g(p, &tmO, r, v, n + c, row0, mine);
#pragma unroll
            for (int k = 0; k + W < 128; ++k) l[k] = l[k + W];
          }
        } else {
          // the upper half's sums to the lower half's warps; a buffer for each of two turns
          float2 *upper = reinterpret_cast<float2 *>(boxes) + turn * 128 + q * 32 + lane;
          float2 sum = make_float2(kLeast, 0.f);
          if (live && good) {
            const int row = row0 + lane;
            sum = sum_exp(p, l, n, wide, target_of(p, row), p.hit + row);
            if (half) *upper = sum;
          }
          if (!(ok = all_take(good))) break;  // the eight warps go on or give up together
          if (live && !half) p.part[(int64_t)(u.n0 >> 7) * p.r.rows_pad + row0 + lane] = join_sums(sum, *upper);
        }
      } else {
        if (!warp_wait(tfull0 + 8 * acc, acc_phase, abort_flag, p.wait, kErrStore)) break;
        fence_after();
        const uint32_t tmem = lanes + (uint32_t)(acc * 256 + c0);
        int kb0;
        if constexpr (MODE == MODE_DX) {
          // (columns past cols stay unwritten: nothing reads them)
          const int w = min(wide, (p.cols - n + 31) / 32 * 32);
          float *acc_at =
              i < tiles.full ? p.acc + ((int64_t)(row0 >> 5) * p.acc_cols + (n >> 5)) * 1024
                             : p.acc_cut + (int64_t)(i - tiles.full) * (128 * CG * p.bn) +
                                   ((pos * 4 + q) * (p.bn / 32) + c0 / 32) * 1024;
          if (row0 < rows && w > 0) take_dx(p, tmem, acc_at, w, k_of(tiles, num_kb, u, i, kb0) == 0);
          release();
        } else {
          const int end = MODE == MODE_G_ONE ? p.width : p.v0 + row0 < p.vocab ? p.cols : 0;
          const int left = min(wide, end - n);
          if (left <= 0) release();
          for (int c = 0; c < left; c += 64) {
            uint32_t v[2][32];
            tmem_ld_32cols(tmem + (uint32_t)c, v[0]);
            tmem_ld_32cols(tmem + (uint32_t)(c + 32), v[1]);
            tmem_ld_wait();
            if (c + 64 >= left) release();
            if constexpr (MODE == MODE_G_ONE) leave_g(p, &tmO, g_row(p, row0 + lane, 0.f), v, n + c, row0, mine);
            else leave_dw(p, &tmO, v, n + c, p.v0 + row0, mine, gain);
          }
        }
      }
    }
    if (copy) copy_few(p, cid, ncl, (int)threadIdx.x - 64);  // (a CTA without a tile)
    if (lane == 0) tma_store_wait_all();
    __syncwarp();
  }
  fence_before();
  __syncthreads();
  if (CG == 2) {
    if (*abort_flag) {  // the other CTA's copies into this one may still be landing
      const uint64_t t0 = global_ns();
      while (global_ns() - t0 < 100000ull) __nanosleep(1000);
    }
    cluster_sync_all();  // the leader's MMAs read both CTAs' memory
  }
  fence_after();
  if (warp == 1) tmem_dealloc<CG>(tmem_base, 512);
}

// ---------------------------------------------------------------- loss and dx by row
struct LossParams {
  LossArgs a;
  Rows r;
  const float2 *part;
  const float *hit;
  int tile_m, bn, tiles_n, places;  // of the product
};

// 32 rows a block, 32 threads a row over the tiles of the vocabulary.  (In fp64 the
// logarithm of 32 rows took 10 us; 8192 rows of 512 tiles now 17.)
constexpr int kLossThreads = 1024;
__global__ void __launch_bounds__(kLossThreads) loss_kernel(const LossParams p) {
  pdl_launch_dependents();
  pdl_wait();
  constexpr int Y = kLossThreads / 32, U = 4;
  __shared__ float2 sh[Y][33];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int64_t row = (int64_t)blockIdx.x * 32 + x;
  // where a row's sums are, or -1
  const auto slot_of = [&](int64_t i) {
    if (p.r.count) return p.r.slot[i];
    return valid_target(p.a, i) < 0 ? -1 : (int)i;
  };
  const int slot = row < p.a.rows ? slot_of(row) : -1;
  const Tiles tiles = tiles_of(row_count(p.r, p.a.rows), p.tile_m, p.tiles_n, p.bn, p.places);
  const float2 none = make_float2(kLeast, 0.f);
  float2 sum = none;
  if (slot >= 0) {
    // a slot for each 128 of the vocabulary; a tile has left its sums in the first of
    // its slots, the second half of a cut one in its own
    for (int i0 = y; i0 < p.tiles_n; i0 += Y * U) {
      float2 v[U][2];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * Y;
        const float2 *part = p.part + ((int64_t)i * p.bn >> 7) * p.r.rows_pad + slot;
        v[u][0] = i < p.tiles_n ? part[0] : none;
        v[u][1] = i < p.tiles_n && p.bn == 256 && i * 256 + 128 < p.a.vocab && tile_at(tiles, slot / p.tile_m, i) >= tiles.full
                      ? part[p.r.rows_pad]
                      : none;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) sum = join_sums(join_sums(sum, v[u][0]), v[u][1]);
    }
  }
  sh[y][x] = sum;
  __syncthreads();
  // the 32 sums of a row by a warp
  const float2 mine = sh[x][y];
  float m = mine.x;
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float s = mine.y * exp_fast(mine.x - m);
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const int64_t to = (int64_t)blockIdx.x * 32 + y;
  if (x != 0 || to >= p.a.rows) return;
  const int at = slot_of(to);
  const float rest = logf(s);
  p.a.loss[to] = at < 0 ? 0.f : (m - p.hit[at]) + rest;
  if (p.a.lse) p.a.lse[to] = at < 0 ? 0.f : m + rest;
}

struct DxParams {
  LossArgs a;
  Rows r;
  const float *acc, *acc_cut;
  const uint8_t *w;  // W, rows on 16 bytes ...
  int64_t ldw;       // ... this far apart
  int tile_m, bn, tiles_n, places, piece_kb, acc_cols;  // of the product
  int vec;  // dx's rows start on 16 bytes
};
// 32 rows, a row a lane, by 4 Q columns from `col` on: the parts (part_at apart) added in
// order, U of them read at once, scaled and rounded.
template <int Q, int U>
__device__ __forceinline__ void round_dx(const DxParams &p, const float4 *from, int parts, int64_t part_at, int rb, int col,
                                         int count, float gain) {
  const int i = rb * 32 + (threadIdx.x & 31), left = p.a.cols - col;
  const float rest = p.r.rest && i < count ? p.r.rest[i] : 0.f;  // (see leave_rest)
  const int token = p.r.rest && i < count ? p.r.target[i] : 0;
  float4 v[Q];
#pragma unroll
  for (int k = 0; k < Q; ++k) v[k] = from[k * 32];
  uint32_t row[2 * Q];
  if (rest != 0.f) {
    const uint16_t *from_w = reinterpret_cast<const uint16_t *>(p.w + (int64_t)token * p.ldw) + col;
#pragma unroll
    for (int k = 0; k < Q / 2; ++k) {
      if (8 * k + 8 <= left) {
        const uint4 u = reinterpret_cast<const uint4 *>(from_w)[k];
        row[4 * k] = u.x, row[4 * k + 1] = u.y, row[4 * k + 2] = u.z, row[4 * k + 3] = u.w;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int c = 8 * k + 2 * e;
          row[4 * k + e] = (c < left ? from_w[c] : 0u) | (c + 1 < left ? (uint32_t)from_w[c + 1] << 16 : 0u);
        }
      }
    }
  }
  for (int s = 1; s < parts; s += U) {
    float4 w[U][Q];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < Q; ++k)
        w[u][k] = s + u < parts ? from[(s + u) * part_at + k * 32] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < Q; ++k)
        v[k].x += w[u][k].x, v[k].y += w[u][k].y, v[k].z += w[u][k].z, v[k].w += w[u][k].w;
  }
  if (i >= count || (!p.r.count && valid_target(p.a, i) < 0)) return;
  if (rest != 0.f) {
#pragma unroll
    for (int k = 0; k < Q; ++k) {
      v[k].x = fmaf(rest, unpack(p.a.tx, row[2 * k], 0), v[k].x), v[k].y = fmaf(rest, unpack(p.a.tx, row[2 * k], 1), v[k].y);
      v[k].z = fmaf(rest, unpack(p.a.tx, row[2 * k + 1], 0), v[k].z), v[k].w = fmaf(rest, unpack(p.a.tx, row[2 * k + 1], 1), v[k].w);
    }
  }
  uint32_t w[2 * Q];
#pragma unroll
  for (int k = 0; k < Q; ++k) {
    w[2 * k] = pack2(p.a.tx, v[k].x * gain, v[k].y * gain);
    w[2 * k + 1] = pack2(p.a.tx, v[k].z * gain, v[k].w * gain);
  }
  uint16_t *to = static_cast<uint16_t *>(p.a.dx) + (int64_t)(p.r.count ? p.r.row[i] : i) * p.a.lddx + col;
  if (p.vec && left >= 4 * Q) {
#pragma unroll
    for (int k = 0; k < Q / 2; ++k)
      reinterpret_cast<uint4 *>(to)[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
  } else {
#pragma unroll
    for (int e = 0; e < 4 * Q; ++e)
      if (e < left) to[e] = (uint16_t)(w[e >> 1] >> (e & 1) * 16);
  }
}
// A warp 32 x 32 of the whole tiles' sums (64 bytes of a row), neighbouring warps
// neighbouring blocks, row block by row block; then 32 x 8 of the cut tiles', whose many
// parts want more warps; then the rows that do not count.  (6144 x 4096: 33 us; the
// sums tile by tile 55; a tile's columns a warp, accesses 32 KB apart, 200.)
__global__ void __launch_bounds__(256, 4) dx_kernel(const DxParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, count = live_rows(p.r, p.a.rows);  // (0: r.row holds nothing)
  const float gain = *p.r.gain * (p.a.tx == MM_F16 ? 1.f / kF16Gain : 1.f);
  const uint32_t warps = gridDim.x * 8, warp = blockIdx.x * 8 + (threadIdx.x >> 5);
  const Tiles tiles = tiles_of(max(1, count), p.tile_m, p.tiles_n, p.bn, p.places, max_parts_of(p.piece_kb));
  const int log_rows = p.tile_m == 256 ? 3 : 2, log_cols = p.bn == 256 ? 3 : 2;  // blocks of 32 a tile
  if (tiles.full > 0) {
    // (as many blocks as there are 4 KB of sums: they count in 32 bits)
    const uint32_t blocks = (uint32_t)((count + 31) / 32) * (uint32_t)p.acc_cols;
    for (uint32_t b = warp; b < blocks; b += warps) {
      const int rb = (int)(b / (uint32_t)p.acc_cols), cb = (int)(b - (uint32_t)rb * (uint32_t)p.acc_cols);
      if (tile_at(tiles, rb >> log_rows, cb >> log_cols) < tiles.full)
        round_dx<8, 1>(p, reinterpret_cast<const float4 *>(p.acc) + (int64_t)b * 256 + lane, 1, 0, rb, cb * 32, count, gain);
    }
  }
  const int log_strips = log_cols + 2, log_units = log_rows + log_strips;
  const uint32_t cut = (uint32_t)(tiles.tiles_m * tiles.tiles_n - tiles.full) << log_units;
  for (uint32_t b = warp; b < cut; b += warps) {
    const int t = (int)(b >> log_units), r = (int)(b >> log_strips) & ((1 << log_rows) - 1);
    const int strip = (int)b & ((1 << log_strips) - 1);
    const Unit u = unit_at(tiles, p.bn, tiles.full + t * tiles.parts);
    const int rb = (u.tm << log_rows) + r, col = u.n0 + strip * 8;
    if (rb * 32 >= count || col >= p.a.cols) continue;
    const float4 *from = reinterpret_cast<const float4 *>(p.acc_cut) + (int64_t)t * tiles.parts * p.tile_m * p.bn / 4 +
                         ((r << log_cols) + (strip >> 2)) * 256 + (strip & 3) * 64 + lane;
    round_dx<2, 4>(p, from, tiles.parts, (int64_t)p.tile_m * p.bn / 4, rb, col, count, gain);
  }
  uint16_t *dx = static_cast<uint16_t *>(p.a.dx);
  for (int64_t row = warp; row < p.a.rows; row += warps)
    if (p.r.count ? p.r.slot[row] < 0 : valid_target(p.a, row) < 0)
      for (int c = lane; c < p.a.cols; c += 32) dx[row * p.a.lddx + c] = 0;
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

int token_tiles(int vocab) { return (int)keys_of(vocab, kLogTileTokens); }
int64_t cell_count(const Rows &r, int vocab) { return r.rows_pad / kCellRows + token_tiles(vocab); }
Rows cut_rows(Cut &cut, const LossArgs &a, bool backward, bool direct) {
  Rows r;
  std::memset(&r, 0, sizeof r);
  r.rows_pad = (a.rows + kRowTile - 1) / kRowTile * kRowTile;
  r.ldx = ((int64_t)a.cols + 7) / 8 * 8;
  r.gain = cut.take<float>(1);
  if (direct) {
    if (backward) r.x = cut.take<uint16_t>(128 * r.ldx);
    return r;
  }
  r.count = cut.take<int>(1);
  r.slot = cut.take<int>(a.rows);
  r.row = cut.take<int>(a.rows);
  r.target = cut.take<int>(r.rows_pad);
  if (backward) {
    r.ratio = cut.take<float>(r.rows_pad);
    r.lse = cut.take<float>(r.rows_pad);
  }
  r.x = cut.take<uint16_t>((int64_t)r.rows_pad * r.ldx);
  return r;
}

// (sorted, of many rows: room for twice as many (tile, row) as there are rows, where they are
// not counted)
mm_status launch_gather(const LossArgs &a, const Rows &r, bool backward, const PackRows &pack, uint2 *sorted, LaunchCtx &ctx) {
  const int sms = ctx.dev->info.sms;
  GatherParams p{a, r, backward, 0, std::min(a.rows, std::max(2 * sms, kCountedRows / kGatherThreads)), pack};
  while (p.log_threads < 9 && (32ll << p.log_threads) < r.ldx) ++p.log_threads;  // (up to four pieces each)
  const PackShape copy = pack_shape(pack.rows, pack.ld16, kGatherThreads, 8 * sms);
  p.pack.log_threads = copy.log_threads;
  const dim3 grid((unsigned)(p.blocks + copy.blocks));
  cudaError_t e;
  if (r.cells) {  // (a block's rows: no more than its threads)
    const SortedParams q{p, sorted, token_tiles(a.vocab), cell_count(r, a.vocab) * kCellRows * kTileTokens / 8};
    if (sorted) {
      mm_status st = sort_tokens({a.targets, a.ti, a.vocab, a.rows, kLogTileTokens, sorted, sorted + a.rows}, ctx);
      if (st != MM_OK) return st;
      e = launch_pdl(gather_sorted_kernel, grid, dim3(kGatherThreads), 0, ctx.stream, dim3(1), q);
    } else {
      e = launch_pdl(gather_counted_kernel, grid, dim3(kGatherThreads), 0, ctx.stream, dim3(1), q);
    }
  } else {
    e = launch_pdl(gather_kernel, grid, dim3(kGatherThreads), 0, ctx.stream, dim3(1), p);
  }
  if (e != cudaSuccess) return cuda_error(e, "cross_entropy launch (gather)");
  count_operator_launch();
  return MM_OK;
}

// The maps of a product's operands: rows of 16-bit elements, in boxes of 64 elements
// (128 bytes, swizzled) by `box_rows`.
mm_status rows_map(CUtensorMap *map, int tx, const void *p, int64_t cols, int64_t rows, int64_t ld, int box_rows) {
  return encode_map_2d(map, tx == MM_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, p,
                       (uint64_t)cols, (uint64_t)rows, (uint64_t)ld * 2, 64, (uint32_t)box_rows,
                       CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int MODE, int CG>
cudaLaunchConfig_t tile_config(int grid, cudaStream_t s, cudaLaunchAttribute *at) {
  at->id = cudaLaunchAttributeClusterDimension;
  at->val.clusterDim.x = CG;
  at->val.clusterDim.y = at->val.clusterDim.z = 1;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)grid);
  lc.blockDim = dim3(tile_threads(MODE, CG));
  lc.dynamicSmemBytes = Ring<MODE, CG>::kSmem;
  lc.stream = s;
  lc.attrs = at;
  lc.numAttrs = 1;
  return lc;
}
// Set-up once a device, and how many pairs (or CTAs) run at once.
template <int MODE, int CG>
mm_status tile_places(LaunchCtx &ctx, int *places) {
  static PerDevice<int> fits;
  const cudaError_t err = fits.get(ctx.dev->info.ordinal, places, [](int *n) -> cudaError_t {
    cudaError_t e = cudaFuncSetAttribute(tile_kernel<MODE, CG>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)Ring<MODE, CG>::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute at;
    const cudaLaunchConfig_t lc = tile_config<MODE, CG>(CG, nullptr, &at);
    return cudaOccupancyMaxActiveClusters(n, tile_kernel<MODE, CG>, &lc);
  });
  if (err != cudaSuccess) return cuda_error(err, "cross_entropy set-up");
  if (*places < 1) return set_error(MM_ERR_UNSUPPORTED, "no tile of cross_entropy fits on this device");
  return MM_OK;
}

// A form of the products: few rows on single SMs.
struct Form {
  int cg;      // 1 or 2
  int a_rows;  // of A that a CTA loads
  int tile_m() const { return 128 * cg; }
};
Form form_of(int rows) {
  return rows > 128 ? Form{2, 128} : Form{1, rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128};
}

struct Maps {
  CUtensorMap a, b, bh, o;
};

// M, N: the product's (M as if every row counted).
template <int MODE, int CG>
mm_status launch_tiles(TileParams &p, const Maps &m, int64_t M, LaunchCtx &ctx) {
  mm_status st = tile_places<MODE, CG>(ctx, &p.places);
  if (st != MM_OK) return st;
  const int64_t tiles = (M + 128 * CG - 1) / (128 * CG) * p.tiles_n;
  if (tiles >= 1 << 30) return set_error(MM_ERR_UNSUPPORTED, "too many tiles");
  const int grid = CG * (int)std::min<int64_t>(MODE == MODE_DX ? p.places : p.bn == 256 ? 2 * tiles : tiles, p.places);
  cudaError_t e = launch_pdl(tile_kernel<MODE, CG>, dim3((unsigned)grid), dim3(tile_threads(MODE, CG)), Ring<MODE, CG>::kSmem, ctx.stream,
                             dim3(CG), m.a, m.b, m.bh, m.o, p);
  if (e != cudaSuccess) return cuda_error(e, "cross_entropy launch");
  count_operator_launch();
  return MM_OK;
}
template <int MODE>
mm_status launch_tiles(Form f, TileParams &p, const Maps &m, int64_t M, LaunchCtx &ctx) {
  return f.cg == 1 ? launch_tiles<MODE, 1>(p, m, M, ctx) : launch_tiles<MODE, 2>(p, m, M, ctx);
}

// Width of a product's tiles along N.
int tile_width(int64_t N) { return N <= 128 ? 128 : 256; }

// The same for few rows, whose products read W once: the SMs' shares as equal as tiles
// of a multiple of 32 make them (32000 tokens: 143 tiles of 224 on 152 SMs, 125 of 256).
int tile_width_few(int64_t N, int places) {
  int best = 256;
  int64_t least = INT64_MAX;
  for (int w = 256; w >= 128; w -= 32) {
    const int64_t tiles = (N + w - 1) / w, rem = tiles % places;
    // (the last wave's tiles are halved where that fits: w 256 only)
    const int64_t span = tiles / places * w + (rem == 0 ? 0 : w == 256 && 2 * rem <= places ? w / 2 : w);
    if (span < least) least = span, best = w;
  }
  return best;
}

// x W^T over `width` tokens from v0 on, LSE or G.
mm_status logits_maps(Maps *m, TileParams &p, Form f, const TmaRows &w, int places) {
  p.a_rows = f.a_rows;
  p.bn = f.cg == 1 ? tile_width_few(p.width, places) : tile_width(p.width);
  p.tiles_n = (p.width + p.bn - 1) / p.bn;
  p.num_kb = (p.cols + 63) / 64;
  const char *base = static_cast<const char *>(w.p) + (int64_t)p.v0 * w.ld;
  const int64_t tokens = std::min(p.width, p.vocab - p.v0);
  mm_status st;
  if (p.r.count && (st = rows_map(&m->a, p.tx, p.r.x, p.cols, p.r.rows_pad, p.r.ldx, f.a_rows)) != MM_OK) return st;
  if ((st = rows_map(&m->b, p.tx, base, p.cols, tokens, w.ld / 2, p.bn / f.cg)) != MM_OK) return st;
  return rows_map(&m->bh, p.tx, base, p.cols, tokens, w.ld / 2, p.bn / f.cg / 2);
}

// W where TMA can read it: in place, or to be copied (by pack).
mm_status place_weight(const LossArgs &a, TmaRows *w, PackRows *pack, LaunchCtx &ctx) {
  std::memset(pack, 0, sizeof *pack);
  *w = TmaRows{a.weight, a.ldw * 2, a.vocab, (int64_t)a.cols * 2};
  const int64_t ld16 = (w->bytes + 15) / 16 * 16;
  if (addressable(*w)) {
    if (a.vocab == 1) w->ld = ld16;  // (a distance that is never used, as maps want it)
    return MM_OK;
  }
  void *to = nullptr;
  mm_status st = get_scratch(ctx, SCRATCH_REPACK, (size_t)(ld16 * a.vocab), &to);
  if (st != MM_OK) return st;
  *pack = pack_job(w->p, w->ld, w->rows, w->bytes, to, ld16, 0);  // (shared out where it is launched)
  w->p = to;
  w->ld = ld16;
  return MM_OK;
}
// Few rows that TMA reads as they lie, and W too: see Rows.
bool is_direct(const LossArgs &a, Form f) {
  return f.cg == 1 && addressable(TmaRows{a.x, a.ldx * 2, a.rows, 0}) && addressable(TmaRows{a.weight, a.ldw * 2, a.vocab, 0});
}
mm_status direct_map(CUtensorMap *map, const LossArgs &a, Form f) {
  return rows_map(map, a.tx, a.x, a.cols, a.rows, a.rows == 1 ? ((int64_t)a.cols + 7) / 8 * 8 : a.ldx, f.a_rows);
}

TileParams tile_params(const LossArgs &a, LaunchCtx &ctx) {
  TileParams p;
  std::memset(&p, 0, sizeof p);
  p.cols = a.cols;
  p.vocab = a.vocab;
  p.tx = a.tx;
  p.x = a.x;
  p.targets = a.targets;
  p.lse = a.lse;
  p.dloss = a.dloss;
  p.ldx = a.ldx;
  p.ti = a.ti;
  p.rows = a.rows;
  p.wait = operator_waits(ctx);
  return p;
}

// No columns: every logit is 0.
__global__ void __launch_bounds__(256) flat_loss_kernel(const LossArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= a.rows) return;
  const float v = valid_target(a, i) >= 0 ? logf((float)a.vocab) : 0.f;
  a.loss[i] = v;
  if (a.lse) a.lse[i] = v;
}

}  // namespace

mm_status launch_cross_entropy(const LossArgs &a, LaunchCtx &ctx) {
  if (a.cols == 0 || a.vocab == 0) {
    cudaError_t e = launch_pdl(flat_loss_kernel, dim3((unsigned)((a.rows + 255) / 256)), dim3(256), 0, ctx.stream, dim3(1), a);
    if (e != cudaSuccess) return cuda_error(e, "cross_entropy launch (no products)");
    count_operator_launch();
    return MM_OK;
  }
  TileParams p = tile_params(a, ctx);
  const Form f = form_of(a.rows);
  const bool direct = is_direct(a, f);
  Cut cut;
  for (int pass = 0; pass < 2; ++pass) {
    cut.used = 0;
    p.r = cut_rows(cut, a, false, direct);
    p.hit = cut.take<float>(p.r.rows_pad);
    p.part = cut.take<float2>(((int64_t)a.vocab + 127) / 128 * p.r.rows_pad);
    if (pass == 0) {
      void *w = nullptr;
      mm_status st = get_scratch(ctx, SCRATCH_WORKSPACE, cut.used, &w);
      if (st != MM_OK) return st;
      cut.base = static_cast<char *>(w);
    }
  }
  mm_status st;
  TmaRows w;
  PackRows pack;
  Maps m;
  if ((st = place_weight(a, &w, &pack, ctx)) != MM_OK) return st;
  if (!direct && (st = launch_gather(a, p.r, false, pack, nullptr, ctx)) != MM_OK) return st;
  p.width = a.vocab;
  if ((st = logits_maps(&m, p, f, w, ctx.dev->info.sms)) != MM_OK) return st;
  if (direct && (st = direct_map(&m.a, a, f)) != MM_OK) return st;
  m.o = m.a;  // (none)
  if ((st = launch_tiles<MODE_LSE>(f, p, m, a.rows, ctx)) != MM_OK) return st;
  LossParams l{a, p.r, p.part, p.hit, f.tile_m(), p.bn, p.tiles_n, p.places};
  cudaError_t e = launch_pdl(loss_kernel, dim3((unsigned)((a.rows + 31) / 32)), dim3(kLossThreads), 0, ctx.stream, dim3(1), l);
  if (e != cudaSuccess) return cuda_error(e, "cross_entropy launch (loss)");
  count_operator_launch();
  return MM_OK;
}

mm_status launch_cross_entropy_backward(const LossArgs &a, LaunchCtx &ctx) {
  if (a.rows == 0) return write_zeros(a.dweight, a.lddw, a.vocab, a.cols, a.tx, ctx);
  if (a.vocab == 0) return write_zeros(a.dx, a.lddx, a.rows, a.cols, a.tx, ctx);
  TileParams p = tile_params(a, ctx);
  const Form f = form_of(a.rows);
  const int64_t rows_pad = ((int64_t)a.rows + kRowTile - 1) / kRowTile * kRowTile;
  // Pieces of the vocabulary of equal size, whole tiles, whose g takes kPieceBytes
  // at most (and at least one tile).
  constexpr int64_t kPieceBytes = 512ll << 20;
  const int64_t most = std::max<int64_t>(256, kPieceBytes / (rows_pad * 2) / 256 * 256);
  const int64_t pieces = (a.vocab + most - 1) / most;
  const int piece = (int)std::min(((a.vocab + pieces - 1) / pieces + 255) / 256 * 256, ((int64_t)a.vocab + 63) / 64 * 64);
  // dx: sums of all tiles, and of the parts of cut ones, at most one a place
  p.acc_cols = (a.cols + 31) / 32;
  const int bn_cols = tile_width(a.cols), tiles_cols = (a.cols + bn_cols - 1) / bn_cols;
  int dx_places = 0;
  mm_status st = f.cg == 1 ? tile_places<MODE_DX, 1>(ctx, &dx_places) : tile_places<MODE_DX, 2>(ctx, &dx_places);
  if (st != MM_OK) return st;
  const bool direct = is_direct(a, f), many = f.cg == 2;
  const bool sorts = many && a.rows > kCountedRows;
  if (sorts && (st = sort_ready(ctx)) != MM_OK) return st;
  Cut cut;
  uint16_t *g = nullptr;
  uint2 *sorted = nullptr;
  for (int pass = 0; pass < 2; ++pass) {
    cut.used = 0;
    p.r = cut_rows(cut, a, true, direct);
    g = cut.take<uint16_t>(rows_pad * piece);
    if (a.dx) {
      p.acc = cut.take<float>(rows_pad * p.acc_cols * 32);
      p.acc_cut = cut.take<float>((int64_t)dx_places * f.tile_m() * bn_cols);
    }
    if (many) {
      p.r.rest = cut.take<float>(p.r.rows_pad);
      p.r.first = cut.take<int>(token_tiles(a.vocab) + 1);
      p.r.cells = cut.take<uint16_t>(cell_count(p.r, a.vocab) * kCellRows * kTileTokens);
      if (sorts) sorted = cut.take<uint2>(2 * (int64_t)a.rows);
    }
    if (pass == 0) {
      void *w = nullptr;
      if ((st = get_scratch(ctx, SCRATCH_WORKSPACE, cut.used, &w)) != MM_OK) return st;
      cut.base = static_cast<char *>(w);
    }
  }
  TmaRows w;
  PackRows pack;
  if ((st = place_weight(a, &w, &pack, ctx)) != MM_OK) return st;
  p.dw = static_cast<uint16_t *>(a.dweight);
  p.lddw = a.lddw;
  p.vec = (uintptr_t)a.dweight % 16 == 0 && a.lddw % 8 == 0 && a.cols % 8 == 0 && a.lddw < (1LL << 37);
  if (!direct && (st = launch_gather(a, p.r, true, pack, sorted, ctx)) != MM_OK) return st;
  p.piece_kb = piece / 64;
  p.low = f.cg == 2 ? 0 : direct && a.rows <= kFewestRows ? kFewestRows : 128;
  p.boxes = p.low ? 2 : 1;
  p.g = g;
  p.ldg = piece;
  for (p.v0 = 0; p.v0 < a.vocab; p.v0 += piece) {
    Maps m;
    p.first = p.v0 == 0;
    p.width = std::min(piece, (a.vocab - p.v0 + 63) / 64 * 64);
    if ((st = logits_maps(&m, p, f, w, ctx.dev->info.sms)) != MM_OK) return st;
    if (direct && (st = direct_map(&m.a, a, f)) != MM_OK) return st;
    if ((st = rows_map(&m.o, p.tx, g, p.width, rows_pad, piece, 32)) != MM_OK) return st;
    if ((st = f.cg == 2 && p.num_kb <= kChunkKb ? launch_tiles<MODE_G_ONE, 2>(p, m, a.rows, ctx)
                                                : launch_tiles<MODE_G>(f, p, m, a.rows, ctx)) != MM_OK)
      return st;
    p.bn = bn_cols;
    p.tiles_n = tiles_cols;
    if (a.dx) {
      p.num_kb = p.width / 64;
      if ((st = rows_map(&m.a, p.tx, g, p.width, rows_pad, piece, f.a_rows)) != MM_OK) return st;
      if ((st = rows_map(&m.b, p.tx, static_cast<const char *>(w.p) + (int64_t)p.v0 * w.ld, a.cols,
                         std::min(p.width, a.vocab - p.v0), w.ld / 2, 64)) != MM_OK)
        return st;
      m.bh = m.o = m.b;  // (boxes of 64: the same for half tiles)
      if ((st = launch_tiles<MODE_DX>(f, p, m, a.rows, ctx)) != MM_OK) return st;
    }
    if (a.dweight) {
      if ((st = rows_map(&m.a, p.tx, g, p.width, rows_pad, piece, 64)) != MM_OK) return st;
      if ((st = rows_map(&m.b, p.tx, p.r.x, a.cols, direct ? 128 : rows_pad, p.r.ldx, 64)) != MM_OK) return st;
      m.bh = m.o = m.b;
      if (many && (st = rows_map(&m.bh, p.tx, p.r.cells, kTileTokens, cell_count(p.r, a.vocab) * kCellRows, kTileTokens, kCellRows)) != MM_OK)
        return st;
      if (p.vec && (st = rows_map(&m.o, p.tx, a.dweight, a.cols, a.vocab, a.vocab == 1 ? p.r.ldx : a.lddw, 32)) != MM_OK)
        return st;
      st = a.rows > kLongRows ? launch_tiles<MODE_DW_LONG, 2>(p, m, p.width, ctx) : launch_tiles<MODE_DW, 2>(p, m, p.width, ctx);
      if (st != MM_OK) return st;
    }
  }
  if (!a.dx) return MM_OK;
  DxParams d{a, p.r, p.acc, p.acc_cut, static_cast<const uint8_t *>(w.p), w.ld, f.tile_m(), bn_cols, tiles_cols, dx_places, p.piece_kb, p.acc_cols,
             (uintptr_t)a.dx % 16 == 0 && (a.lddx % 8 == 0 || a.rows == 1)};
  cudaError_t e = launch_pdl(dx_kernel, dim3((unsigned)(4 * ctx.dev->info.sms)),
                             dim3(256), 0, ctx.stream, dim3(1), d);
  if (e != cudaSuccess) return cuda_error(e, "cross_entropy_backward launch (dx)");
  count_operator_launch();
  return MM_OK;
}

}  // namespace mm
