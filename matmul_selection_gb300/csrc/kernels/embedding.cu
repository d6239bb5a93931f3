// Rows of a matrix by token number, and the gradient to the matrix.
//
//   out[t] = scale W[token[t]]
//   dW[v]  = base[v] + scale sum over {t : token[t] = v} of dout[t]
//
// Forward: memory traffic, the rows read and written once, a power of two of threads to
// a row.  8192 x 4096 bf16 19 us (7 TB/s, the frequent rows from L2), one row 3.
//
// Backward: the places t are sorted by token (stable), so that the rows of one
// token stand together and are added in the order of t, in registers, without
// atomics.  Threads take nearly equal chunks of the sorted places, however often a token
// occurs; a token of many places leaves fp32 parts, a chunk each, which a second kernel
// adds in order.  8192 x 4096 bf16 into 32000 rows 63 us: the rows 39 (6.8 TB/s), the sums
// 17, the parts 5; 65536 x 1024 into 131072 of fp32 147.
#include <algorithm>

#include "../embed_chunks.h"
#include "../operators.h"
#include "../per_device.h"
#include "indices.cuh"
#include "pieces.cuh"
#include "row_copy.cuh"
#include "tcgen05.cuh"

namespace mm {

namespace {

constexpr int kE = 8;  // elements of a piece: 16 bytes of the 16-bit types

// ---------------------------------------------------------------- forward
// Pieces (16 bytes, or single elements of rows that start anywhere) a thread has in
// flight.
template <bool EDGES>
constexpr int kEmbedPieces = EDGES ? 16 : 4;
template <int TW, int TO, bool EDGES>
__global__ void __launch_bounds__(256) embed_kernel(const EmbedArgs a, int log_threads) {
  constexpr int E = EDGES ? 1 : kE, N = kEmbedPieces<EDGES>;
  pdl_launch_dependents();
  pdl_wait();
  const int threads = 1 << log_threads, t = threadIdx.x & (threads - 1);
  const int64_t r = (int64_t)blockIdx.x * (256 >> log_threads) + (threadIdx.x >> log_threads);
  if (r >= a.rows) return;
  const int64_t token = load_token(a.tokens, a.ti, r, a.vocab);
  const float scale = token < a.vocab ? a.scale : 0.f;  // (zeros, whatever the scale)
  const int step = threads * E;
  for (int j0 = t * E; j0 < a.cols; j0 += N * step) {
    float v[N][E];
    const int n = token < a.vocab ? pieces_below<N>(j0, step, a.cols) : 0;
    load_pieces<TW>(a.weight, token * a.ldw + j0, step, n, v);
#pragma unroll
    for (int k = 0; k < N; ++k) {
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
  const int64_t each = whole ? kEmbedPieces<false> : kEmbedPieces<true>;
  while (log_threads < 8 && each << log_threads < pieces) ++log_threads;
  const int64_t rows = 256 >> log_threads;
  const dim3 grid((unsigned)((a.rows + rows - 1) / rows));
  return whole ? launch_pdl(embed_kernel<TW, TO, false>, grid, dim3(256), 0, ctx.stream, dim3(1), a, log_threads)
               : launch_pdl(embed_kernel<TW, TO, true>, grid, dim3(256), 0, ctx.stream, dim3(1), a, log_threads);
}

// ---------------------------------------------------------------- sort, and the rows of the others
// Least significant digit first, up to 9 bits a pass (a vocabulary below 2^18 takes two), by
// one CTA or one cluster of eight.  Each warp has a run of consecutive places: it counts its
// digits, the counts of all become places, and it goes over its run again; equal
// digits keep their order because a warp takes 32 at a time, ranked by matching.
// The places lie in global memory (L2) between passes, so any number of them sorts.
//
// dW's rows are written meanwhile, as zeros or the base's, by the other CTAs of the
// launch, those that the sums will write again among them.  (Untouched rows written
// beside the sums instead: 76 -> 88 us at 8192 x 4096 into 32000, 150 -> 191 at 65536 x
// 1024 into 131072.)  One CTA sorts where that takes no longer than the rows, since clusters
// of eight find room on 120 of the 152 SMs only: 8192 x 4096 63 us, by eight 68.
constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32, kMaxSortCtas = 8;
constexpr int kDigit = 9, kBins = 1 << kDigit;
constexpr size_t kSortSmem = (kSortWarps * kBins + kBins + 32) * sizeof(uint32_t);

struct SortParams {
  const void *tokens;
  int ti;
  int64_t vocab;
  int drop;            // tokens that differ in this many low bits only are one key
  int rows, passes, digit, ctas;  // bits a pass; ctas: 1 or kMaxSortCtas
  uint2 *to, *other;   // (key, place)
  uint32_t *spanning;  // set to 0: how many tokens the sums will have left in parts (or null)
  // the rows
  const uint8_t *base;  // null: zeros
  uint8_t *dweight;
  int64_t bytes, ldb, ldw;  // of a row and between rows, in bytes
  int64_t fill_rows;        // rows that follow one another without a gap count as one
};

__device__ __forceinline__ uint32_t cluster_u32(uint32_t addr, int rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(tc::map_to_rank(addr, (uint32_t)rank)) : "memory");
  return v;
}

__device__ __forceinline__ void sort_places(const SortParams &p, uint32_t *smem) {
  uint32_t(*off)[kBins] = reinterpret_cast<uint32_t(*)[kBins]>(smem);
  uint32_t *count = smem + kSortWarps * kBins, *warp_sum = count + kBins;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31, rank = (int)blockIdx.x;
  const int lo = (int)((int64_t)p.rows * rank / p.ctas), n = (int)((int64_t)p.rows * (rank + 1) / p.ctas) - lo;
  const int w0 = lo + (int)((int64_t)n * warp / kSortWarps), w1 = lo + (int)((int64_t)n * (warp + 1) / kSortWarps);
  const uint32_t below = (1u << lane) - 1;
  const int bins = 1 << p.digit;
  const auto sync = [&] {  // of all CTAs that sort
    if (p.ctas > 1) tc::cluster_sync_all();
    else __syncthreads();
  };
  constexpr int K = 8;
  uint2 *src = nullptr, *dst = p.passes & 1 ? p.to : p.other;  // the last pass ends in `to`
  for (int pass = 0; pass < p.passes; ++pass) {
    const int shift = pass * p.digit;
    const auto pair_at = [&](int i) {  // (written by other SMs: past L1)
      if (pass) return __ldcg(src + i);
      const int64_t v = load_token(p.tokens, p.ti, i, p.vocab);
      return make_uint2((uint32_t)(v < p.vocab ? v >> p.drop : keys_of(p.vocab, p.drop)), (uint32_t)i);
    };
    // the run, 32 K places at a time, and which lanes have equal digits; a run of one batch
    // stays in registers
    uint2 v[K] = {};
    uint32_t same[K];
    const auto digit = [&](int k, int i0) {
      return i0 + k * 32 + lane < w1 ? (v[k].x >> shift) & (bins - 1) : (uint32_t)kBins;
    };
    const auto load = [&](int i0) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int i = i0 + k * 32 + lane;
        v[k] = i < w1 ? pair_at(i) : make_uint2(0, 0);
      }
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (i0 + k * 32 < w1) same[k] = __match_any_sync(0xffffffffu, digit(k, i0));
    };
    for (int b = lane; b < bins; b += 32) off[warp][b] = 0;
    __syncwarp();
    for (int i0 = w0; i0 < w1; i0 += 32 * K) {
      load(i0);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (i0 + k * 32 >= w1) break;
        const uint32_t d = digit(k, i0);
        if (d < kBins && !(same[k] & below)) off[warp][d] += __popc(same[k]);
        __syncwarp();
      }
    }
    __syncthreads();
    if (t < bins) {
      uint32_t sum = 0;
#pragma unroll 16
      for (int w = 0; w < kSortWarps; ++w) {
        const uint32_t c = off[w][t];
        off[w][t] = sum;
        sum += c;
      }
      count[t] = sum;
    }
    sync();
    uint32_t before = 0, total = 0, sum = 0;
    if (t < bins) {
      const uint32_t addr = tc::smem_u32(count + t);
      uint32_t c[kMaxSortCtas];
#pragma unroll
      for (int r = 0; r < kMaxSortCtas; ++r) c[r] = r >= p.ctas ? 0 : p.ctas > 1 ? cluster_u32(addr, r) : count[t];
#pragma unroll
      for (int r = 0; r < kMaxSortCtas; ++r) before += r < rank ? c[r] : 0, total += c[r];
      sum = total;
    }
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t u = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += u;
    }
    if (lane == 31) warp_sum[warp] = sum;
    __syncthreads();
    if (t < bins) {
      uint32_t at = before + sum - total;
      for (int w = 0; w < warp; ++w) at += warp_sum[w];
#pragma unroll 16
      for (int w = 0; w < kSortWarps; ++w) off[w][t] += at;
    }
    __syncthreads();
    for (int i0 = w0; i0 < w1; i0 += 32 * K) {
      if (w1 - w0 > 32 * K) load(i0);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (i0 + k * 32 >= w1) break;
        const uint32_t d = digit(k, i0);
        if (d < kBins) dst[off[warp][d] + __popc(same[k] & below)] = v[k];
        __syncwarp();
        if (d < kBins && !(same[k] & below)) off[warp][d] += __popc(same[k]);
        __syncwarp();
      }
    }
    sync();  // (releases and acquires the places, too)
    src = dst;
    dst = dst == p.to ? p.other : p.to;
  }
}

// Row v of dW as zeros or the base's, by `threads` threads (this is the t-th): pieces of 16
// bytes as dW has them.
template <bool BASE>
__device__ __forceinline__ void write_row(const SortParams &p, int64_t v, int t, int threads) {
  constexpr int U = 4;  // pieces read before the first is stored
  uint8_t *to = p.dweight + v * p.ldw;
  const uint8_t *from = BASE ? p.base + v * p.ldb : nullptr;
  const int64_t first = -(int64_t)(reinterpret_cast<uintptr_t>(to) & 15);
  for (int64_t b0 = first + t * 16; b0 < p.bytes; b0 += threads * 16 * U) {
    RowPiece<2> x[U];
    const auto whole = [&](int64_t b) { return b >= 0 && b + 16 <= p.bytes; };
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int64_t b = b0 + k * threads * 16;
      if (BASE && whole(b)) x[k].load(from, p.bytes, b);
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int64_t b = b0 + k * threads * 16;
      if (whole(b)) {
        *reinterpret_cast<uint4 *>(to + b) = BASE ? x[k].value(from, p.bytes, b) : make_uint4(0, 0, 0, 0);
      } else {  // a row's ends
        for (int64_t e = max(b, (int64_t)0); e < min(b + 16, p.bytes); e += 2)
          *reinterpret_cast<uint16_t *>(to + e) = BASE ? *reinterpret_cast<const uint16_t *>(from + e) : (uint16_t)0;
      }
    }
  }
}
// Threads to a row: a power of two, up to 256, with up to four pieces each.
__device__ __forceinline__ int log_row_threads(int64_t bytes) {
  int n = 0;
  while (n < 8 && (64ll << n) < bytes + 15) ++n;
  return n;
}
// All rows, by `threads` threads, of which this is one.
__device__ __forceinline__ void write_rows(const SortParams &p, int64_t thread, int64_t threads) {
  if (p.fill_rows == 1) {
    if (p.base) write_row<true>(p, 0, (int)thread, (int)threads);
    else write_row<false>(p, 0, (int)thread, (int)threads);
    return;
  }
  const int log_threads = log_row_threads(p.bytes), t = (int)thread & ((1 << log_threads) - 1);
  for (int64_t v = thread >> log_threads; v < p.fill_rows; v += threads >> log_threads) {
    if (p.base) write_row<true>(p, v, t, 1 << log_threads);
    else write_row<false>(p, v, t, 1 << log_threads);
  }
}

__global__ void __launch_bounds__(kSortThreads) embed_sort_kernel(const SortParams p) {
  pdl_launch_dependents();
  pdl_wait();
  extern __shared__ uint32_t sort_smem[];
  if ((int)blockIdx.x < p.ctas) {
    if (p.spanning && blockIdx.x == 0 && threadIdx.x == 0) *p.spanning = 0;
    sort_places(p, sort_smem);
    return;
  }
  write_rows(p, ((int64_t)blockIdx.x - p.ctas) * kSortThreads + threadIdx.x,
             ((int64_t)gridDim.x - p.ctas) * kSortThreads);
}
// The rows alone, where there are no places.
__global__ void __launch_bounds__(256) embed_rows_kernel(const SortParams p) {
  pdl_launch_dependents();
  pdl_wait();
  write_rows(p, (int64_t)blockIdx.x * 256 + threadIdx.x, (int64_t)gridDim.x * 256);
}

// ---------------------------------------------------------------- sums
struct SumParams {
  EmbedBwdArgs a;
  const uint2 *sorted;  // (token, place)
  float *parts;         // [chunk][2][cols]: a token from the chunk before; one that goes on
  uint32_t *spanning;   // [0] how many tokens go past the end of the chunk where they begin,
                        // [1 ...] those chunks, in any order
  int chunk, chunks;
  int log_threads;
  int across;           // blocks for all chunks of a slab of columns
};
constexpr int kGroupPlaces = kMaxChunk + kSnap + 2;

// The base's piece of a token's row.
template <int TW, int E>
__device__ __forceinline__ Piece<TW, E> base_piece(const EmbedBwdArgs &a, int64_t token, int j) {
  return Piece<TW, E>::load(at<TW>(a.base, token * a.ldb + j));
}
template <int TW, int E>
__device__ __forceinline__ void write_sum(const EmbedBwdArgs &a, int64_t token, int j, const float (&sum)[E],
                                          const Piece<TW, E> &base) {
  float v[E];
#pragma unroll
  for (int e = 0; e < E; ++e) v[e] = fmaf(a.scale, sum[e], a.base ? base.get(e) : 0.f);
  store_piece<TW>(a.dweight, token * a.lddw + j, v);
}

// A chunk of places to a power of two of threads, a piece of the columns each.
// BASE: there is one; its row is read with the token's first, ahead of the sum (read when
// the sum was written it held up every token: 5000 x 1001 23 us).
template <int TW, int TO, int E, bool BASE>
__global__ void __launch_bounds__(256, kSumBlocks) embed_sum_kernel(const SumParams p) {
  // rows read before the first is added (as the registers hold)
  constexpr int U = E == 1 ? (BASE ? 8 : 16) : BASE ? (TW == MM_F32 || TO == MM_F32 ? 2 : 4) : TO == MM_F32 ? 4 : 8;
  constexpr int kPlaces = (256 >> kMinLogThreads) * kGroupPlaces;
  __shared__ uint32_t tokens[kPlaces];
  __shared__ int64_t starts[kPlaces];  // of a place's row of dout
  __shared__ int borders[256 >> kMinLogThreads][2];
  pdl_launch_dependents();
  pdl_wait();
  const EmbedBwdArgs &a = p.a;
  const int threads = 1 << p.log_threads, t = threadIdx.x & (threads - 1), group = threadIdx.x >> p.log_threads;
  const int slab = (int)blockIdx.x / p.across;
  const int chunk = ((int)blockIdx.x - slab * p.across) * (256 >> p.log_threads) + group;
  const int j = (slab * threads + t) * E;
  const int64_t i0 = (int64_t)chunk * p.chunk;
  const int left = places_left(a.rows, i0, p.chunk);
  const uint32_t none = (uint32_t)a.vocab;
  // the places of the chunk and those that may be taken over, and the one before
  uint32_t *mine = tokens + group * kGroupPlaces + 1;
  int64_t *start = starts + group * kGroupPlaces + 1;
  for (int i = t - 1; i <= p.chunk + kSnap; i += threads) {
    const uint2 s = reads_place(i0, i, left) ? p.sorted[i0 + i] : make_uint2(none, 0);
    mine[i] = s.x;
    start[i] = (int64_t)s.y * a.lddo;
  }
  if (t < 2) borders[group][t] = kSnap + 1;
  __syncthreads();
  for (int k = 0; k < 2; ++k)
    for (int i = t; i <= kSnap; i += threads)
      if (mine[k * p.chunk + i - 1] != mine[k * p.chunk + i]) atomicMin(&borders[group][k], i);
  __syncthreads();
  const int from = chunk == 0 || borders[group][0] > kSnap ? 0 : borders[group][0];
  const int n = min(left, p.chunk + (borders[group][1] > kSnap ? 0 : borders[group][1]));
  if (from >= n || j >= a.cols) return;
  uint32_t token = mine[from];
  bool from_before = mine[from - 1] == token;
  Piece<TW, E> base;
  float sum[E];
#pragma unroll
  for (int e = 0; e < E; ++e) sum[e] = 0.f;
  const auto leave = [&](bool goes_on) {
    if (from_before || goes_on) {
      store_piece<MM_F32>(p.parts, ((int64_t)chunk * 2 + (from_before ? 0 : 1)) * a.cols + j, sum);
      if (!from_before && j == 0) p.spanning[1 + atomicAdd(p.spanning, 1u)] = (uint32_t)chunk;
    } else {
      write_sum<TW, E>(a, token, j, sum, base);
    }
  };
  for (int i = from; i < n; i += U) {
    Piece<TO, E> v[U];
    Piece<TW, E> b[BASE ? U : 1];
    if constexpr (BASE) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i + u < n && mine[i + u] != none && (i + u == from || mine[i + u] != mine[i + u - 1]))
          b[u] = base_piece<TW, E>(a, mine[i + u], j);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i + u < n && mine[i + u] != none) v[u] = Piece<TO, E>::load(at<TO>(a.dout, start[i + u] + j));
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i + u >= n) break;
      const uint32_t next = mine[i + u];
      if (next != token) {
        leave(false);
        token = next;
        from_before = false;
        if constexpr (BASE) base = b[u];
#pragma unroll
        for (int e = 0; e < E; ++e) sum[e] = 0.f;
      }
      if (token == none) return;
      if constexpr (BASE) {
        if (i + u == from) base = b[0];
      }
#pragma unroll
      for (int e = 0; e < E; ++e) sum[e] += v[u].get(e);
    }
  }
  leave(mine[n] == token);
}

// Tokens whose places go past a chunk's end: their parts, 64 threads of V columns each a
// block, the chunks in four runs that are added in order.
template <int TW, int V>
__global__ void __launch_bounds__(256) embed_join_kernel(const SumParams p) {
  __shared__ float runs[4][64][V + 1];
  pdl_launch_dependents();
  pdl_wait();
  const EmbedBwdArgs &a = p.a;
  const int x = threadIdx.x & 63, y = threadIdx.x >> 6;
  const int j = ((int)blockIdx.x * 64 + x) * V, total = (int)p.spanning[0];
  for (int s = (int)blockIdx.y; s < total; s += (int)gridDim.y) {
    const int c = (int)p.spanning[1 + s];
    const uint32_t token = p.sorted[(int64_t)(c + 1) * p.chunk].x;
    int more = 0;  // the chunks after c that begin inside the token's run
    for (int k = c + 1;; k += 256) {
      const int at = k + (int)threadIdx.x;
      const int64_t inside = (int64_t)at * p.chunk + kSnap;  // (the border stayed in the token's run)
      const int here = __syncthreads_count(at < p.chunks && inside < a.rows && p.sorted[inside].x == token);
      more += here;
      if (here < 256) break;
    }
    const int k0 = (int)((int64_t)more * y / 4), k1 = (int)((int64_t)more * (y + 1) / 4);
    float sum[V];
#pragma unroll
    for (int e = 0; e < V; ++e) sum[e] = 0.f;
    if (j < a.cols) {
      const int64_t part = (int64_t)(c + 1) * 2 * a.cols + j;
      if (y == 0) load_piece<MM_F32>(p.parts, part - a.cols, sum);  // the second of chunk c
      for (int k = k0; k < k1; k += 8) {
        float v[8][V];
#pragma unroll
        for (int u = 0; u < 8; ++u)
          if (k + u < k1) load_piece<MM_F32>(p.parts, part + (int64_t)(k + u) * 2 * a.cols, v[u]);
#pragma unroll
        for (int u = 0; u < 8; ++u)
          if (k + u < k1)
#pragma unroll
            for (int e = 0; e < V; ++e) sum[e] += v[u][e];
      }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) runs[y][x][e] = sum[e];
    __syncthreads();
    if (y == 0 && j < a.cols) {
#pragma unroll
      for (int e = 0; e < V; ++e) sum[e] = ((sum[e] + runs[1][x][e]) + runs[2][x][e]) + runs[3][x][e];
      Piece<TW, V> base;
      if (a.base) base = base_piece<TW, V>(a, token, j);
      write_sum<TW, V>(a, token, j, sum, base);
    }
    __syncthreads();
  }
}

// Whether rows move in whole pieces, else in single elements.
bool whole_pieces(const EmbedBwdArgs &a) {
  const int bw = dtype_bytes(a.tw), bo = dtype_bytes(a.to);
  return a.cols % kE == 0 && (uintptr_t)a.dout % 16 == 0 && (uintptr_t)a.dweight % 16 == 0 &&
         (uintptr_t)a.base % 16 == 0 && (a.lddo * bo % 16 == 0 || a.rows == 1) &&
         (a.vocab == 1 || (a.lddw * bw % 16 == 0 && a.ldb * bw % 16 == 0));
}

template <int TW, int TO>
mm_status embed_sums(const EmbedBwdArgs &a, const SumParams &p, const SumShape &shape, LaunchCtx &ctx) {
  const bool whole = whole_pieces(a);
  const dim3 grid((unsigned)(shape.across * shape.slabs));
  const auto kernel = whole ? (a.base ? embed_sum_kernel<TW, TO, kE, true> : embed_sum_kernel<TW, TO, kE, false>)
                            : (a.base ? embed_sum_kernel<TW, TO, 1, true> : embed_sum_kernel<TW, TO, 1, false>);
  cudaError_t e = launch_pdl(kernel, grid, dim3(256), 0, ctx.stream, dim3(1), p);
  if (e != cudaSuccess) return cuda_error(e, "embedding_backward launch");
  count_operator_launch();
  if (p.chunks == 1) return MM_OK;
  // (slabs of columns along x: there may be more than the 65535 that y takes)
  const int64_t columns = whole ? 256 : 64, join_slabs = (a.cols + columns - 1) / columns;
  const int64_t across = std::max<int64_t>(1, std::min<int64_t>(p.chunks - 1, 8 * ctx.dev->info.sms / join_slabs));
  e = launch_pdl(whole ? embed_join_kernel<TW, 4> : embed_join_kernel<TW, 1>, dim3((unsigned)join_slabs, (unsigned)across), dim3(256), 0,
                 ctx.stream, dim3(1), p);
  if (e != cudaSuccess) return cuda_error(e, "embedding_backward launch (join)");
  count_operator_launch();
  return MM_OK;
}

// Set-up once a device, and how many clusters sort at once.
mm_status sort_places_at_once(LaunchCtx &ctx, int *clusters) {
  static PerDevice<int> fits;
  const cudaError_t err = fits.get(ctx.dev->info.ordinal, clusters, [](int *n) -> cudaError_t {
    cudaError_t e = cudaFuncSetAttribute(embed_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSortSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = kMaxSortCtas;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(kMaxSortCtas);
    lc.blockDim = dim3(kSortThreads);
    lc.dynamicSmemBytes = kSortSmem;
    lc.attrs = &at;
    lc.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(n, embed_sort_kernel, &lc);
  });
  if (err != cudaSuccess) return cuda_error(err, "sort set-up");
  if (*clusters < 1) return set_error(MM_ERR_UNSUPPORTED, "no cluster of CTAs fits on this device");
  return MM_OK;
}
// f's passes over the keys' bits, and its launch beside `row_ctas` that write rows.
mm_status launch_sort(SortParams &f, int row_ctas, LaunchCtx &ctx) {
  int bits = 1;  // of the keys up to that of none
  while (keys_of(f.vocab, f.drop) >> bits) ++bits;
  f.passes = (bits + kDigit - 1) / kDigit;
  f.digit = (bits + f.passes - 1) / f.passes;
  cudaError_t e = launch_pdl(embed_sort_kernel, dim3((unsigned)(f.ctas + row_ctas)), dim3(kSortThreads), kSortSmem,
                             ctx.stream, dim3((unsigned)f.ctas), f);
  if (e != cudaSuccess) return cuda_error(e, "sort launch");
  count_operator_launch();
  return MM_OK;
}
// Places that one CTA sorts where nothing else runs beside it.
constexpr int64_t kAlonePlaces = 2048;

// f(type of one, type of the other) as constants.
template <typename F>
auto with_type(int t, F &&f) {
  if (t == MM_BF16) return f(std::integral_constant<int, MM_BF16>());
  if (t == MM_F16) return f(std::integral_constant<int, MM_F16>());
  return f(std::integral_constant<int, MM_F32>());
}

}  // namespace

mm_status sort_ready(LaunchCtx &ctx) {
  int clusters;
  return sort_places_at_once(ctx, &clusters);
}

mm_status sort_tokens(const SortArgs &a, LaunchCtx &ctx) {
  SortParams f;
  std::memset(&f, 0, sizeof f);
  f.tokens = a.tokens;
  f.ti = a.ti;
  f.vocab = a.vocab;
  f.drop = a.drop;
  f.rows = a.rows;
  f.ctas = a.rows <= kAlonePlaces ? 1 : kMaxSortCtas;
  f.to = static_cast<uint2 *>(a.to);
  f.other = static_cast<uint2 *>(a.other);
  return launch_sort(f, 0, ctx);
}

mm_status launch_embedding(const EmbedArgs &a, LaunchCtx &ctx) {
  const cudaError_t e = with_type(a.tw, [&](auto tw) {
    return with_type(a.to, [&](auto to) { return embed_launch<decltype(tw)::value, decltype(to)::value>(a, ctx); });
  });
  if (e != cudaSuccess) return cuda_error(e, "embedding launch");
  count_operator_launch();
  return MM_OK;
}

mm_status launch_embedding_backward(const EmbedBwdArgs &a, LaunchCtx &ctx) {
  const int64_t es = dtype_bytes(a.tw);
  SumParams p;
  std::memset(&p, 0, sizeof p);
  p.a = a;
  const SumShape shape = sum_shape(a.rows, whole_pieces(a) ? a.cols / kE : a.cols, ctx.dev->info.sms);
  if (!shape.fits) return set_error(MM_ERR_UNSUPPORTED, "too many blocks");
  p.chunk = shape.chunk;
  p.chunks = shape.chunks;
  p.log_threads = shape.log_threads;
  p.across = (int)shape.across;
  SortParams f;
  std::memset(&f, 0, sizeof f);
  f.base = static_cast<const uint8_t *>(a.base);
  f.dweight = static_cast<uint8_t *>(a.dweight);
  f.bytes = a.cols * es;
  f.ldb = a.ldb * es;
  f.ldw = a.lddw * es;
  f.vocab = f.fill_rows = a.vocab;
  if (a.lddw == a.cols && (!a.base || a.ldb == a.cols)) {
    f.bytes *= a.vocab;
    f.fill_rows = 1;
  }
  const bool fills = a.base != a.dweight;  // else only the touched rows
  if (a.rows == 0) {
    if (!fills) return MM_OK;
    cudaError_t e = launch_pdl(embed_rows_kernel, dim3((unsigned)(8 * ctx.dev->info.sms)), dim3(256), 0, ctx.stream, dim3(1), f);
    if (e != cudaSuccess) return cuda_error(e, "embedding_backward launch (rows)");
    count_operator_launch();
    return MM_OK;
  }
  const auto whole = [](int64_t bytes) { return ((size_t)bytes + 255) / 256 * 256; };
  const size_t pairs = whole(a.rows * (int64_t)sizeof(uint2)), list = whole((p.chunks + 1) * (int64_t)sizeof(uint32_t));
  // as many CTAs as run at once: the first sort, the others write rows
  int clusters;
  mm_status st = sort_places_at_once(ctx, &clusters);
  if (st != MM_OK) return st;
  // One CTA sorts within 10 us and 3.7 ns a place (65536: 243 us; eight 42), and rows are
  // written at 5 TB/s or more.
  const int64_t written = fills ? f.bytes * f.fill_rows : 0;
  f.ctas = a.rows <= kAlonePlaces || (50 << 20) + a.rows * 18500 <= written ? 1 : kMaxSortCtas;
  const int row_ctas = !fills ? 0 : f.ctas == 1 ? ctx.dev->info.sms - 1 : std::max(1, clusters - 1) * kMaxSortCtas;
  void *scratch = nullptr;
  st = get_scratch(ctx, SCRATCH_WORKSPACE, 2 * pairs + list + (size_t)p.chunks * 2 * a.cols * sizeof(float), &scratch);
  if (st != MM_OK) return st;
  char *w = static_cast<char *>(scratch);
  f.to = reinterpret_cast<uint2 *>(w);
  f.other = reinterpret_cast<uint2 *>(w + pairs);
  f.spanning = p.spanning = reinterpret_cast<uint32_t *>(w + 2 * pairs);
  p.parts = reinterpret_cast<float *>(w + 2 * pairs + list);
  p.sorted = f.to;
  f.tokens = a.tokens;
  f.ti = a.ti;
  f.rows = (int)a.rows;
  if ((st = launch_sort(f, row_ctas, ctx)) != MM_OK) return st;
  return with_type(a.tw, [&](auto tw) {
    return with_type(a.to, [&](auto to) { return embed_sums<decltype(tw)::value, decltype(to)::value>(a, p, shape, ctx); });
  });
}

}  // namespace mm
