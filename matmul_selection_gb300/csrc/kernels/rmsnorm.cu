// Root-mean-square norm with the residual's addition, and its gradients.
//
//   h = x + residual, rstd = 1 / sqrt(mean(h^2) + eps), y = h rstd w
//   8-bit output: scale = max|y| / 448, q = e4m3(y / scale)
//   g = dy w, dx = dh + rstd (g - h rstd^2 mean(g h)), dw = sum_rows dy h rstd
//
// All of it is memory traffic: each input is read once and each output
// written once when a row stays in registers between its statistics and its
// outputs.  T threads (a warp to a block) hold a row, V pieces of 16 bytes a
// thread; max|y| is max|h w| rstd, so the 8-bit form needs no third pass.
// Statistics are fp32 sums.  Measured, bf16 8192 x 4096 with the residual: to bf16
// 42 us (6.4 TB/s), to e4m3 40 (5.9), backward 46 (5.8).  Rows longer than the
// registers hold, and rows that do not start on 16 bytes, have forms of their own
// below.
#include <algorithm>

#include "../operators.h"
#include "tcgen05.cuh"
#include "values.cuh"

namespace mm {

namespace {

constexpr float kE4m3Max = 448.f;

// ---------------------------------------------------------------- elements
constexpr __host__ __device__ int bytes_of(int t) { return t == MM_F32 ? 4 : 2; }

// E neighbours of type TX as they lie in memory, in registers: one access of
// 2 to 16 bytes (two of 16 for eight fp32).
template <int TX, int E>
struct Piece {
  static constexpr int kBytes = E * bytes_of(TX);
  uint32_t w[(kBytes + 3) / 4];
  static __device__ __forceinline__ Piece load(const void *p) {
    Piece x;
    if constexpr (kBytes == 2) {
      x.w[0] = *static_cast<const uint16_t *>(p);
    } else if constexpr (kBytes == 4) {
      x.w[0] = *static_cast<const uint32_t *>(p);
    } else if constexpr (kBytes == 8) {
      const uint2 v = *static_cast<const uint2 *>(p);
      x.w[0] = v.x, x.w[1] = v.y;
    } else {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i) {
        const uint4 v = static_cast<const uint4 *>(p)[i];
        x.w[4 * i] = v.x, x.w[4 * i + 1] = v.y, x.w[4 * i + 2] = v.z, x.w[4 * i + 3] = v.w;
      }
    }
    return x;
  }
  __device__ __forceinline__ void store(void *p) const {
    if constexpr (kBytes == 2) {
      *static_cast<uint16_t *>(p) = (uint16_t)w[0];
    } else if constexpr (kBytes == 4) {
      *static_cast<uint32_t *>(p) = w[0];
    } else if constexpr (kBytes == 8) {
      *static_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i)
        static_cast<uint4 *>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
  }
  __device__ __forceinline__ float get(int e) const {
    if constexpr (TX == MM_F32) return __uint_as_float(w[e]);
    if constexpr (TX == MM_BF16) return __uint_as_float(e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
    const __half2 v = *reinterpret_cast<const __half2 *>(&w[e / 2]);
    return e & 1 ? __high2float(v) : __low2float(v);
  }
  static __device__ __forceinline__ Piece of(const float (&v)[E]) {
    Piece x;
    if constexpr (TX == MM_F32) {
#pragma unroll
      for (int e = 0; e < E; ++e) x.w[e] = __float_as_uint(v[e]);
    } else {
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const float hi = e + 1 < E ? v[(e + 1) % E] : 0.f;
        if constexpr (TX == MM_BF16) {
          const __nv_bfloat162 y = __floats2bfloat162_rn(v[e], hi);
          x.w[e / 2] = *reinterpret_cast<const uint32_t *>(&y);
        } else {
          const __half2 y = __floats2half2_rn(v[e], hi);
          x.w[e / 2] = *reinterpret_cast<const uint32_t *>(&y);
        }
      }
    }
    return x;
  }
};
template <int TX>
__device__ __forceinline__ const void *at(const void *p, int64_t i) {
  return static_cast<const char *>(p) + i * bytes_of(TX);
}
template <int TX, int E>
__device__ __forceinline__ void load_piece(const void *p, int64_t i, float (&out)[E]) {
  const Piece<TX, E> x = Piece<TX, E>::load(at<TX>(p, i));
#pragma unroll
  for (int e = 0; e < E; ++e) out[e] = x.get(e);
}
template <int TX, int E>
__device__ __forceinline__ void store_piece(void *p, int64_t i, const float (&v)[E]) {
  Piece<TX, E>::of(v).store(static_cast<char *>(p) + i * bytes_of(TX));
}
// The same for a type that is known only at run time (the same for every
// thread).
template <int E>
__device__ __forceinline__ void load_piece(const void *p, int t, int64_t i, float (&out)[E]) {
  if (t == MM_BF16) load_piece<MM_BF16>(p, i, out);
  else if (t == MM_F16) load_piece<MM_F16>(p, i, out);
  else load_piece<MM_F32>(p, i, out);
}
// N pieces `step` elements apart, those below `n`, the others zeros.  The type is
// looked at once, outside the loop: looked at a piece, with its conversion in the
// branch, each load was waited for before the next was issued.
template <int TX, int E, int N>
__device__ __forceinline__ void load_pieces(const void *p, int64_t i, int64_t step, int n, float (&out)[N][E]) {
#pragma unroll
  for (int k = 0; k < N; ++k) {
    if (k < n) {
      load_piece<TX>(p, i + k * step, out[k]);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) out[k][e] = 0.f;
    }
  }
}
template <int E, int N>
__device__ __forceinline__ void load_pieces(const void *p, int t, int64_t i, int64_t step, int n,
                                            float (&out)[N][E]) {
  if (t == MM_BF16) load_pieces<MM_BF16>(p, i, step, n, out);
  else if (t == MM_F16) load_pieces<MM_F16>(p, i, step, n, out);
  else load_pieces<MM_F32>(p, i, step, n, out);
}
// The piece that starts `shift` elements (the same for every thread) into the
// first of two that follow one another.
template <int TX, int E>
__device__ __forceinline__ Piece<TX, E> shifted(const Piece<TX, E> &first, const Piece<TX, E> &second, int shift) {
  constexpr int W = (Piece<TX, E>::kBytes + 3) / 4;  // words
  const int words = shift * bytes_of(TX) / 4, bits = bytes_of(TX) == 2 ? (shift & 1) * 16 : 0;
  uint32_t w[2 * W];
#pragma unroll
  for (int j = 0; j < W; ++j) w[j] = first.w[j], w[W + j] = second.w[j];
#pragma unroll
  for (int b = W / 2; b > 0; b /= 2)
#pragma unroll
    for (int j = 0; j + b < 2 * W; ++j) w[j] = words & b ? w[j + b] : w[j];
  Piece<TX, E> x;
#pragma unroll
  for (int j = 0; j < W; ++j) x.w[j] = bytes_of(TX) == 2 ? __funnelshift_r(w[j], w[j + 1], bits) : w[j];
  return x;
}
// The same as load_pieces for pieces that start `shift` elements into a whole
// one: the two whole ones that hold a piece are loaded (the second of them is the
// next thread's first) and shifted in registers.
template <int TX, int E, int N>
__device__ __forceinline__ void load_pieces_at(const void *p, int64_t i, int64_t step, int n, int shift,
                                               float (&out)[N][E]) {
  if (shift == 0) return load_pieces<TX>(p, i, step, n, out);
  using P = Piece<TX, E>;
  P first[N], second[N];
#pragma unroll
  for (int k = 0; k < N; ++k)
    if (k < n) {
      first[k] = P::load(at<TX>(p, i + k * step - shift));
      second[k] = P::load(at<TX>(p, i + k * step - shift + E));
    }
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const P x = shifted(first[k], second[k], shift);
#pragma unroll
    for (int e = 0; e < E; ++e) out[k][e] = k < n ? x.get(e) : 0.f;
  }
}
template <int E, int N>
__device__ __forceinline__ void load_pieces_at(const void *p, int t, int64_t i, int64_t step, int n, int shift,
                                               float (&out)[N][E]) {
  if (t == MM_BF16) load_pieces_at<MM_BF16>(p, i, step, n, shift, out);
  else if (t == MM_F16) load_pieces_at<MM_F16>(p, i, step, n, shift, out);
  else load_pieces_at<MM_F32>(p, i, step, n, shift, out);
}
// How far into a whole piece of E elements element i lies.
template <int E>
__device__ __forceinline__ int piece_shift(const void *p, int element_bytes, int64_t i) {
  return (int)(((uintptr_t)p / element_bytes + (uint64_t)i) % E);
}
// How many of the N pieces i, i + step, ... start below `end`.
template <int N>
__device__ __forceinline__ int pieces_below(int64_t i, int64_t step, int64_t end) {
  int n = 0;
#pragma unroll
  for (int k = 0; k < N; ++k) n += i + k * step < end;
  return n;
}
template <int E>
__device__ __forceinline__ void store_piece(void *p, int t, int64_t i, const float (&v)[E]) {
  if (t == MM_BF16) {
    store_piece<MM_BF16>(p, i, v);
  } else if (t == MM_F16) {
    store_piece<MM_F16>(p, i, v);
  } else if (t == MM_F32) {
    store_piece<MM_F32>(p, i, v);
  } else {
    if constexpr (E % 2 == 0) {
      struct alignas(E) Bytes {
        uint16_t v[E / 2];
      } b;
#pragma unroll
      for (int e = 0; e < E; e += 2)
        b.v[e / 2] = __nv_cvt_float2_to_fp8x2(make_float2(v[e], v[e + 1]), __NV_SATFINITE, __NV_E4M3);
      *reinterpret_cast<Bytes *>(static_cast<uint8_t *>(p) + i) = b;
    } else {
      static_cast<uint8_t *>(p)[i] = to_e4m3(v[0]);
    }
  }
}

// ---------------------------------------------------------------- sums over a row's threads
// T threads (a warp, or the block) hold a row.  The sum (the warps' in order)
// in every thread.
template <int T>
__device__ __forceinline__ float row_sum(float v, float *sh) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (T > 32) {
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    v = sh[0];
#pragma unroll
    for (int w = 1; w < T / 32; ++w) v += sh[w];
  }
  return v;
}
// The sum of one value and the largest of another's bits (of non-negative
// floats: a NaN's bits are above every number's, so a NaN anywhere is the
// largest), at one barrier.
template <int T>
__device__ __forceinline__ void row_sum_max(float &v, uint32_t &m, float *sh) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  m = __reduce_max_sync(0xffffffffu, m);
  if constexpr (T > 32) {
    uint32_t *shm = reinterpret_cast<uint32_t *>(sh + T / 32);
    if ((threadIdx.x & 31) == 0) {
      sh[threadIdx.x >> 5] = v;
      shm[threadIdx.x >> 5] = m;
    }
    __syncthreads();
    v = sh[0];
    m = shm[0];
#pragma unroll
    for (int w = 1; w < T / 32; ++w) {
      v += sh[w];
      m = max(m, shm[w]);
    }
  }
}

// The scale of an 8-bit row: max|y| / 448, 1 for a row of zeros, and no
// smaller than the least normal float, so that its reciprocal is finite.  A
// NaN stays one.
__device__ __forceinline__ float row_scale(float amax) {
  const float s = amax / kE4m3Max;
  return amax == 0.f ? 1.f : s < 0x1p-126f ? 0x1p-126f : s;
}

// ---------------------------------------------------------------- forward
// T threads a row (a warp, eight of them a block, or a block), V pieces of E
// elements a thread: the row of T V E elements or fewer stays in registers.
// Pieces past cols are not accessed (without EDGES cols is a multiple of E).
// EDGES: rows that start anywhere.  The pieces are those that y stores whole; an
// input that lies otherwise is read by whole pieces of its own, two for one (h
// that lies otherwise is stored an element at a time).  Only pieces whose reads
// stay inside the row are taken so; the elements before and behind, 29 at most,
// go to the row's first threads, one each.  An element is read by other threads
// than the one that writes it only where x or the residual is not an output.
template <int TX, int E, int T, int V, bool EDGES>
__global__ void __launch_bounds__(T == 32 ? 256 : T) rmsnorm_rows_kernel(const NormArgs a) {
  constexpr int ROWS = T == 32 ? 8 : 1;
  pdl_launch_dependents();
  pdl_wait();
  __shared__ float sh[2 * (T / 32)];
  const int t = threadIdx.x % T;
  const int64_t r = (int64_t)blockIdx.x * ROWS + threadIdx.x / T;
  if (T == 32 && r >= a.rows) return;  // (no barrier below)
  int head = 0, end = a.cols, edge = -1;  // the pieces' [head, end), and this thread's element outside
  int sx = 0, sr = 0, sw = 0;
  bool whole_h = true;
  if constexpr (EDGES) {
    head = (E - piece_shift<E>(a.y, a.scale ? 1 : a.ty == MM_F32 ? 4 : 2, r * a.ldy)) % E;
    sx = piece_shift<E>(a.x, bytes_of(TX), r * a.ldx + head);
    if (a.residual) sr = piece_shift<E>(a.residual, bytes_of(TX), r * a.ldr + head);
    sw = piece_shift<E>(a.weight, a.tw == MM_F32 ? 4 : 2, head);
    whole_h = piece_shift<E>(a.h, bytes_of(TX), r * a.ldh + head) == 0;
    if (sx | sr | sw) {  // [j - shift, j - shift + 2 E) of a piece at j lies inside
      head += E;
      end = a.cols - (E - 1);
    }
    end = head + max(0, end - head) / E * E;
    if (end == head) head = end = min(head, a.cols);
    if (t < head) edge = t;
    else if (end + t - head < a.cols) edge = end + t - head;
  }
  const int j0 = head + t * E;
  const int n = max(0, (end - j0 + T * E - 1) / (T * E));  // this thread's pieces
  float h[V][E], w[V][E];
  float eh = 0.f, ew = 0.f;
  load_pieces_at<TX>(a.x, r * a.ldx + j0, T * E, n, EDGES ? sx : 0, h);
  if (EDGES && edge >= 0) eh = load_value(a.x, TX, r * a.ldx + edge);
  if (a.residual) {
    float res[V][E];
    load_pieces_at<TX>(a.residual, r * a.ldr + j0, T * E, n, EDGES ? sr : 0, res);
    if (EDGES && edge >= 0) eh += load_value(a.residual, TX, r * a.ldr + edge);
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < E; ++e) h[v][e] += res[v][e];
  }
  load_pieces_at(a.weight, a.tw, j0, T * E, n, EDGES ? sw : 0, w);
  if (EDGES && edge >= 0) ew = load_value(a.weight, a.tw, edge);
  float ss = eh * eh;
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int e = 0; e < E; ++e) ss += h[v][e] * h[v][e];
  if (a.h) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int j = j0 + v * T * E;
      if (j >= end) break;
      if (!EDGES || whole_h) {
        store_piece<TX>(a.h, r * a.ldh + j, h[v]);
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) store_value(a.h, TX, r * a.ldh + j + e, h[v][e]);
      }
    }
    if (EDGES && edge >= 0) store_value(a.h, TX, r * a.ldh + edge, eh);
  }
  if (a.scale) {
    uint32_t big = 0;  // of |h w|: y is this times rstd
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (j0 + v * T * E < end)
#pragma unroll
        for (int e = 0; e < E; ++e) {
          h[v][e] *= w[v][e];
          big = max(big, __float_as_uint(fabsf(h[v][e])));
        }
    if (EDGES && edge >= 0) {
      eh *= ew;
      big = max(big, __float_as_uint(fabsf(eh)));
    }
    row_sum_max<T>(ss, big, sh);
    const float rstd = 1.f / sqrtf(ss / (float)a.cols + a.eps);
    const float scale = row_scale(__uint_as_float(big) * rstd);
    // Two factors in turn, y first: their product is 448 / max|h w|, which is
    // beyond fp32 for rows below 1.3e-36.
    const float inv = 1.f / scale;
    if (t == 0) {
      a.scale[r] = scale;
      if (a.rstd) a.rstd[r] = rstd;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int j = j0 + v * T * E;
      if (j < end) {
#pragma unroll
        for (int e = 0; e < E; ++e) h[v][e] = h[v][e] * rstd * inv;
        store_piece(a.y, MM_E4M3, r * a.ldy + j, h[v]);
      }
    }
    if (EDGES && edge >= 0) static_cast<uint8_t *>(a.y)[r * a.ldy + edge] = to_e4m3(eh * rstd * inv);
  } else {
    ss = row_sum<T>(ss, sh);
    const float rstd = 1.f / sqrtf(ss / (float)a.cols + a.eps);
    if (a.rstd && t == 0) a.rstd[r] = rstd;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int j = j0 + v * T * E;
      if (j < end) {
#pragma unroll
        for (int e = 0; e < E; ++e) h[v][e] = h[v][e] * rstd * w[v][e];
        store_piece(a.y, a.ty, r * a.ldy + j, h[v]);
      }
    }
    if (EDGES && edge >= 0) store_value(a.y, a.ty, r * a.ldy + edge, eh * rstd * ew);
  }
}

// Rows of any length, E elements an access: a block of 1024 a row, two passes
// over it (the second reads what the first left in L1 and L2).
template <int TX, int E>
__global__ void __launch_bounds__(1024) rmsnorm_long_kernel(const NormArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ float sh[64];
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    constexpr int U = E == 1 ? 4 : 2;  // pieces in flight
    float ss = 0.f;
    uint32_t big = 0;
    for (int j0 = threadIdx.x * E; j0 < a.cols; j0 += U * 1024 * E) {
      const int n = pieces_below<U>(j0, 1024 * E, a.cols);
      float h[U][E], s[U][E] = {}, w[U][E];
      load_pieces<TX>(a.x, r * a.ldx + j0, 1024 * E, n, h);
      if (a.residual) load_pieces<TX>(a.residual, r * a.ldr + j0, 1024 * E, n, s);
      if (a.scale) load_pieces(a.weight, a.tw, j0, 1024 * E, n, w);
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float x = h[u][e] + s[u][e];
          ss += x * x;
          if (a.scale) big = max(big, __float_as_uint(fabsf(x * w[u][e])));
        }
    }
    __syncthreads();  // the previous row's sums have been read
    row_sum_max<1024>(ss, big, sh);
    const float rstd = 1.f / sqrtf(ss / (float)a.cols + a.eps);
    float inv = 1.f;
    if (a.scale) {
      const float scale = row_scale(__uint_as_float(big) * rstd);
      inv = 1.f / scale;
      if (threadIdx.x == 0) a.scale[r] = scale;
    }
    if (a.rstd && threadIdx.x == 0) a.rstd[r] = rstd;
    for (int j0 = threadIdx.x * E; j0 < a.cols; j0 += U * 1024 * E) {
      const int n = pieces_below<U>(j0, 1024 * E, a.cols);
      float h[U][E], s[U][E] = {}, w[U][E];
      load_pieces<TX>(a.x, r * a.ldx + j0, 1024 * E, n, h);
      if (a.residual) load_pieces<TX>(a.residual, r * a.ldr + j0, 1024 * E, n, s);
      load_pieces(a.weight, a.tw, j0, 1024 * E, n, w);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (u < n) {
          const int j = j0 + u * 1024 * E;
#pragma unroll
          for (int e = 0; e < E; ++e) h[u][e] += s[u][e];
          if (a.h) store_piece<TX>(a.h, r * a.ldh + j, h[u]);
#pragma unroll
          for (int e = 0; e < E; ++e) {
            h[u][e] = h[u][e] * rstd * w[u][e];
            if (a.scale) h[u][e] *= inv;
          }
          store_piece(a.y, a.ty, r * a.ldy + j, h[u]);
        }
    }
  }
}

template <typename K, typename... Args>
mm_status launch(K kern, int64_t blocks, int threads, LaunchCtx &ctx, const char *what, Args... args) {
  cudaError_t e = launch_pdl(kern, dim3((unsigned)blocks), dim3((unsigned)threads), 0, ctx.stream, dim3(1), args...);
  if (e != cudaSuccess) return cuda_error(e, what);
  count_operator_launch();
  return MM_OK;
}

// The largest power of two of elements (at most `most`) that divides cols and
// that all rows and operands are aligned to.
struct Alignment {
  uint64_t bits = 0;  // byte addresses and distances, per element size
  int cols;
  void operand(const void *p, int64_t ld, int64_t rows, int es) {
    if (!p) return;
    // in elements of this operand: an access of E elements needs E es bytes
    bits |= (uint64_t)(uintptr_t)p / es;
    if (rows > 1) bits |= (uint64_t)ld;
  }
  int elements(int most) const {
    const uint64_t b = bits | (uint64_t)cols;
    int e = most;
    while (e > 1 && b % e) e /= 2;
    return e;
  }
};

int type_size(int t) { return t == MM_E4M3 ? 1 : dtype_bytes(t); }

template <int TX, int E, int T, int V, bool EDGES>
mm_status rows_form(const NormArgs &a, LaunchCtx &ctx) {
  constexpr int ROWS = T == 32 ? 8 : 1;
  const int64_t blocks = (a.rows + ROWS - 1) / ROWS;
  if (blocks >= (1LL << 31)) return set_error(MM_ERR_UNSUPPORTED, "too many rows");
  return launch(rmsnorm_rows_kernel<TX, E, T, V, EDGES>, blocks, T == 32 ? 256 : T, ctx, "rmsnorm launch", a);
}
template <int TX, int E>
mm_status long_form(const NormArgs &a, LaunchCtx &ctx) {
  return launch(rmsnorm_long_kernel<TX, E>, std::min<int64_t>(a.rows, 2 * ctx.dev->info.sms), 1024, ctx,
                "rmsnorm launch (long rows)", a);
}

// A warp a row up to 128 pieces, then a block of 256 to 1024 (8192 x 4096 bf16:
// 42 us, 6.4 TB/s; to e4m3 40 us).  Rows that start anywhere: up to 256 elements a
// warp and an element an access (its pieces would leave most lanes idle: 100000 x
// 101 f16 29 us against 63), above that in pieces and blocks half as large, since
// the reads of two pieces for one need the registers (8192 x 4097 bf16 52 us, an
// element an access 75; 33000 x 1001 50 and 62; with the aligned rows' blocks
// 16384 x 1601 58 us, with these 47).
template <int TX, bool EDGES>
mm_status forward_form(const NormArgs &a, LaunchCtx &ctx) {
  constexpr int E = 16 / bytes_of(TX);
  const int pieces = a.cols / E;
  if (EDGES && a.cols <= 128) return rows_form<TX, 1, 32, 4, false>(a, ctx);
  if (EDGES && a.cols <= 256) return rows_form<TX, 1, 32, 8, false>(a, ctx);
  if (pieces <= 64) return rows_form<TX, E, 32, 2, EDGES>(a, ctx);
  if (EDGES && pieces <= 128) return rows_form<TX, E, 64, 2, EDGES>(a, ctx);
  if (pieces <= 128) return rows_form<TX, E, 32, 4, EDGES>(a, ctx);
  if (EDGES && pieces <= 256) return rows_form<TX, E, 128, 2, EDGES>(a, ctx);
  if (pieces <= 256) return rows_form<TX, E, 256, 1, EDGES>(a, ctx);
  if (pieces <= 512) return rows_form<TX, E, 256, 2, EDGES>(a, ctx);
  if (pieces <= 1024) return rows_form<TX, E, 512, 2, EDGES>(a, ctx);
  if (pieces <= 2048) return rows_form<TX, E, 1024, 2, EDGES>(a, ctx);
  if constexpr (E == 4)
    if (pieces <= 4096) return rows_form<TX, E, 1024, 4, EDGES>(a, ctx);
  return long_form<TX, EDGES ? 1 : E>(a, ctx);
}

template <int TX>
mm_status forward_type(const NormArgs &a, LaunchCtx &ctx) {
  Alignment al;
  al.cols = a.cols;
  al.operand(a.x, a.ldx, a.rows, type_size(a.tx));
  al.operand(a.residual, a.ldr, a.rows, type_size(a.tx));
  al.operand(a.weight, 0, 1, type_size(a.tw));
  al.operand(a.h, a.ldh, a.rows, type_size(a.tx));
  al.operand(a.y, a.ldy, a.rows, type_size(a.ty));
  constexpr int most = 16 / bytes_of(TX);
  if (al.elements(most) == most) return forward_form<TX, false>(a, ctx);
  // In place at another distance than y's: see the kernel's last sentence.
  const uint64_t d = (uint64_t)(uintptr_t)a.h / bytes_of(TX) - (uint64_t)(uintptr_t)a.y / type_size(a.ty);
  const bool alike = d % most == 0 && (a.rows == 1 || (uint64_t)(a.ldh - a.ldy) % most == 0);
  if (a.h && (a.h == a.x || a.h == a.residual) && !alike) return long_form<TX, 1>(a, ctx);
  return forward_form<TX, true>(a, ctx);
}

// ---------------------------------------------------------------- backward
// Three forms, by the length of a row.  Each block walks the
// rows blockIdx.x, blockIdx.x + gridDim.x, ... (or its warps do) and keeps its
// sums of dy h rstd in registers; the blocks' sums go to a workspace and a
// second kernel adds them in block order.
//
// What a thread does with a piece of a row: its share of sum(dy w h) and
// sum(h^2), then, when the sums are there, its dx and its part of dw.
template <int TX, int E>
struct BwdPiece {
  using P = Piece<TX, E>;
  static __device__ __forceinline__ void sums(const P &dy, const P &h, const float (&w)[E], float &dot, float &ss) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float x = h.get(e);
      dot += dy.get(e) * w[e] * x;
      ss += x * x;
    }
  }
  static __device__ __forceinline__ void outputs(const P &dy, const P &h, const P *dh, const float (&w)[E], float rs,
                                                 float c, float (&dx)[E], float (&dw)[E]) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float g = dy.get(e), x = h.get(e);
      dx[e] = rs * (g * w[e] - x * c);
      if (dh) dx[e] += dh->get(e);
      dw[e] += g * x * rs;
    }
  }
};
__device__ __forceinline__ int64_t partial_ld(int cols) { return (int64_t)(cols + 3) / 4 * 4; }

// Short rows: a warp a row, eight warps a block, no barrier until the end,
// where the warps' sums are added in order.
template <int TX, int E, int V>
__global__ void __launch_bounds__(256) rmsnorm_bwd_warps_kernel(const NormBwdArgs a, float *partial) {
  using P = Piece<TX, E>;
  pdl_launch_dependents();
  pdl_wait();
  __shared__ float sums[8][32 * V * E];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float w[V][E], dw[V][E] = {};
  load_pieces(a.weight, a.tw, lane * E, 32 * E, max(0, (a.cols - lane * E + 32 * E - 1) / (32 * E)), w);
  const float per_col = 1.f / (float)a.cols;
  for (int64_t r = (int64_t)blockIdx.x * 8 + warp; r < a.rows; r += (int64_t)gridDim.x * 8) {
    P dy[V], h[V], dh[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int j = (v * 32 + lane) * E;
      if (j < a.cols) {
        dy[v] = P::load(at<TX>(a.dy, r * a.lddy + j));
        h[v] = P::load(at<TX>(a.h, r * a.ldh + j));
        if (a.dh) dh[v] = P::load(at<TX>(a.dh, r * a.lddh + j));
      }
    }
    float rs = a.rstd ? a.rstd[r] : 0.f;
    float dot = 0.f, ss = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if ((v * 32 + lane) * E < a.cols) BwdPiece<TX, E>::sums(dy[v], h[v], w[v], dot, ss);
    dot = row_sum<32>(dot, nullptr);
    if (!a.rstd) rs = 1.f / sqrtf(row_sum<32>(ss, nullptr) / (float)a.cols + a.eps);
    const float c = dot * per_col * rs * rs;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int j = (v * 32 + lane) * E;
      if (j < a.cols) {
        float dx[E];
        BwdPiece<TX, E>::outputs(dy[v], h[v], a.dh ? &dh[v] : nullptr, w[v], rs, c, dx, dw[v]);
        store_piece<TX>(a.dx, r * a.lddx + j, dx);
      }
    }
  }
  if (!partial) return;
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int e = 0; e < E; ++e) sums[warp][(v * 32 + lane) * E + e] = dw[v][e];
  __syncthreads();
  for (int j = threadIdx.x; j < a.cols; j += 256) {
    float s = sums[0][j];
#pragma unroll
    for (int k = 1; k < 8; ++k) s += sums[k][j];
    partial[blockIdx.x * partial_ld(a.cols) + j] = s;
  }
}

// Rows of whole 16-byte pieces: a block a row at a time, its dy, h and dh
// brought by bulk copies into a ring of rows in shared memory, so that what is
// in flight (up to 200 KB an SM) does not depend on registers.  (Rows held in
// registers, the next one's loads issued ahead: 85 us at 8192 x 4096 bf16, 47 %
// of HBM's rate.)  Both passes read the row from shared memory.  A stage is
// refilled after the next row's barrier, which every thread reaches only when
// it is done with the row before.
// EDGES: rows that start anywhere, as in the forward kernel: dx's pieces, inputs
// that lie otherwise read two pieces for one, the elements before and behind one a
// thread, straight from memory, a row ahead.  The grid is a multiple of E blocks,
// so that a block's rows all lie alike and its sums keep their columns; bulk
// copies take what of a row is whole pieces.
constexpr int kMaxRing = 8, kErrRing = 0xb01;
// A row in the ring: what lies before it in its first 16 bytes comes with it.
template <bool EDGES>
constexpr __host__ __device__ uint32_t ring_row(uint32_t bytes) {
  return EDGES ? (bytes + 30) / 16 * 16 : bytes;
}
// One thread starts the copies of a row.
template <int TX, bool EDGES>
__device__ __forceinline__ void ring_fill(const NormBwdArgs &a, int64_t r, uint32_t dst, uint32_t bar) {
  const uint32_t bytes = (uint32_t)a.cols * bytes_of(TX), row = ring_row<EDGES>(bytes), parts = a.dh ? 3 : 2;
  if constexpr (!EDGES) {
    tc::mbar_expect_tx_one(bar, parts * row);
    tc::bulk_load(dst, at<TX>(a.dy, r * a.lddy), row, bar);
    tc::bulk_load(dst + row, at<TX>(a.h, r * a.ldh), row, bar);
    if (a.dh) tc::bulk_load(dst + 2 * row, at<TX>(a.dh, r * a.lddh), row, bar);
  } else {
    const char *p[3] = {static_cast<const char *>(at<TX>(a.dy, r * a.lddy)),
                        static_cast<const char *>(at<TX>(a.h, r * a.ldh)),
                        static_cast<const char *>(at<TX>(a.dh, a.dh ? r * a.lddh : 0))};
    uint32_t skip[3], size[3], all = 0;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const uint32_t off = (uint32_t)(uintptr_t)p[k] & 15u;
      skip[k] = (16u - off) & 15u;
      size[k] = k < (int)parts && skip[k] < bytes ? (bytes - skip[k]) & ~15u : 0u;
      all += size[k];
    }
    tc::mbar_expect_tx_one(bar, all);
#pragma unroll
    for (int k = 0; k < 3; ++k)
      if (size[k]) tc::bulk_load(dst + k * row + (skip[k] ? 16u : 0u), p[k] + skip[k], size[k], bar);
  }
}
// After a wait that gave up, by the thread that fills the ring: no copy is in flight
// any more (waited for with a limit).  A stage's barrier is in a phase of either
// parity, and waiting for the other one returns at once.
static __device__ __noinline__ void ring_drain(const uint64_t *full, int stages, int *err) {
  for (int s = 0; s < 2 * stages; ++s) tc::wait_drain_slow(tc::smem_u32(full + s / 2), s & 1, err, kErrRing);
}
// Where the columns of a block's rows lie: the pieces' [head, end); how far into
// whole pieces the inputs' are; where the inputs' pieces start in the ring's row.
struct RingPlace {
  int head, end, s_dy, s_h, s_dh, s_w;
  uint32_t o_dy, o_h, o_dh;
  // the element outside the pieces that the t-th of a row's threads has, or -1
  __device__ __forceinline__ int edge(int t, int cols) const {
    return t < head ? t : end + t - head < cols ? end + t - head : -1;
  }
};
template <int TX, bool EDGES>
__device__ __forceinline__ RingPlace ring_place(const NormBwdArgs &a, int64_t r) {
  constexpr int E = 16 / bytes_of(TX), es = bytes_of(TX);
  const uint32_t row = ring_row<EDGES>((uint32_t)a.cols * es);
  RingPlace p{0, a.cols, 0, 0, 0, 0, 0, row, 2 * row};
  if constexpr (EDGES) {
    p.head = (E - piece_shift<E>(a.dx, es, r * a.lddx)) % E;
    p.s_dy = piece_shift<E>(a.dy, es, r * a.lddy + p.head);
    p.s_h = piece_shift<E>(a.h, es, r * a.ldh + p.head);
    if (a.dh) p.s_dh = piece_shift<E>(a.dh, es, r * a.lddh + p.head);
    p.s_w = piece_shift<E>(a.weight, a.tw == MM_F32 ? 4 : 2, p.head);
    if (p.s_dy | p.s_h | p.s_dh | p.s_w) {  // [j - shift, j - shift + 2 E) of a piece at j lies inside
      p.head += E;
      p.end = a.cols - (E - 1);
    }
    p.end = p.head + max(0, p.end - p.head) / E * E;
    if (p.end == p.head) p.head = p.end = min(p.head, a.cols);
    // whole pieces: a multiple of 16 bytes into the row's place
    p.o_dy += (uint32_t)((piece_shift<E>(a.dy, es, r * a.lddy) + p.head - p.s_dy) * es);
    p.o_h += (uint32_t)((piece_shift<E>(a.h, es, r * a.ldh) + p.head - p.s_h) * es);
    if (a.dh) p.o_dh += (uint32_t)((piece_shift<E>(a.dh, es, r * a.lddh) + p.head - p.s_dh) * es);
  }
  return p;
}
template <int TX, bool EDGES>
__device__ __forceinline__ Piece<TX, 16 / bytes_of(TX)> ring_piece(const uint8_t *p, int i, int shift) {
  using P = Piece<TX, 16 / bytes_of(TX)>;
  const P x = P::load(p + i * 16);
  return EDGES && shift ? shifted(x, P::load(p + i * 16 + 16), shift) : x;
}

template <int TX, int T, int V, int PER_SM, bool EDGES>
__global__ void __launch_bounds__(T, PER_SM) rmsnorm_bwd_ring_kernel(const NormBwdArgs a, float *partial, int stages,
                                                              Waits wait) {
  constexpr int E = 16 / bytes_of(TX);
  using P = Piece<TX, E>;
  pdl_launch_dependents();
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ float sh[2][2 * (T / 32)];
  __shared__ __align__(8) uint64_t full[kMaxRing + 1];  // a stage each; the test hook's
  const int t = threadIdx.x;
  const uint32_t stage_bytes = (a.dh ? 3 : 2) * ring_row<EDGES>((uint32_t)a.cols * bytes_of(TX));
  if (t == 0) {
    for (int s = 0; s <= kMaxRing; ++s) tc::mbar_init(tc::smem_u32(full + s), 1);
    tc::mbar_init_fence();
  }
  __syncthreads();
  pdl_wait();
  auto fill = [&](int64_t r, int s) {
    ring_fill<TX, EDGES>(a, r, tc::smem_u32(ring) + (uint32_t)s * stage_bytes, tc::smem_u32(full + s));
  };
  if (t == 0)
    for (int s = 0; s < stages; ++s)
      if (blockIdx.x + (int64_t)s * gridDim.x < a.rows) fill(blockIdx.x + (int64_t)s * gridDim.x, s);
  const RingPlace at_row = ring_place<TX, EDGES>(a, blockIdx.x);
  const int head = at_row.head, edge = EDGES ? at_row.edge(t, a.cols) : -1;
  const int n = max(0, (at_row.end - head - t * E + T * E - 1) / (T * E));  // this thread's pieces
  float w[V][E], dw[V][E] = {};
  load_pieces_at(a.weight, a.tw, head + t * E, T * E, n, EDGES ? at_row.s_w : 0, w);
  float ew = 0.f, edw = 0.f, next_dy = 0.f, next_h = 0.f, next_dh = 0.f;
  auto load_edge = [&](int64_t r) {
    if (!EDGES || edge < 0 || r >= a.rows) return;
    next_dy = load_value(a.dy, TX, r * a.lddy + edge);
    next_h = load_value(a.h, TX, r * a.ldh + edge);
    if (a.dh) next_dh = load_value(a.dh, TX, r * a.lddh + edge);
  };
  if (EDGES && edge >= 0) ew = load_value(a.weight, a.tw, edge);
  load_edge(blockIdx.x);
  const float per_col = 1.f / (float)a.cols;
  int s = 0, side = 0;
  uint32_t phase = 0;
  // A wait ran into its limit: no further one is waited for, and the ring is not
  // filled again (a barrier would be armed twice).
  bool gave_up = wait.stall && !tc::thread_wait(tc::smem_u32(full + kMaxRing), 0, wait, kErrRing);
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const float given = a.rstd ? a.rstd[r] : 0.f;
    const uint8_t *stage = ring + (size_t)s * stage_bytes;
    auto dy = [&](int i) { return ring_piece<TX, EDGES>(stage + at_row.o_dy, i, at_row.s_dy); };
    auto h = [&](int i) { return ring_piece<TX, EDGES>(stage + at_row.o_h, i, at_row.s_h); };
    const float edy = next_dy, eh = next_h, edh = next_dh;
    load_edge(r + gridDim.x);
    float dot = edy * ew * eh, ss = eh * eh;
    if (!gave_up && !tc::thread_wait(tc::smem_u32(full + s), phase, wait, kErrRing)) gave_up = true;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int i = v * T + t;
      if (v < n) BwdPiece<TX, E>::sums(dy(i), h(i), w[v], dot, ss);
    }
    // two sets of shared sums in turn: one barrier a row
    dot = row_sum<T>(dot, sh[side]);
    float rs = given;
    if (!a.rstd) rs = 1.f / sqrtf(row_sum<T>(ss, sh[side] + T / 32) / (float)a.cols + a.eps);
    side ^= 1;
    // every thread is done with the row before: its stage takes the row `stages` after it
    const int64_t r_next = r + (int64_t)(stages - 1) * gridDim.x;
    if (t == 0 && !gave_up && r != blockIdx.x && r_next < a.rows) fill(r_next, s == 0 ? stages - 1 : s - 1);
    const float c = dot * per_col * rs * rs;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int i = v * T + t;
      if (v < n) {
        float dx[E];
        P d;
        if (a.dh) d = ring_piece<TX, EDGES>(stage + at_row.o_dh, i, at_row.s_dh);
        BwdPiece<TX, E>::outputs(dy(i), h(i), a.dh ? &d : nullptr, w[v], rs, c, dx, dw[v]);
        store_piece<TX>(a.dx, r * a.lddx + head + i * E, dx);
      }
    }
    if (EDGES && edge >= 0) {
      store_value(a.dx, TX, r * a.lddx + edge, rs * (edy * ew - eh * c) + edh);
      edw += edy * eh * rs;
    }
    if (++s == stages) {
      s = 0;
      phase ^= 1;
    }
  }
  if (partial) {
    float *out = partial + blockIdx.x * partial_ld(a.cols);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int j = head + (v * T + t) * E;
      if (v < n) {
        if constexpr (!EDGES) {
          store_piece<MM_F32>(out, j, dw[v]);
        } else {
#pragma unroll
          for (int e = 0; e < E; ++e) out[j + e] = dw[v][e];
        }
      }
    }
    if (EDGES && edge >= 0) out[edge] = edw;
  }
  if (gave_up && t == 0) ring_drain(full, stages, wait.err);
}

// Longer rows: a cluster a row, each CTA a quarter of the columns, as above in
// rows that start anywhere.  The rows of a whole ring are summed before the
// CTAs' sums are exchanged, so that the cluster meets once for up to eight rows.
// 2048 x 16384 f32 104 us (5.1 TB/s; in two passes over memory 127), 127 x 16385
// 16 (19), 1000 x 32768 bf16 72 (109).  Clusters of eight with a full ring an SM
// find room for fewer than half as many rows at a time: 234, 25, 144.
constexpr int kCluster = 4;
template <int TX, int T, int V>
__global__ void __launch_bounds__(T, 1) rmsnorm_bwd_cluster_kernel(const NormBwdArgs whole, float *partial,
                                                                   int stages, Waits wait) {
  constexpr int E = 16 / bytes_of(TX), WARPS = T / 32;
  static_assert(WARPS >= kMaxRing, "a warp a row of the ring");
  using P = Piece<TX, E>;
  pdl_launch_dependents();
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ float2 warp_sums[kMaxRing][WARPS];
  __shared__ float2 sums[2][kMaxRing][kCluster];
  __shared__ float edges[kMaxRing][3][32];  // dy, h, dh outside the pieces; [0][31]: the given rstd
  __shared__ __align__(8) uint64_t full[kMaxRing + 1];  // a stage each; the test hook's
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int rank = (int)blockIdx.x % kCluster;
  const int64_t first = blockIdx.x / kCluster, hop = gridDim.x / kCluster;
  const int slice = (whole.cols + kCluster - 1) / kCluster, col0 = rank * slice;
  NormBwdArgs a = whole;  // this CTA's columns
  a.cols = min(slice, whole.cols - col0);
  a.dy = at<TX>(whole.dy, col0);
  a.h = at<TX>(whole.h, col0);
  if (whole.dh) a.dh = at<TX>(whole.dh, col0);
  a.dx = static_cast<char *>(whole.dx) + (int64_t)col0 * bytes_of(TX);
  a.weight = static_cast<const char *>(whole.weight) + (int64_t)col0 * (whole.tw == MM_F32 ? 4 : 2);
  // the slices differ by a column or so: the largest one's ring in every CTA
  const uint32_t stage_bytes = (a.dh ? 3 : 2) * ring_row<true>((uint32_t)slice * bytes_of(TX));
  if (t == 0) {
    for (int s = 0; s <= kMaxRing; ++s) tc::mbar_init(tc::smem_u32(full + s), 1);
    tc::mbar_init_fence();
  }
  tc::cluster_sync_all();  // the others run: their memory may be written
  pdl_wait();
  const int64_t count = (a.rows - first + hop - 1) / hop;  // rows of this cluster
  auto fill = [&](int64_t k, int s) {
    ring_fill<TX, true>(a, first + k * hop, tc::smem_u32(ring) + (uint32_t)s * stage_bytes, tc::smem_u32(full + s));
  };
  if (t == 0)
    for (int s = 0; s < stages && s < count; ++s) fill(s, s);
  const RingPlace at_row = ring_place<TX, true>(a, first);
  const int head = at_row.head, edge = at_row.edge(lane, a.cols);
  const int n = max(0, (at_row.end - head - t * E + T * E - 1) / (T * E));  // this thread's pieces
  float e_dy = 0.f, e_h = 0.f, e_dh = 0.f;
  auto load_edges = [&](int64_t k) {  // a warp a row of the ring that starts with the k-th
    k += warp;
    if (warp >= stages || k >= count) return;
    const int64_t r = first + k * hop;
    if (edge >= 0) {
      e_dy = load_value(a.dy, TX, r * a.lddy + edge);
      e_h = load_value(a.h, TX, r * a.ldh + edge);
      if (a.dh) e_dh = load_value(a.dh, TX, r * a.lddh + edge);
    }
    if (lane == 31 && a.rstd) e_dy = a.rstd[r];
  };
  load_edges(0);
  float w[V][E], dw[V][E] = {};
  load_pieces_at(a.weight, a.tw, head + t * E, T * E, n, at_row.s_w, w);
  const float ew = edge >= 0 ? load_value(a.weight, a.tw, edge) : 0.f;
  float edw = 0.f;
  const float per_col = 1.f / (float)whole.cols;
  int side = 0;
  bool gave_up = wait.stall && !tc::thread_wait(tc::smem_u32(full + kMaxRing), 0, wait, kErrRing);  // as in the ring
  for (int64_t k0 = 0; k0 < count; k0 += stages, side ^= 1) {
    const int nb = (int)min((int64_t)stages, count - k0);
    if (warp < stages) edges[warp][0][lane] = e_dy, edges[warp][1][lane] = e_h, edges[warp][2][lane] = e_dh;
    __syncthreads();
    for (int s = 0; s < nb; ++s) {
      const uint8_t *stage = ring + (size_t)s * stage_bytes;
      float dot = 0.f, ss = 0.f;
      if (warp == 0 && edge >= 0) {
        const float eh = edges[s][1][lane];
        dot = edges[s][0][lane] * ew * eh;
        ss = eh * eh;
      }
      if (!gave_up && !tc::thread_wait(tc::smem_u32(full + s), (uint32_t)side, wait, kErrRing)) gave_up = true;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (v < n)
          BwdPiece<TX, E>::sums(ring_piece<TX, true>(stage + at_row.o_dy, v * T + t, at_row.s_dy),
                                ring_piece<TX, true>(stage + at_row.o_h, v * T + t, at_row.s_h), w[v], dot, ss);
      dot = row_sum<32>(dot, nullptr);
      ss = row_sum<32>(ss, nullptr);
      if (lane == 0) warp_sums[s][warp] = make_float2(dot, ss);
    }
    __syncthreads();
    if (warp < nb) {
      const float2 x = lane < WARPS ? warp_sums[warp][lane] : make_float2(0.f, 0.f);
      const float dot = row_sum<32>(x.x, nullptr), ss = row_sum<32>(x.y, nullptr);
      if (lane < kCluster) {
        const uint32_t to = tc::map_to_rank(tc::smem_u32(&sums[side][warp][rank]), (uint32_t)lane);
        tc::st_cluster_f32(to, dot);
        tc::st_cluster_f32(to + 4, ss);
      }
    }
    // `side`'s sums are written again after the next meeting, which no CTA comes to
    // before it has read these.
    tc::cluster_sync_all();
    load_edges(k0 + stages);
    for (int s = 0; s < nb; ++s) {
      const uint8_t *stage = ring + (size_t)s * stage_bytes;
      const int64_t r = first + (k0 + s) * hop;
      float dot = 0.f, ss = 0.f;
#pragma unroll
      for (int q = 0; q < kCluster; ++q) dot += sums[side][s][q].x, ss += sums[side][s][q].y;
      const float rs = a.rstd ? edges[s][0][31] : 1.f / sqrtf(ss / (float)whole.cols + a.eps);
      const float c = dot * per_col * rs * rs;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int i = v * T + t;
        if (v < n) {
          float dx[E];
          P d;
          if (a.dh) d = ring_piece<TX, true>(stage + at_row.o_dh, i, at_row.s_dh);
          BwdPiece<TX, E>::outputs(ring_piece<TX, true>(stage + at_row.o_dy, i, at_row.s_dy),
                                   ring_piece<TX, true>(stage + at_row.o_h, i, at_row.s_h), a.dh ? &d : nullptr, w[v],
                                   rs, c, dx, dw[v]);
          store_piece<TX>(a.dx, r * a.lddx + head + i * E, dx);
        }
      }
      if (warp == 0 && edge >= 0) {
        const float g = edges[s][0][lane], x = edges[s][1][lane];
        store_value(a.dx, TX, r * a.lddx + edge, rs * (g * ew - x * c) + edges[s][2][lane]);
        edw += g * x * rs;
      }
      __syncthreads();  // the stage, and in the end the edges, have been read
      if (t == 0 && !gave_up && k0 + stages + s < count) fill(k0 + stages + s, s);
    }
  }
  if (partial) {
    float *out = partial + first * partial_ld(whole.cols) + col0;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (v < n)
#pragma unroll
        for (int e = 0; e < E; ++e) out[head + (v * T + t) * E + e] = dw[v][e];
    if (warp == 0 && edge >= 0) out[edge] = edw;
  }
  if (gave_up && t == 0) ring_drain(full, stages, wait.err);
}

// Longer rows still, and dy of another type than h: 1 / rms and the mean of g h of each row (two
// floats a row), then columns in slices, each thread walking down the rows.
template <int TX, int E>
__global__ void __launch_bounds__(1024) rmsnorm_bwd_stats_kernel(const NormBwdArgs a, float2 *stats) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ float sh[64];
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    float dot = 0.f, ss = 0.f;
    constexpr int U = E == 1 ? 4 : 2;  // pieces in flight
    for (int j0 = threadIdx.x * E; j0 < a.cols; j0 += U * 1024 * E) {
      float dy[U][E], h[U][E], w[U][E];
      const int n = pieces_below<U>(j0, 1024 * E, a.cols);
      load_pieces(a.dy, a.ty, r * a.lddy + j0, 1024 * E, n, dy);
      load_pieces<TX>(a.h, r * a.ldh + j0, 1024 * E, n, h);
      load_pieces(a.weight, a.tw, j0, 1024 * E, n, w);
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < E; ++e) {
          dot += dy[u][e] * w[u][e] * h[u][e];
          ss += h[u][e] * h[u][e];
        }
    }
    __syncthreads();
    dot = row_sum<1024>(dot, sh);
    ss = row_sum<1024>(ss, sh + 32);
    if (threadIdx.x == 0) {
      const float rs = a.rstd ? a.rstd[r] : 1.f / sqrtf(ss / (float)a.cols + a.eps);
      stats[r] = make_float2(rs, dot / (float)a.cols * rs * rs);
    }
  }
}
template <int TX, int E>
__global__ void __launch_bounds__(256) rmsnorm_bwd_cols_kernel(const NormBwdArgs a, const float2 *stats,
                                                               float *partial) {
  pdl_launch_dependents();
  pdl_wait();
  const int j = ((int)blockIdx.x * 256 + (int)threadIdx.x) * E;
  if (j >= a.cols) return;
  float w[E], dw[E] = {};
  load_piece(a.weight, a.tw, j, w);
  constexpr int U = E == 1 ? 4 : 2;  // rows in flight
  for (int64_t r0 = blockIdx.y; r0 < a.rows; r0 += (int64_t)U * gridDim.y) {
    float dy[U][E], h[U][E], dh[U][E] = {};
    float2 s[U];
    const int n = pieces_below<U>(r0, gridDim.y, a.rows);
    load_pieces(a.dy, a.ty, r0 * a.lddy + j, gridDim.y * a.lddy, n, dy);
    load_pieces<TX>(a.h, r0 * a.ldh + j, gridDim.y * a.ldh, n, h);
    if (a.dh) load_pieces<TX>(a.dh, r0 * a.lddh + j, gridDim.y * a.lddh, n, dh);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (u < n) s[u] = stats[r0 + (int64_t)u * gridDim.y];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = r0 + (int64_t)u * gridDim.y;
      if (r < a.rows) {
        float dx[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
          dx[e] = dh[u][e] + s[u].x * (dy[u][e] * w[e] - h[u][e] * s[u].y);
          dw[e] += dy[u][e] * h[u][e] * s[u].x;
        }
        store_piece<TX>(a.dx, r * a.lddx + j, dx);
      }
    }
  }
  if (partial) store_piece<MM_F32>(partial, (int64_t)blockIdx.y * ((a.cols + 3) / 4 * 4) + j, dw);
}

// dweight: the parts of each column added in a fixed order: thread y of 32 adds
// every 32nd part, eight loads in flight, then the 32 sums are added in order.
__global__ void __launch_bounds__(1024) rmsnorm_dweight_kernel(const float *partial, int parts, int cols,
                                                               void *dweight, int tw) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ float sh[32][33];
  const int c = threadIdx.x & 31, y = threadIdx.x >> 5, j = (int)blockIdx.x * 32 + c;
  const int64_t ld = partial_ld(cols);
  float s = 0.f;
  if (j < cols)
    for (int q = y; q < parts; q += 8 * 32) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = q + 32 * k < parts ? partial[(int64_t)(q + 32 * k) * ld + j] : 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) s += v[k];
    }
  sh[y][c] = s;
  __syncthreads();
  if (y < 4) {  // four warps, eight columns each: lane (column, quarter of the sums)
    const int col = y * 8 + (c & 7), part = c >> 3;
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) v += sh[part * 8 + k][col];
    v += __shfl_down_sync(0xffffffffu, v, 16);
    v += __shfl_down_sync(0xffffffffu, v, 8);
    const int jj = (int)blockIdx.x * 32 + col;
    if (c < 8 && jj < cols) store_value(dweight, tw, jj, v);
  }
}

mm_status partial_space(const NormBwdArgs &a, int64_t parts, size_t more, LaunchCtx &ctx, float **out) {
  void *w = nullptr;
  const size_t bytes = (size_t)parts * (size_t)((a.cols + 3) / 4 * 4) * sizeof(float) + more;
  mm_status st = get_scratch(ctx, SCRATCH_WORKSPACE, bytes, &w);
  *out = static_cast<float *>(w);
  return st;
}

mm_status add_parts(const NormBwdArgs &a, const float *partial, int parts, LaunchCtx &ctx) {
  return launch(rmsnorm_dweight_kernel, (a.cols + 31) / 32, 1024, ctx, "rmsnorm_backward launch (dweight)", partial,
                parts, a.cols, a.dweight, a.tw);
}

// `blocks` blocks of a kernel that leaves a part of dweight a block.
template <typename K, typename... Args>
mm_status bwd_blocks(const NormBwdArgs &a, K kern, int64_t blocks, int threads, size_t smem, LaunchCtx &ctx,
                     Args... args) {
  float *partial = nullptr;
  mm_status st;
  if (a.dweight && (st = partial_space(a, blocks, 0, ctx, &partial)) != MM_OK) return st;
  cudaError_t e = launch_pdl(kern, dim3((unsigned)blocks), dim3((unsigned)threads), smem, ctx.stream, dim3(1), a,
                             partial, args...);
  if (e != cudaSuccess) return cuda_error(e, "rmsnorm_backward launch");
  count_operator_launch();
  return a.dweight ? add_parts(a, partial, (int)blocks, ctx) : MM_OK;
}

template <int TX, int E, int V>
mm_status bwd_warps_form(const NormBwdArgs &a, LaunchCtx &ctx) {
  // as many blocks as are resident at once: one more would be a second, nearly
  // empty round over its share of the rows (65536 x 512 bf16: 2 an SM 50 us, 3 60)
  static PerDevice<int> fits;
  auto kern = rmsnorm_bwd_warps_kernel<TX, E, V>;
  int per_sm = 0;
  const cudaError_t err = fits.get(ctx.dev->info.ordinal, &per_sm, [&](int *n) {
    return cudaOccupancyMaxActiveBlocksPerMultiprocessor(n, kern, 256, 0);
  });
  if (err != cudaSuccess) return cuda_error(err, "rmsnorm_backward set-up");
  const int64_t blocks = std::min<int64_t>((a.rows + 7) / 8, (int64_t)std::max(1, per_sm) * ctx.dev->info.sms);
  return bwd_blocks(a, kern, blocks, 256, 0, ctx);
}

constexpr size_t kRingBytes = 208 << 10;  // of an SM's shared memory

template <int TX, int T, int V, int PER_SM, bool EDGES>
mm_status bwd_ring_form(const NormBwdArgs &a, LaunchCtx &ctx) {
  static PerDevice<int> set_up;
  auto kern = rmsnorm_bwd_ring_kernel<TX, T, V, PER_SM, EDGES>;
  int done;
  const cudaError_t err = set_up.get(ctx.dev->info.ordinal, &done, [&](int *) {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRingBytes);
  });
  if (err != cudaSuccess) return cuda_error(err, "rmsnorm_backward set-up");
  const size_t stage = (size_t)(a.dh ? 3 : 2) * ring_row<EDGES>((uint32_t)a.cols * bytes_of(TX));
  const int stages = (int)std::min<size_t>(kMaxRing, kRingBytes / PER_SM / stage);
  if (stages < 2) return set_error(MM_ERR_UNSUPPORTED, "rmsnorm_backward: no two rows fit the ring");
  constexpr int E = 16 / bytes_of(TX);
  const int64_t most = (int64_t)PER_SM * ctx.dev->info.sms;
  const int64_t blocks = std::min<int64_t>(a.rows, EDGES ? std::max<int64_t>(E, most / E * E) : most);
  return bwd_blocks(a, kern, blocks, T, stages * stage, ctx, stages, operator_waits(ctx));
}

template <int TX, int T, int V>
mm_status bwd_cluster_form(const NormBwdArgs &a, LaunchCtx &ctx) {
  static PerDevice<int> fits;
  auto kern = rmsnorm_bwd_cluster_kernel<TX, T, V>;
  int resident = 0;  // clusters
  const cudaError_t err = fits.get(ctx.dev->info.ordinal, &resident, [&](int *n) -> cudaError_t {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRingBytes);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute cluster = {};
    cluster.id = cudaLaunchAttributeClusterDimension;
    cluster.val.clusterDim.x = kCluster;
    cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
    cudaLaunchConfig_t config = {};
    config.gridDim = dim3(kCluster);
    config.blockDim = dim3(T);
    config.dynamicSmemBytes = kRingBytes;
    config.attrs = &cluster;
    config.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(n, kern, &config);
  });
  if (err != cudaSuccess) return cuda_error(err, "rmsnorm_backward set-up");
  constexpr int E = 16 / bytes_of(TX);
  const size_t stage = (size_t)(a.dh ? 3 : 2) * ring_row<true>((uint32_t)((a.cols + kCluster - 1) / kCluster) * bytes_of(TX));
  const int stages = (int)std::min<size_t>(kMaxRing, kRingBytes / stage);
  if (stages < 1) return set_error(MM_ERR_UNSUPPORTED, "rmsnorm_backward: no row fits the ring");
  // a cluster's rows all lie alike: a multiple of E clusters, or one row each
  const int64_t most = std::max<int64_t>(E, resident / E * E);
  const int64_t clusters = std::min<int64_t>(a.rows, most);
  float *partial = nullptr;
  mm_status st;
  if (a.dweight && (st = partial_space(a, clusters, 0, ctx, &partial)) != MM_OK) return st;
  cudaError_t e = launch_pdl(kern, dim3((unsigned)(clusters * kCluster)), dim3(T), stages * stage, ctx.stream,
                             dim3(kCluster), a, partial, stages, operator_waits(ctx));
  if (e != cudaSuccess) return cuda_error(e, "rmsnorm_backward launch (clusters)");
  count_operator_launch();
  return a.dweight ? add_parts(a, partial, (int)clusters, ctx) : MM_OK;
}

template <int TX, int E>
mm_status bwd_long_form(const NormBwdArgs &a, LaunchCtx &ctx) {
  const int64_t slices = ((int64_t)a.cols + 256 * E - 1) / (256 * E);
  const int64_t down = std::max<int64_t>(1, std::min<int64_t>(a.rows, 8 * ctx.dev->info.sms / slices));
  float *partial = nullptr;
  mm_status st = partial_space(a, a.dweight ? down : 0, (size_t)a.rows * sizeof(float2), ctx, &partial);
  if (st != MM_OK) return st;
  float2 *stats = reinterpret_cast<float2 *>(partial + (a.dweight ? down * ((a.cols + 3) / 4 * 4) : 0));
  st = launch(rmsnorm_bwd_stats_kernel<TX, E>, std::min<int64_t>(a.rows, 2 * ctx.dev->info.sms), 1024, ctx,
              "rmsnorm_backward launch (statistics)", a, stats);
  if (st != MM_OK) return st;
  cudaError_t e = launch_pdl(rmsnorm_bwd_cols_kernel<TX, E>, dim3((unsigned)slices, (unsigned)down), dim3(256), 0,
                             ctx.stream, dim3(1), a, (const float2 *)stats, a.dweight ? partial : (float *)nullptr);
  if (e != cudaSuccess) return cuda_error(e, "rmsnorm_backward launch (columns)");
  count_operator_launch();
  return a.dweight ? add_parts(a, partial, (int)down, ctx) : MM_OK;
}

template <int TX, bool EDGES>
mm_status bwd_form(const NormBwdArgs &a, LaunchCtx &ctx) {
  constexpr int E = 16 / bytes_of(TX);
  const int pieces = a.cols / E;
  if (a.ty == TX) {
    if constexpr (!EDGES) {
      if (pieces <= 32) return bwd_warps_form<TX, E, 1>(a, ctx);
      if (pieces <= 64) return bwd_warps_form<TX, E, 2>(a, ctx);
      if (pieces <= 128) return bwd_warps_form<TX, E, 4>(a, ctx);
    } else {
      // Rows that start anywhere: up to 512 elements a warp and an element an
      // access (50000 x 333 bf16: 49 us; the ring with 64 threads 84), above that
      // the ring (33000 x 1001 74 us, an element an access 91; 8192 x 4097 70 and
      // 130; 2000 x 16383 84 and 201).
      if (a.cols <= 128) return bwd_warps_form<TX, 1, 4>(a, ctx);
      if (a.cols <= 256) return bwd_warps_form<TX, 1, 8>(a, ctx);
      if (a.cols <= 512) return bwd_warps_form<TX, 1, 16>(a, ctx);
      if (pieces <= 128) return bwd_ring_form<TX, 128, 1, 8, EDGES>(a, ctx);
    }
    // Threads and blocks an SM, measured (bf16, us for 33.5 M values in rows of
    // 2048 / 4096 / 8192): 256 x 5 52.6 (x 4 66, x 3 76) / 512 x 2 50.6 (256 x
    // 3 56; 512 x 3, of which two fit, 72) / 512 x 2 53 (1024 x 1 55)
    if (pieces <= 256) return bwd_ring_form<TX, 256, 1, 5, EDGES>(a, ctx);
    if (pieces <= 512) return bwd_ring_form<TX, 512, 1, 2, EDGES>(a, ctx);
    if (pieces <= 1024) return bwd_ring_form<TX, 512, 2, 2, EDGES>(a, ctx);
    if (pieces <= 2048) return bwd_ring_form<TX, 1024, 2, 1, EDGES>(a, ctx);
    const int in_slice = (a.cols + kCluster - 1) / kCluster / E;
    if (in_slice <= 512) return bwd_cluster_form<TX, 512, 1>(a, ctx);
    if (in_slice <= 1024) return bwd_cluster_form<TX, 512, 2>(a, ctx);
    if (in_slice <= 2048) return bwd_cluster_form<TX, 1024, 2>(a, ctx);
  }
  return bwd_long_form<TX, EDGES ? 1 : E>(a, ctx);
}

template <int TX>
mm_status bwd_type(const NormBwdArgs &a, LaunchCtx &ctx) {
  Alignment al;
  al.cols = a.cols;
  al.operand(a.dy, a.lddy, a.rows, type_size(a.ty));
  al.operand(a.dh, a.lddh, a.rows, type_size(a.tx));
  al.operand(a.h, a.ldh, a.rows, type_size(a.tx));
  al.operand(a.weight, 0, 1, type_size(a.tw));
  al.operand(a.dx, a.lddx, a.rows, type_size(a.tx));
  constexpr int most = 16 / bytes_of(TX);
  return al.elements(most) == most ? bwd_form<TX, false>(a, ctx) : bwd_form<TX, true>(a, ctx);
}

}  // namespace

mm_status launch_rmsnorm(const NormArgs &a, LaunchCtx &ctx) {
  return a.tx == MM_BF16  ? forward_type<MM_BF16>(a, ctx)
         : a.tx == MM_F16 ? forward_type<MM_F16>(a, ctx)
                          : forward_type<MM_F32>(a, ctx);
}

mm_status launch_rmsnorm_backward(const NormBwdArgs &a, LaunchCtx &ctx) {
  if (a.rows == 0)  // dweight of no rows
    return add_parts(a, nullptr, 0, ctx);
  return a.tx == MM_BF16  ? bwd_type<MM_BF16>(a, ctx)
         : a.tx == MM_F16 ? bwd_type<MM_F16>(a, ctx)
                          : bwd_type<MM_F32>(a, ctx);
}

}  // namespace mm
