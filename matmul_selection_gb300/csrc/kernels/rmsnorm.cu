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
// Statistics are fp32 sums.  Rows longer than the registers hold, and rows that
// do not start on 16 bytes, have forms of their own below.
#include <algorithm>
#include <type_traits>

#include "../operators.h"
#include "values.cuh"

namespace mm {

namespace {

constexpr float kE4m3Max = 448.f;

// ---------------------------------------------------------------- elements
template <int TX>
struct Elem {  // bf16
  using T = __nv_bfloat16;
  static __device__ __forceinline__ float get(T v) { return __bfloat162float(v); }
  static __device__ __forceinline__ T put(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Elem<MM_F16> {
  using T = __half;
  static __device__ __forceinline__ float get(T v) { return __half2float(v); }
  static __device__ __forceinline__ T put(float v) { return __float2half_rn(v); }
};
template <>
struct Elem<MM_F32> {
  using T = float;
  static __device__ __forceinline__ float get(T v) { return v; }
  static __device__ __forceinline__ T put(float v) { return v; }
};

// E neighbours of type TX as one access.
template <int TX, int E>
struct alignas(E * sizeof(typename Elem<TX>::T)) Piece {
  typename Elem<TX>::T v[E];
};
template <int TX, int E>
__device__ __forceinline__ void load_piece(const void *p, int64_t i, float (&out)[E]) {
  const Piece<TX, E> x = *reinterpret_cast<const Piece<TX, E> *>(static_cast<const typename Elem<TX>::T *>(p) + i);
#pragma unroll
  for (int e = 0; e < E; ++e) out[e] = Elem<TX>::get(x.v[e]);
}
template <int TX, int E>
__device__ __forceinline__ void store_piece(void *p, int64_t i, const float (&v)[E]) {
  Piece<TX, E> x;
#pragma unroll
  for (int e = 0; e < E; ++e) x.v[e] = Elem<TX>::put(v[e]);
  *reinterpret_cast<Piece<TX, E> *>(static_cast<typename Elem<TX>::T *>(p) + i) = x;
}
// The same for a type that is known only at run time (the same for every
// thread).
template <int E>
__device__ __forceinline__ void load_piece(const void *p, int t, int64_t i, float (&out)[E]) {
  if (t == MM_BF16) load_piece<MM_BF16>(p, i, out);
  else if (t == MM_F16) load_piece<MM_F16>(p, i, out);
  else load_piece<MM_F32>(p, i, out);
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
// T threads a row (256 threads a block, or T), V pieces of E elements a thread:
// the row of T V E elements or fewer stays in registers.  Pieces past cols are
// not accessed (cols is a multiple of E).
template <int TX, int E, int T, int V>
__global__ void __launch_bounds__(T < 256 ? 256 : T) rmsnorm_rows_kernel(const NormArgs a) {
  constexpr int ROWS = T < 256 ? 256 / T : 1;
  pdl_launch_dependents();
  pdl_wait();
  __shared__ float sh[2 * (T / 32)];
  const int t = threadIdx.x % T;
  const int64_t r = (int64_t)blockIdx.x * ROWS + threadIdx.x / T;
  if (T < 256 && r >= a.rows) return;  // (T = 32: no barrier below)
  float h[V][E];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int j = (v * T + t) * E;
    if (j < a.cols) {
      load_piece<TX>(a.x, r * a.ldx + j, h[v]);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) h[v][e] = 0.f;
    }
  }
  if (a.residual) {
    float res[V][E];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int j = (v * T + t) * E;
      if (j < a.cols) {
        load_piece<TX>(a.residual, r * a.ldr + j, res[v]);
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) res[v][e] = 0.f;
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < E; ++e) h[v][e] += res[v][e];
  }
  float w[V][E];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int j = (v * T + t) * E;
    if (j < a.cols) load_piece(a.weight, a.tw, j, w[v]);
  }
  float ss = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int e = 0; e < E; ++e) ss += h[v][e] * h[v][e];
  if (a.h) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int j = (v * T + t) * E;
      if (j < a.cols) store_piece<TX>(a.h, r * a.ldh + j, h[v]);
    }
  }
  float inv = 1.f;
  if (a.scale) {
    uint32_t big = 0;  // of |h w|: y is this times rstd
#pragma unroll
    for (int v = 0; v < V; ++v)
      if ((v * T + t) * E < a.cols)
#pragma unroll
        for (int e = 0; e < E; ++e) {
          h[v][e] *= w[v][e];
          big = max(big, __float_as_uint(fabsf(h[v][e])));
        }
    row_sum_max<T>(ss, big, sh);
    const float rstd = 1.f / sqrtf(ss / (float)a.cols + a.eps);
    const float scale = row_scale(__uint_as_float(big) * rstd);
    inv = rstd * (1.f / scale);
    if (t == 0) {
      a.scale[r] = scale;
      if (a.rstd) a.rstd[r] = rstd;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int j = (v * T + t) * E;
      if (j < a.cols) {
#pragma unroll
        for (int e = 0; e < E; ++e) h[v][e] *= inv;
        store_piece(a.y, MM_E4M3, r * a.ldy + j, h[v]);
      }
    }
  } else {
    ss = row_sum<T>(ss, sh);
    const float rstd = 1.f / sqrtf(ss / (float)a.cols + a.eps);
    if (a.rstd && t == 0) a.rstd[r] = rstd;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int j = (v * T + t) * E;
      if (j < a.cols) {
#pragma unroll
        for (int e = 0; e < E; ++e) h[v][e] = h[v][e] * rstd * w[v][e];
        store_piece(a.y, a.ty, r * a.ldy + j, h[v]);
      }
    }
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
    float ss = 0.f;
    uint32_t big = 0;
    for (int j = threadIdx.x * E; j < a.cols; j += 1024 * E) {
      float h[E];
      load_piece<TX>(a.x, r * a.ldx + j, h);
      if (a.residual) {
        float s[E];
        load_piece<TX>(a.residual, r * a.ldr + j, s);
#pragma unroll
        for (int e = 0; e < E; ++e) h[e] += s[e];
      }
#pragma unroll
      for (int e = 0; e < E; ++e) ss += h[e] * h[e];
      if (a.scale) {
        float w[E];
        load_piece(a.weight, a.tw, j, w);
#pragma unroll
        for (int e = 0; e < E; ++e) big = max(big, __float_as_uint(fabsf(h[e] * w[e])));
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
    for (int j = threadIdx.x * E; j < a.cols; j += 1024 * E) {
      float h[E], w[E];
      load_piece<TX>(a.x, r * a.ldx + j, h);
      if (a.residual) {
        float s[E];
        load_piece<TX>(a.residual, r * a.ldr + j, s);
#pragma unroll
        for (int e = 0; e < E; ++e) h[e] += s[e];
      }
      load_piece(a.weight, a.tw, j, w);
      if (a.h) store_piece<TX>(a.h, r * a.ldh + j, h);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        h[e] = h[e] * rstd * w[e];
        if (a.scale) h[e] *= inv;
      }
      store_piece(a.y, a.ty, r * a.ldy + j, h);
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

template <int TX, int E, int T, int V>
mm_status rows_form(const NormArgs &a, LaunchCtx &ctx) {
  constexpr int ROWS = T < 256 ? 256 / T : 1;
  const int64_t blocks = (a.rows + ROWS - 1) / ROWS;
  if (blocks >= (1LL << 31)) return set_error(MM_ERR_UNSUPPORTED, "too many rows");
  return launch(rmsnorm_rows_kernel<TX, E, T, V>, blocks, T < 256 ? 256 : T, ctx, "rmsnorm launch", a);
}

// A warp a row up to 128 pieces, then a block of 256 to 1024.
template <int TX, int E>
mm_status forward_form(const NormArgs &a, LaunchCtx &ctx) {
  const int pieces = (a.cols + E - 1) / E;
  if (pieces <= 64) return rows_form<TX, E, 32, 2>(a, ctx);
  if (pieces <= 128) return rows_form<TX, E, 32, 4>(a, ctx);
  if (pieces <= 256) return rows_form<TX, E, 256, 1>(a, ctx);
  if constexpr (E > 1) {
    if (pieces <= 512) return rows_form<TX, E, 256, 2>(a, ctx);
    if (pieces <= 1024) return rows_form<TX, E, 512, 2>(a, ctx);
    if (pieces <= 2048) return rows_form<TX, E, 1024, 2>(a, ctx);
  } else {
    if (pieces <= 1024) return rows_form<TX, E, 256, 4>(a, ctx);
    if (pieces <= 2048) return rows_form<TX, E, 512, 4>(a, ctx);
    if (pieces <= 4096) return rows_form<TX, E, 1024, 4>(a, ctx);
    if (pieces <= 6144) return rows_form<TX, E, 1024, 6>(a, ctx);
    if (pieces <= 8192) return rows_form<TX, E, 1024, 8>(a, ctx);
    if (pieces <= 16384) return rows_form<TX, E, 1024, 16>(a, ctx);
  }
  return launch(rmsnorm_long_kernel<TX, E>, std::min<int64_t>(a.rows, 2 * ctx.dev->info.sms), 1024, ctx,
                "rmsnorm launch (long rows)", a);
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
  constexpr int most = 16 / sizeof(typename Elem<TX>::T);
  return al.elements(most) == most ? forward_form<TX, most>(a, ctx) : forward_form<TX, 1>(a, ctx);
}

// ---------------------------------------------------------------- backward
// A block of T threads walks rows blockIdx.x, blockIdx.x + gridDim.x, ...; a
// thread holds the same V pieces of E columns of each (as they lie in memory,
// dy of x's type) and its own sums of dy h rstd.  The weight comes from L1 each
// time.  The blocks' sums go to a workspace and a second kernel adds them in
// block order.
template <int TX, int E, int T, int V>
__global__ void __launch_bounds__(T) rmsnorm_bwd_kernel(const NormBwdArgs a, float *partial) {
  using P = Piece<TX, E>;
  using X = typename Elem<TX>::T;
  pdl_launch_dependents();
  pdl_wait();
  __shared__ float sh[2][2 * (T / 32)];
  const int t = threadIdx.x;
  float dw[V][E];
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int e = 0; e < E; ++e) dw[v][e] = 0.f;
  P dy[V], h[V], dh[V];
  auto load = [&](int64_t r) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int j = (v * T + t) * E;
      if (j < a.cols) {
        dy[v] = *reinterpret_cast<const P *>(static_cast<const X *>(a.dy) + r * a.lddy + j);
        h[v] = *reinterpret_cast<const P *>(static_cast<const X *>(a.h) + r * a.ldh + j);
        if (a.dh) dh[v] = *reinterpret_cast<const P *>(static_cast<const X *>(a.dh) + r * a.lddh + j);
      }
    }
  };
  int side = 0;
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    load(r);
    const float given = a.rstd ? a.rstd[r] : 0.f;
    float dot = 0.f, ss = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int j = (v * T + t) * E;
      if (j < a.cols) {
        float w[E];
        load_piece(a.weight, a.tw, j, w);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float x = Elem<TX>::get(h[v].v[e]);
          dot += Elem<TX>::get(dy[v].v[e]) * w[e] * x;
          ss += x * x;
        }
      }
    }
    // two sets of shared sums in turn: one barrier a row
    dot = row_sum<T>(dot, sh[side]);
    float rs = given;
    if (!a.rstd) {
      ss = row_sum<T>(ss, sh[side] + T / 32);
      rs = 1.f / sqrtf(ss / (float)a.cols + a.eps);
    }
    side ^= 1;
    const float c = dot / (float)a.cols * rs * rs;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int j = (v * T + t) * E;
      if (j < a.cols) {
        float w[E], dx[E];
        load_piece(a.weight, a.tw, j, w);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float g = Elem<TX>::get(dy[v].v[e]), x = Elem<TX>::get(h[v].v[e]);
          dx[e] = rs * (g * w[e] - x * c);
          if (a.dh) dx[e] += Elem<TX>::get(dh[v].v[e]);
          dw[v][e] += g * x * rs;
        }
        store_piece<TX>(a.dx, r * a.lddx + j, dx);
      }
    }
  }
  if (partial)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int j = (v * T + t) * E;
      if (j < a.cols) store_piece<MM_F32>(partial, (int64_t)blockIdx.x * ((a.cols + 3) / 4 * 4) + j, dw[v]);
    }
}

// Rows too long for the registers: 1 / rms and the mean of g h of each row (two
// floats a row), then columns in slices, each thread walking down the rows.
template <int TX, int E>
__global__ void __launch_bounds__(1024) rmsnorm_bwd_stats_kernel(const NormBwdArgs a, float2 *stats) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ float sh[64];
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    float dot = 0.f, ss = 0.f;
    for (int j = threadIdx.x * E; j < a.cols; j += 1024 * E) {
      float dy[E], h[E], w[E];
      load_piece(a.dy, a.ty, r * a.lddy + j, dy);
      load_piece<TX>(a.h, r * a.ldh + j, h);
      load_piece(a.weight, a.tw, j, w);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        dot += dy[e] * w[e] * h[e];
        ss += h[e] * h[e];
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
  for (int64_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
    float dy[E], h[E], dx[E];
    load_piece(a.dy, a.ty, r * a.lddy + j, dy);
    load_piece<TX>(a.h, r * a.ldh + j, h);
    const float2 s = stats[r];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      dx[e] = s.x * (dy[e] * w[e] - h[e] * s.y);
      dw[e] += dy[e] * h[e] * s.x;
    }
    if (a.dh) {
      float dh[E];
      load_piece<TX>(a.dh, r * a.lddh + j, dh);
#pragma unroll
      for (int e = 0; e < E; ++e) dx[e] += dh[e];
    }
    store_piece<TX>(a.dx, r * a.lddx + j, dx);
  }
  if (partial) store_piece<MM_F32>(partial, (int64_t)blockIdx.y * ((a.cols + 3) / 4 * 4) + j, dw);
}

// dweight: the parts of each column added in their order, by runs: thread y of
// eight adds every eighth part, then the eight sums are added.
__global__ void __launch_bounds__(256) rmsnorm_dweight_kernel(const float *partial, int parts, int cols, void *dweight,
                                                              int tw) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ float sh[8][33];
  const int c = threadIdx.x & 31, y = threadIdx.x >> 5, j = (int)blockIdx.x * 32 + c;
  const int64_t ld = (cols + 3) / 4 * 4;
  float s = 0.f;
  if (j < cols) {
    int q = y;
    for (; q + 24 < parts; q += 32) {
      float v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = partial[(int64_t)(q + 8 * k) * ld + j];
#pragma unroll
      for (int k = 0; k < 4; ++k) s += v[k];
    }
    for (; q < parts; q += 8) s += partial[(int64_t)q * ld + j];
  }
  sh[y][c] = s;
  __syncthreads();
  if (y == 0 && j < cols) {
#pragma unroll
    for (int k = 1; k < 8; ++k) s += sh[k][c];
    store_value(dweight, tw, j, s);
  }
}

mm_status partial_space(const NormBwdArgs &a, int64_t parts, size_t more, LaunchCtx &ctx, float **out) {
  void *w = nullptr;
  const size_t bytes = (size_t)parts * (size_t)((a.cols + 3) / 4 * 4) * sizeof(float) + more;
  mm_status st = get_scratch(*ctx.dev, ctx.stream, SCRATCH_WORKSPACE, bytes, &w);
  *out = static_cast<float *>(w);
  return st;
}

mm_status add_parts(const NormBwdArgs &a, const float *partial, int parts, LaunchCtx &ctx) {
  return launch(rmsnorm_dweight_kernel, (a.cols + 31) / 32, 256, ctx, "rmsnorm_backward launch (dweight)", partial,
                parts, a.cols, a.dweight, a.tw);
}

template <int TX, int E, int T, int V>
mm_status bwd_rows_form(const NormBwdArgs &a, int per_sm, LaunchCtx &ctx) {
  const int64_t blocks = std::min<int64_t>(a.rows, (int64_t)per_sm * ctx.dev->info.sms);
  float *partial = nullptr;
  mm_status st;
  if (a.dweight && (st = partial_space(a, blocks, 0, ctx, &partial)) != MM_OK) return st;
  st = launch(rmsnorm_bwd_kernel<TX, E, T, V>, blocks, T, ctx, "rmsnorm_backward launch", a, partial);
  if (st != MM_OK || !a.dweight) return st;
  return add_parts(a, partial, (int)blocks, ctx);
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

template <int TX, int E>
mm_status bwd_form(const NormBwdArgs &a, LaunchCtx &ctx) {
  const int pieces = (a.cols + E - 1) / E;
  if (a.ty == TX) {
    if (pieces <= 128) return bwd_rows_form<TX, E, 128, 1>(a, 8, ctx);
    if (pieces <= 256) return bwd_rows_form<TX, E, 256, 1>(a, 4, ctx);
    if (pieces <= 512) return bwd_rows_form<TX, E, 256, 2>(a, 3, ctx);
    if (pieces <= 1024) return bwd_rows_form<TX, E, 512, 2>(a, 2, ctx);
    if (pieces <= 2048) return bwd_rows_form<TX, E, 1024, 2>(a, 1, ctx);
    if constexpr (E == 1)
      if (pieces <= 8192) return bwd_rows_form<TX, E, 1024, 8>(a, 1, ctx);
  }
  return bwd_long_form<TX, E>(a, ctx);
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
  constexpr int most = 16 / sizeof(typename Elem<TX>::T);
  return al.elements(most) == most ? bwd_form<TX, most>(a, ctx) : bwd_form<TX, 1>(a, ctx);
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
