// Pieces of rows in registers: neighbouring elements by one access, converted to
// fp32 and back, and pieces that start anywhere read as two whole ones.
#pragma once

#include "values.cuh"

namespace mm {
namespace {

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

}  // namespace
}  // namespace mm
