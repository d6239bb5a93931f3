// Products of few rows with quantised weights, held [N][K]:
//   4-bit  (at most 16 rows) out[m, n] = sum_k A[m, k] s[n, k / group] (q[n, k] - z[n, k / group])
//   e4m3   (at most 8) out[m, n] = scale_a[m] scale_b[n] sum_k A[m, k] B[n, k]
// One pass over the weights, which is what bounds them.  A CTA of eight
// computing warps owns R = 16 WR rows of the weights; WR warps side by side
// take 16 rows each, and WK = 8 / WR of them take turns along K, a panel (128
// bytes of each row) at a time.  The fewer rows A has, the fewer rows of the
// weights share its panels: R = 8 M keeps A's traffic from L2 below the
// weights'.  Panels of weights and of A come by TMA through a ring; the MMA is
// the warp-level one with the weights as its 16-row operand:
//   4-bit  ldmatrix hands each lane 8 neighbouring codes of a row and its
//          lane's 16 bytes of A hold the same 8 k; q - z is exact in 16 bits,
//          and the scale multiplies the fp32 sum of its group.
//   e4m3   m16n8k32 on the bytes as they are.
// The warps' parts (and those of a cluster's CTAs, which split K where there
// are few rows of weights) meet in the owner's shared memory and are added in
// order: one launch, the same bits every time.  Where K is not split a CTA stays
// and takes tiles in turn, its ring running on over them.
// Measured: e4m3 1 x 16384 x 8192 (in this form) 23.5 us, 5.7 TB/s, HBM-bound;
// 4-bit, groups of 128, 1 x 19456 x 16384 41 us (4.0 TB/s), 1 x 16384 x 8192 22, 16
// x 16384 x 8192 f16 with zero points 32.2 (2.3 TB/s): the instructions that make
// weights of codes, in 64 % (one row) and 45 % (16 rows) of the issue slots with the
// 16 computing warps an SM that registers allow.  1 x 4096 x 4096: 4.6 (e4m3 5.2), a
// launch's chain.
#include <algorithm>

#include "../operators.h"
#include "tcgen05.cuh"
#include "values.cuh"
#include "w4.cuh"

namespace mm {

namespace {

using namespace tc;

enum Format { FMT_W4_BF16 = MM_BF16, FMT_W4_F16 = MM_F16, FMT_E4M3 = MM_E4M3 };

constexpr int kWarps = 8;
constexpr int kThreads = 32 * (kWarps + 2);  // and two copying warps
constexpr int kStages = 4;
constexpr uint32_t kWeightsB = 16384, kRowsB = 8192;  // a stage's weights and rows of A
constexpr uint32_t kStageB = kWeightsB + kRowsB;
constexpr uint32_t kPartsB = 8192, kSlackB = 4096;  // (rows of A past M are read, not used)
constexpr size_t kSmem = kStages * kStageB + kSlackB + kPartsB + 1024 + 128;
constexpr int kErrCopy = 0xa01, kErrMma = 0xa02;

struct GemvParams {
  void *out;
  int64_t ldc;
  int tc;
  int M, N;
  int panels, panels_per_rank;
  const float *sa, *sb;
  W4Scales w;
  Waits wait;
};

// The loads and MMAs of a panel are left for the compiler to order (they are
// not volatile): what keeps them between the wait for the stage and its
// release is data, an address that is defined after the wait and sums that are
// complete before the release (see after_wait, before_release).
__device__ __forceinline__ void ldmatrix_x4(uint32_t a, uint32_t (&r)[4]) {
  asm("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(a));
}
__device__ __forceinline__ uint4 lds_16(uint32_t a) {
  uint4 v;
  asm("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t after_wait(uint32_t a) {
  asm volatile("" : "+r"(a)::"memory");
  return a;
}
template <int MT>
__device__ __forceinline__ void before_release(float (&acc)[MT][4]) {
#pragma unroll
  for (int m = 0; m < MT; ++m)
    asm volatile("" : "+f"(acc[m][0]), "+f"(acc[m][1]), "+f"(acc[m][2]), "+f"(acc[m][3])::"memory");
}
// D (16 x 8, fp32) += A (16 rows of weights) . B (8 rows of A).
template <int F>
__device__ __forceinline__ void mma_16x8(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
#define MM_MMA_SYNC(SHAPE_TYPES)                                                                        \
  asm("mma.sync.aligned." SHAPE_TYPES " {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};" \
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])                                         \
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1))
  if constexpr (F == FMT_W4_BF16) MM_MMA_SYNC("m16n8k16.row.col.f32.bf16.bf16.f32");
  if constexpr (F == FMT_W4_F16) MM_MMA_SYNC("m16n8k16.row.col.f32.f16.f16.f32");
  if constexpr (F == FMT_E4M3) MM_MMA_SYNC("m16n8k32.row.col.f32.e4m3.e4m3.f32");
#undef MM_MMA_SYNC
}
// The same into fresh sums.
template <int F>
__device__ __forceinline__ void mma_16x8_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
#define MM_MMA_SYNC(SHAPE_TYPES)                                                                        \
  asm("mma.sync.aligned." SHAPE_TYPES " {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};" \
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])                                         \
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f))
  if constexpr (F == FMT_W4_BF16) MM_MMA_SYNC("m16n8k16.row.col.f32.bf16.bf16.f32");
  else MM_MMA_SYNC("m16n8k16.row.col.f32.f16.f16.f32");
#undef MM_MMA_SYNC
}

// Where a lane's scales and zero points are: of its two rows, for the 64 codes
// of a panel from 64 t on (lane t of four), entry h those from 64 t + 32 h
// (TWO: groups of 32; else both entries are one).  A row past N stands for the
// last, and a group past the last one for that: their results are not used, or
// see scales_below_k.
struct ScaleCursor {
  const char *s[2];
  const uint8_t *z[2];
  int g, step, last;
};
struct PanelScales {
  uint32_t s[2][2];  // [row][h], as in memory
  uint32_t z[2][2];
};
__device__ __forceinline__ ScaleCursor scale_cursor(const W4Scales &w, int n, int k0, int k_step) {
  ScaleCursor c;
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int64_t at = (int64_t)min(n + 8 * r, w.N - 1) * w.lds;
    c.s[r] = static_cast<const char *>(w.s) + at * (w.ts == MM_F32 ? 4 : 2);
    c.z[r] = w.z + at;  // (not read without zero points)
  }
  c.g = k0 >> w.group_shift;
  c.step = k_step >> w.group_shift;
  c.last = w.groups - 1;
  return c;
}
template <bool TWO>
__device__ __forceinline__ void load_panel_scales(const W4Scales &w, ScaleCursor &c, PanelScales &s) {
#pragma unroll
  for (int h = 0; h < (TWO ? 2 : 1); ++h) {
    const int g = min(c.g + h, c.last);
    if (w.ts == MM_F32) {
#pragma unroll
      for (int r = 0; r < 2; ++r) s.s[r][h] = reinterpret_cast<const uint32_t *>(c.s[r])[g];
    } else {
#pragma unroll
      for (int r = 0; r < 2; ++r) s.s[r][h] = reinterpret_cast<const uint16_t *>(c.s[r])[g];
    }
    if (w.z) {
#pragma unroll
      for (int r = 0; r < 2; ++r) s.z[r][h] = c.z[r][g];
    }
  }
  c.g += c.step;
}
// Of K's last panel: where an entry's codes (from k on) all lie past K its scale is
// 0, so that an infinite scale of the last group stays with that group's codes.
template <bool TWO>
__device__ __forceinline__ void scales_below_k(PanelScales &s, int k, int K) {
#pragma unroll
  for (int h = 0; h < (TWO ? 2 : 1); ++h)
    if (k + 32 * h >= K) s.s[0][h] = s.s[1][h] = 0u;
}
// A byte b under a byte of zeros is b 2^-133 as a bf16 (and b 2^-24 as an f16):
// the denormals and the first binade lie on one line.  So a pair of codes that
// came in one byte needs two masks and one byte permutation, and one FMA, exact,
// makes (q - z) 2^-6 (f16: 2^-9) of both: the high code's factor is 1/16 of the
// low one's.  The results are scaled back when they are stored.
template <int F>
struct Unpack {
  static constexpr bool B = F == FMT_W4_BF16;
  static constexpr uint32_t kFactors = B ? 0x7d007f00u : 0x68007800u;  // 2^127 and 2^123; 2^15 and 2^11
  static constexpr uint32_t kMinus = B ? 0xff00ff00u : 0xf800f800u;    // -2^127; -2^15
  static constexpr float kBack = B ? 64.f : 512.f;
  using T = typename Pair16<F>::T;
  static __device__ __forceinline__ T minus_zero(uint32_t z) {  // -z 2^-6, twice
    return __hmul2(bits_as<T>((z & 15u) * 0x00010001u), bits_as<T>(kMinus));
  }
  static __device__ __forceinline__ uint32_t pair(uint32_t lo, uint32_t hi, int i, T minus_z) {
    uint32_t both;  // byte i of lo; zeros (lo's sign, which is 0); byte i of hi; zeros
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(both) : "r"(lo), "r"(hi), "r"(0x8480 + 0x1111 * i));
    return as_bits(__hfma2(bits_as<T>(both), bits_as<T>(kFactors), minus_z));
  }
};

// A panel of 16 rows of 4-bit weights (256 codes) times 8 MT rows of A.
template <int F, int MT, int XBLOCK, bool TWO, bool Z>
__device__ __forceinline__ void panel_w4(const GemvParams &p, uint32_t wrow, uint32_t xrow, const PanelScales &ps,
                                         float (&acc)[MT][4]) {
  using U = Unpack<F>;
  using T = typename U::T;
  constexpr int E = TWO ? 2 : 1;
  const int lane = threadIdx.x & 31;
  float scale[2][E];
  uint32_t zero[2][E];
  if (p.w.ts == MM_F16) {
#pragma unroll
    for (int i = 0; i < 2 * E; ++i)
      scale[i / E][i % E] = __half2float(__ushort_as_half((unsigned short)ps.s[i / E][i % E]));
  } else {
    const int shift = p.w.ts == MM_BF16 ? 16 : 0;
#pragma unroll
    for (int i = 0; i < 2 * E; ++i) scale[i / E][i % E] = __uint_as_float(ps.s[i / E][i % E] << shift);
  }
  if constexpr (Z)
#pragma unroll
    for (int i = 0; i < 2 * E; ++i) zero[i / E][i % E] = as_bits(U::minus_zero(ps.z[i / E][i % E]));
  const uint32_t rr = lane & 7, mat = lane >> 3;
  // A group of 64 or more is summed 64 codes at a time all the same: scaling
  // costs less than asking whether a group ends, and no branch stands between
  // one pair of chunks and the next.
#pragma unroll (MT == 2 ? 2 : 4)  // (four spill with two blocks of A's rows)
  for (int c2 = 0; c2 < 4; ++c2) {  // two chunks of 32 codes
    uint32_t w[4];  // rows r, r + 8 of the first; of the second
    ldmatrix_x4(wrow + (((2 * c2 + (mat >> 1)) ^ rr) << 4), w);
    const int src = (lane & 28) | c2;
    T z[2];
    float part[MT][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (TWO || h == 0)
#pragma unroll
        for (int r = 0; r < 2; ++r)
          z[r] = Z ? bits_as<T>(__shfl_sync(0xffffffffu, zero[r][h % E], src)) : U::minus_zero(8);
      uint32_t a[2][4];  // row, pairs (0, 1), (2, 3), (4, 5), (6, 7)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint32_t lo = w[2 * h + r] & 0x0f0f0f0fu, hi = w[2 * h + r] & 0xf0f0f0f0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) a[r][i] = U::pair(lo, hi, i, z[r]);
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const uint4 x = lds_16(XBLOCK ? (xrow ^ (uint32_t)(h << 6)) + (uint32_t)(c2 * XBLOCK + m * 1024)
                                      : xrow + (uint32_t)((2 * c2 + h) * 64));
        if (TWO || h == 0) mma_16x8_first<F>(part[m], a[0][0], a[1][0], a[0][1], a[1][1], x.x, x.y);
        else mma_16x8<F>(part[m], a[0][0], a[1][0], a[0][1], a[1][1], x.x, x.y);
        mma_16x8<F>(part[m], a[0][2], a[1][2], a[0][3], a[1][3], x.z, x.w);
      }
      if (TWO || h == 1) {
        const float s0 = __shfl_sync(0xffffffffu, scale[0][h % E], src);
        const float s1 = __shfl_sync(0xffffffffu, scale[1][h % E], src);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          acc[m][0] += s0 * part[m][0], acc[m][1] += s0 * part[m][1];
          acc[m][2] += s1 * part[m][2], acc[m][3] += s1 * part[m][3];
        }
      }
    }
  }
}

// A panel of 16 rows of e4m3 weights (128 bytes) times 8 MT rows of A.
template <int MT>
__device__ __forceinline__ void panel_e4m3(uint32_t wrow, uint32_t xpanel, float (&acc)[MT][4]) {
  const int lane = threadIdx.x & 31;
  const uint32_t rr = lane & 7, mat = lane >> 3;
#pragma unroll
  for (int s = 0; s < 4; s += 2) {
    uint32_t x[MT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)  // chunks 2 s .. 2 s + 3 of 8 rows of A
      ldmatrix_x4(xpanel + (uint32_t)(m * 1024) + rr * 128 + (((2 * s + mat) ^ rr) << 4), x[m]);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t w[4];
      ldmatrix_x4(wrow + (((2 * (s + h) + (mat >> 1)) ^ rr) << 4), w);
#pragma unroll
      for (int m = 0; m < MT; ++m)
        mma_16x8<FMT_E4M3>(acc[m], w[0], w[1], w[2], w[3], x[m][2 * h], x[m][2 * h + 1]);
    }
  }
}

__device__ __forceinline__ void computing_warps_sync() {
  asm volatile("barrier.cta.sync.aligned 1, %0;" ::"n"(32 * kWarps) : "memory");
}
// A panel of A is M rows of 512 bytes, which meet in the banks in pairs.  Where
// a warp reads two blocks of rows of A that costs more than copying the panel in
// four boxes of 128 bytes a row with TMA's swizzle (16 x 16384 x 8192: 37.8 us
// against 32.2; 8 rows: 20.8 against 21.4); this many bytes apart.
template <int F, int WR>
constexpr int kXBlock = F != FMT_E4M3 && WR == 8 ? 2048 : 0;
// Element o of a tile of M x cols from its parts (PARTS of them, or `parts`), in order.
template <int F, int PARTS>
__device__ __forceinline__ void store_sum(const GemvParams &p, const float *buf, int cols, int n0, int o,
                                          int parts = PARTS) {
  const int m = o / cols, n = n0 + o % cols;
  if (n >= p.N) return;
  float v = 0.f;
#pragma unroll
  for (int q = 0; q < (PARTS ? PARTS : parts); ++q) v += buf[q * p.M * cols + o];
  if constexpr (F != FMT_E4M3) v *= Unpack<F>::kBack;
  else v = v * (p.sa ? p.sa[m] : 1.f) * (p.sb ? p.sb[n] : 1.f);
  store_value(p.out, p.tc, (int64_t)m * p.ldc + n, v);
}

template <int F, int WR, bool TWO>
__global__ void __launch_bounds__(kThreads, 2)
    gemv_quant_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                      const GemvParams p) {
  constexpr int WK = kWarps / WR, R = 16 * WR, MT = WR == 8 ? 2 : 1;
  constexpr bool W4 = F != FMT_E4M3;
  constexpr uint32_t XPANEL = kRowsB / WK;  // 2 WR rows of 512 bytes, or 8 MT and more of 128
  constexpr int XBLOCK = kXBlock<F, WR>;
  pdl_launch_dependents();
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  float *parts = reinterpret_cast<float *>(smem + kStages * kStageB + kSlackB);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kStages * kStageB + kSlackB + kPartsB);
  const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * kStages;
  const uint32_t stall = empty0 + 8 * kStages;
  volatile int *abort_flag = reinterpret_cast<volatile int *>(bars + 2 * kStages + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ranks = (int)gridDim.y, rank = (int)blockIdx.y;  // a cluster along y splits K
  const int tile0 = (int)blockIdx.x, tiles = (p.N + R - 1) / R, hop = (int)gridDim.x;
  const int p0 = rank * p.panels_per_rank, np = max(0, min(p.panels_per_rank, p.panels - p0));
  const int steps = (np + WK - 1) / WK;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full0 + 8 * s, 2);  // both copying warps arm their bytes
      mbar_init(empty0 + 8 * s, kWarps);
    }
    mbar_init(stall, 1);
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == kWarps) {
    if (lane == 0) prefetch_tmap(&tmW);
    for (int i = lane; i < min(np, 64); i += 32) tma_prefetch_2d(&tmW, (p0 + i) * 128, tile0 * R);
  }
  if (warp == kWarps + 1 && lane == 0) prefetch_tmap(&tmX);
  if (ranks > 1) cluster_sync_all();  // the others run: their memory may be written
  else __syncthreads();
  pdl_wait();

  if (warp >= kWarps) {
    const bool weights = warp == kWarps;
    const uint32_t bytes = weights ? R * 128 : (uint32_t)p.M * (W4 ? 512u : 128u);
    const uint32_t offset = weights ? 0u : kWeightsB, pitch = weights ? R * 128 : XPANEL;
    const int kx = weights ? 128 : W4 ? 256 : 128;  // a panel in the map's elements
    const int boxes = weights || XBLOCK == 0 ? 1 : 4;
    int n = 0;  // stages filled
    bool ok = true;
    for (int tile = tile0; tile < tiles && ok; tile += hop)
      for (int i = 0; i < steps; ++i, ++n) {
        const int st = n % kStages;
        ok = warp_wait(empty0 + 8 * st, ((uint32_t)(n / kStages) & 1u) ^ 1u, abort_flag, p.wait, kErrCopy);
        if (!ok) break;
        const int nv = min(WK, np - i * WK);
        mbar_expect_tx(full0 + 8 * st, (uint32_t)nv * bytes);
        __syncwarp();
        const int panel = boxes == 4 ? lane >> 2 : lane, box = boxes == 4 ? lane & 3 : 0;
        if (lane < nv * boxes)
          tma_load_2d_lane(smem_u32(smem + st * kStageB + offset) + (uint32_t)panel * pitch + (uint32_t)(box * XBLOCK),
                           weights ? &tmW : &tmX, full0 + 8 * st, (p0 + i * WK + panel) * kx + box * 64,
                           weights ? tile * R : 0);
      }
    __syncwarp();
    for (int f = max(0, n - kStages); f < n; ++f)
      wait_drain(full0 + 8 * (f % kStages), (uint32_t)(f / kStages) & 1u, p.wait, kErrCopy);
    __syncwarp();
  } else {
    const int wr = warp % WR, wk = warp / WR, t = lane & 3;
    const uint32_t stage0 = smem_u32(smem);
    const uint32_t wrow = stage0 + (uint32_t)(wk * R * 128) + (uint32_t)(wr * 16 + ((lane >> 3) & 1) * 8 + (lane & 7)) * 128;
    const uint32_t xpan = stage0 + kWeightsB + (uint32_t)wk * XPANEL;
    // a lane's row of A; past the last, the last once more (its columns of the
    // product are not used, and lanes that read one address share the read)
    // (swizzled, rows 0, 4, 1, 5, ... : two neighbours are in different banks)
    const int xr = min(XBLOCK ? (lane >> 3) + 4 * ((lane >> 2) & 1) : lane >> 2, p.M - 1);
    const uint32_t xrow = xpan + (uint32_t)(XBLOCK ? xr * 128 + (((t ^ xr) & 7) << 4) : xr * 512 + t * 16);
    const int row0 = wr * 16 + (lane >> 2), k0 = (p0 + wk) * 256 + 64 * t;
    ScaleCursor cursor = {};
    PanelScales next = {};
    if constexpr (W4) {
      cursor = scale_cursor(p.w, tile0 * R + row0, k0, WK * 256);
      load_panel_scales<TWO>(p.w, cursor, next);
    }
    int n = 0, buffer = 0;
    // (after a wait that gave up the barriers below are still met)
    bool ok = !p.wait.stall || warp_wait(stall, 0, abort_flag, p.wait, kErrMma);
    for (int tile = tile0; tile < tiles; tile += hop, buffer ^= 1) {
      float acc[MT][4];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][i] = 0.f;
      for (int i = 0; i < steps && ok; ++i, ++n) {
        const int st = n % kStages;
        PanelScales cur = next;
        if constexpr (W4) {
          if (i + 1 == steps) cursor = scale_cursor(p.w, (tile + hop) * R + row0, k0, WK * 256);
          load_panel_scales<TWO>(p.w, cursor, next);
        }
        ok = warp_wait(full0 + 8 * st, (uint32_t)(n / kStages) & 1u, abort_flag, p.wait, kErrMma);
        if (!ok) break;
        if (i * WK + wk < np) {
          const uint32_t off = after_wait((uint32_t)st * kStageB);
          if constexpr (W4) {
            const int panel = p0 + i * WK + wk;
            if (panel == p.panels - 1) scales_below_k<TWO>(cur, panel * 256 + 64 * t, p.w.K);
            if (p.w.z) panel_w4<F, MT, XBLOCK, TWO, true>(p, wrow + off, xrow + off, cur, acc);
            else panel_w4<F, MT, XBLOCK, TWO, false>(p, wrow + off, xrow + off, cur, acc);
          } else {
            panel_e4m3<MT>(wrow + off, xpan + off, acc);
          }
          before_release(acc);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(empty0 + 8 * st);
      }
      const int cs = R / ranks, part = rank * WK + wk;
      // to the owners: CTA r has the columns [r CS, (r + 1) CS) of the R, [part][m][CS]
      float *buf = parts + (ranks == 1 && WK > 1 ? buffer * (kPartsB / 8) : 0);
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int col = wr * 16 + (lane >> 2) + (i >> 1) * 8, row = m * 8 + (XBLOCK ? t + 4 * (i & 1) : 2 * t + (i & 1));
          if (row >= p.M) continue;
          if (WK == 1 && ranks == 1) {  // nothing is left to be added
            if (tile * R + col < p.N)
              store_value(p.out, p.tc, (int64_t)row * p.ldc + tile * R + col, acc[m][i] * Unpack<F>::kBack);
            continue;
          }
          const uint32_t at = smem_u32(buf + (part * p.M + row) * cs + col % cs);
          st_cluster_f32(map_to_rank(at, (uint32_t)(col / cs)), acc[m][i]);
        }
      if (ranks > 1) break;
      // Two buffers: one is written again only past the next tile's barrier,
      // which a warp meets when it has read this one.
      if constexpr (WK > 1) {
        computing_warps_sync();
        for (int o = threadIdx.x; o < p.M * R; o += 32 * kWarps) store_sum<F, WK>(p, buf, R, tile * R, o);
      }
    }
  }
  if (ranks > 1) {
    cluster_sync_all();
    const int cs = R / ranks;
    for (int o = threadIdx.x; o < p.M * cs; o += kThreads) store_sum<F, 0>(p, parts, cs, tile0 * R + rank * cs, o, ranks * WK);
  }
}

template <int F, int WR, bool TWO>
mm_status run(const TmaRows &rx, const TmaRows &rw, int K, GemvParams p, LaunchCtx &ctx) {
  constexpr int WK = kWarps / WR, R = 16 * WR;
  auto kern = gemv_quant_kernel<F, WR, TWO>;
  static PerDevice<int> set_up;
  int done;
  const cudaError_t err = set_up.get(ctx.dev->info.ordinal, &done, [&](int *) {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  });
  if (err != cudaSuccess) return cuda_error(err, "quantised GEMV set-up");
  CUtensorMap mw, mx;
  mm_status st = encode_map_2d(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, rw.p, (uint64_t)rw.bytes, (uint64_t)rw.rows,
                               (uint64_t)rw.ld, 128, R, CU_TENSOR_MAP_SWIZZLE_128B);
  if (st != MM_OK) return st;
  st = F == FMT_E4M3
           ? encode_map_2d(&mx, CU_TENSOR_MAP_DATA_TYPE_UINT8, rx.p, (uint64_t)K, (uint64_t)rx.rows,
                           (uint64_t)rx.ld, 128, (uint32_t)p.M, CU_TENSOR_MAP_SWIZZLE_128B)
           : encode_map_2d(&mx, F == FMT_W4_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                           rx.p, (uint64_t)K, (uint64_t)rx.rows, (uint64_t)rx.ld, kXBlock<F, WR> ? 64 : 256,
                           (uint32_t)p.M, kXBlock<F, WR> ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE);
  if (st != MM_OK) return st;
  p.panels = (int)((rw.bytes + 127) / 128);
  const int tiles = (p.N + R - 1) / R;
  // two CTAs an SM; each rank at least two steps of the ring
  int ranks = 1;
  while (ranks < 8 && (int64_t)tiles * ranks * 2 <= 2 * ctx.dev->info.sms && p.panels >= 2 * ranks * WK) ranks *= 2;
  p.panels_per_rank = ((p.panels + ranks - 1) / ranks + WK - 1) / WK * WK;
  const int columns = ranks > 1 ? tiles : std::min(tiles, 2 * ctx.dev->info.sms);
  cudaError_t e = launch_pdl(kern, dim3((unsigned)columns, (unsigned)ranks), dim3(kThreads), kSmem, ctx.stream,
                             dim3(1, (unsigned)ranks), mw, mx, p);
  if (e != cudaSuccess) return cuda_error(e, "quantised GEMV launch");
  count_operator_launch();
  return MM_OK;
}

template <int F, bool TWO>
mm_status run_rows(const TmaRows &rx, const TmaRows &rw, int K, const GemvParams &p, LaunchCtx &ctx) {
  if (p.M <= 2) return run<F, 1, TWO>(rx, rw, K, p, ctx);
  if (p.M <= 4) return run<F, 2, TWO>(rx, rw, K, p, ctx);
  if constexpr (F != FMT_E4M3)
    if (p.M > 8) return run<F, 8, TWO>(rx, rw, K, p, ctx);
  return run<F, 4, TWO>(rx, rw, K, p, ctx);
}

GemvParams gemv_params(void *out, int64_t ldc, int tc, int M, int N, LaunchCtx &ctx) {
  GemvParams p;
  std::memset(&p, 0, sizeof p);
  p.out = out;
  p.ldc = ldc;
  p.tc = tc;
  p.M = M;
  p.N = N;
  p.wait = operator_waits(ctx);
  return p;
}

}  // namespace

mm_status launch_gemv_w4(const W4Args &a, LaunchCtx &ctx) {
  TmaRows rx{a.A, a.lda * 2, a.M, (int64_t)a.K * 2}, rw{a.codes, a.ldw / 2, a.N, ((int64_t)a.K + 1) / 2};
  mm_status st = align_rows(rx, rw, ctx);
  if (st != MM_OK) return st;
  GemvParams p = gemv_params(a.out, a.ldc, a.tc, a.M, a.N, ctx);
  p.w = w4_scales(a);
  const bool two = a.group == 32;
  if (a.ta == MM_BF16)
    return two ? run_rows<FMT_W4_BF16, true>(rx, rw, a.K, p, ctx) : run_rows<FMT_W4_BF16, false>(rx, rw, a.K, p, ctx);
  return two ? run_rows<FMT_W4_F16, true>(rx, rw, a.K, p, ctx) : run_rows<FMT_W4_F16, false>(rx, rw, a.K, p, ctx);
}

mm_status launch_gemv_q8(const Q8Args &a, LaunchCtx &ctx) {
  TmaRows rx{a.A, a.lda, a.M, a.K}, rw{a.B, a.ldb, a.N, a.K};
  mm_status st = align_rows(rx, rw, ctx);
  if (st != MM_OK) return st;
  GemvParams p = gemv_params(a.out, a.ldc, a.tc, a.M, a.N, ctx);
  p.sa = a.scale_a;
  p.sb = a.scale_b;
  return run_rows<FMT_E4M3, false>(rx, rw, a.K, p, ctx);
}

}  // namespace mm
