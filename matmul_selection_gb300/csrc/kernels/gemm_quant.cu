// Products with quantised weights on tcgen05, both operands K-major:
//   e4m3   out[m, n] = scale_a[m] scale_b[n] sum_k A[m, k] B[n, k]
//          (kind::f8f6f4).  The scales are factors of a whole row or column of
//          the output, so they stay out of the sum: the tensor core adds e4m3
//          products in fp32 and the epilogue multiplies once.
//   4-bit  out[m, n] = sum_k A[m, k] s[n, k / group] (q[n, k] - z[n, k / group])
//          (kind::f16).  The scales change along K, so eight warps turn codes
//          into 16-bit weights on the way into the ring: q - z is exact, its
//          product with the scale is rounded once to A's type.  The codes come
//          by TMA through a ring of their own.
// A stage of the ring holds 128 bytes of K (four MMAs of 32 bytes), in the
// 128-byte swizzle.
//
//   pair   many rows: 256 x 256 output tiles on pairs of SMs
//          (cta_group::2), each SM bringing 128 rows of A and 128 of the
//          weights a stage; persistent, two accumulators in TMEM, so that a
//          tile's epilogue runs under the next tile's main loop.
//   swap   few rows: out^T = W A^T, 128 rows of the weights on the MMA's
//          128-lane side and BN rows of A on the other, so that a short A is
//          not padded to 128 rows.  K is split over the CTAs of a cluster;
//          their fp32 tiles are added through distributed shared memory in
//          rank order, which is one launch, no workspace and the same bits
//          every time.
// Every mbarrier wait is bounded (see tcgen05.cuh); a wait that gives up
// records a code in the operators' error word.
#include <algorithm>
#include <mutex>

#include "../operators.h"
#include "tcgen05.cuh"
#include "values.cuh"

namespace mm {

namespace {

using namespace tc;

// What the weights are held in, and A's type.
enum Format { FMT_E4M3, FMT_W4_BF16, FMT_W4_F16 };
__host__ __device__ constexpr bool is_w4(int f) { return f != FMT_E4M3; }

// Warp 0 copies operands, warp 1 issues MMAs, warps 2-5 store; for 4-bit
// weights warps 6-21 make them and warp 22 copies codes.  The weight-making
// warps work in four groups of four, each on every fourth stage of the ring: a
// stage's chain (a wait, the codes, the arithmetic, the fence to
// the async proxy, the arrival) is then four stages long before it holds the
// MMA up.
constexpr int kGroups = 4, kGroupWarps = 4, kDequantWarps = kGroups * kGroupWarps;
__host__ __device__ constexpr int threads_of(int f) { return is_w4(f) ? 32 * (6 + kDequantWarps + 1) : 192; }
constexpr uint32_t kRowB = 128;  // bytes of K a stage
constexpr int kErrCopy = 0x801, kErrMma = 0x802, kErrStore = 0x803, kErrDrain = 0x804, kErrCodes = 0x805,
              kErrDequant = 0x806;
// A stage of codes: 128 bytes (256 codes, four stages of the operand ring) of
// 128 rows.
constexpr uint32_t kCodeStageB = 128 * 128;
__host__ __device__ constexpr uint32_t code_ring(int f, int stages) { return is_w4(f) ? stages * kCodeStageB : 0; }

struct QuantParams {
  void *out;
  int64_t ldc;
  const float *sa, *sb;
  int tc;
  int M, N;
  int num_kb;       // 128-byte blocks of K
  int tiles_m, tiles_n;
  int full_units;   // pair: units of whole tiles; those after are half tiles
  int total_units;
  int kb_per_rank;  // swap; 4-bit weights: a multiple of 4
  int vec;          // out's rows are 16-byte aligned
  int *err;
  // 4-bit weights
  const void *scales;
  const uint8_t *zeros;
  int64_t lds;
  int ts, group_shift, groups;
  int split_scale;  // the scales' type is not A's
};

// ---------------------------------------------------------------- 4-bit weights
// fp32 to A's type, the same value in both halves.
template <int F>
__device__ __forceinline__ uint32_t both(float v) {
  if constexpr (F == FMT_W4_BF16) {
    const __nv_bfloat162 x = __float2bfloat162_rn(v);
    return *reinterpret_cast<const uint32_t *>(&x);
  } else {
    const __half2 x = __float2half2_rn(v);
    return *reinterpret_cast<const uint32_t *>(&x);
  }
}
template <int F>
__device__ __forceinline__ float first(uint32_t v) {
  if constexpr (F == FMT_W4_BF16) return __low2float(*reinterpret_cast<const __nv_bfloat162 *>(&v));
  return __low2float(*reinterpret_cast<const __half2 *>(&v));
}
template <int F>
struct Pair16 {
  using T = __nv_bfloat162;
};
template <>
struct Pair16<FMT_W4_F16> {
  using T = __half2;
};

// The scale and zero point of 32 codes of a row.
template <int F>
struct GroupScale {
  typename Pair16<F>::T hi, lo, zero;
};

// A scale and a zero point as they lie in memory (loaded a stage of codes
// ahead of their use).
struct RawScale {
  uint32_t s;
  uint32_t z;
};
__device__ __forceinline__ RawScale load_raw_scale(const QuantParams &p, int n, int k) {
  RawScale r{0u, 8u};
  const int g = k >> p.group_shift;
  if (n < p.N && g < p.groups) {
    const int64_t at = (int64_t)n * p.lds + g;
    r.s = p.ts == MM_F32 ? __ldg(static_cast<const uint32_t *>(p.scales) + at)
                         : (uint32_t)__ldg(static_cast<const uint16_t *>(p.scales) + at);
    if (p.zeros) r.z = __ldg(p.zeros + at);
  }
  return r;
}
// A scale of another type than A's is taken as a sum of two of A's type, hi +
// lo, so that a weight is still rounded once (to within 2^-8 of a rounding).
template <int F>
__device__ __forceinline__ GroupScale<F> group_scale(const QuantParams &p, const RawScale &r) {
  using T = typename Pair16<F>::T;
  const float s = p.ts == MM_F32    ? __uint_as_float(r.s)
                  : p.ts == MM_BF16 ? __uint_as_float(r.s << 16)
                                    : __half2float(__ushort_as_half((unsigned short)r.s));
  const uint32_t hi = both<F>(s), lo = p.split_scale ? both<F>(s - first<F>(hi)) : 0u;
  // 128 + z or 1024 + z: the bias that the codes are read with, and the zero point
  const uint32_t zero = (F == FMT_W4_BF16 ? 0x43004300u : 0x64006400u) + (r.z & 15u) * 0x00010001u;
  GroupScale<F> g;
  g.hi = *reinterpret_cast<const T *>(&hi);
  g.lo = *reinterpret_cast<const T *>(&lo);
  g.zero = *reinterpret_cast<const T *>(&zero);
  return g;
}

// Eight codes of a word into eight weights in k order.  A code in the low
// mantissa bits of 128 (bf16) or 1024 (f16) is the number 128 + q or 1024 + q;
// the difference with 128 + z or 1024 + z is exact.
template <int F>
__device__ __forceinline__ uint4 dequant8(uint32_t w, const GroupScale<F> &g, bool split) {
  using T = typename Pair16<F>::T;
  constexpr uint32_t kBias = F == FMT_W4_BF16 ? 0x43004300u : 0x64006400u;
  uint32_t v[4];  // (0, 4), (1, 5), (2, 6), (3, 7)
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t b = ((w >> (4 * i)) & 0x000f000fu) | kBias;
    const T d = __hsub2(*reinterpret_cast<const T *>(&b), g.zero);
    const T x = split ? __hfma2(d, g.hi, __hmul2(d, g.lo)) : __hmul2(d, g.hi);
    v[i] = *reinterpret_cast<const uint32_t *>(&x);
  }
  return make_uint4(__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410),
                    __byte_perm(v[0], v[1], 0x7632), __byte_perm(v[2], v[3], 0x7632));
}

// The weight-making warps' side of the two rings.
struct DequantRing {
  uint8_t *codes;
  uint32_t cfull0, cempty0;  // the code stages' barriers
  uint32_t empty0;           // the operand ring's
  int cs = 0;
  uint32_t cphase = 0;
  uint32_t fill = 0;  // stages of the operand ring filled before this tile
};

// 128 rows (from row n0 of the weights; `rows` of them are needed) of the
// blocks [kb0, kb0 + nk) into the operand ring: each thread a row of its
// group's blocks, those whose place in the ring is the group's modulo 4.
// `slot(stage)` is the address of the stage's 128-byte rows, `arrive(stage)`
// reports one warp.
// A parity wait tells only adjacent phases apart: when a group waits for the
// consumption of fill f - STAGES, its previous fill f - 4 needed that of
// f - 4 - STAGES, which covers f - 2 STAGES only when STAGES >= 4.
template <int F, int STAGES, int CSTAGES, typename Slot, typename Arrive>
__device__ __forceinline__ bool dequant_blocks(const QuantParams &p, DequantRing &r, int n0, int rows,
                                               int kb0, int nk, volatile int *abort_flag, Slot &&slot,
                                               Arrive &&arrive) {
  static_assert(STAGES >= kGroups, "the groups may not run more than a ring ahead");
  const int t = (int)threadIdx.x - 32 * 6, row = t & 127, lane = t & 31;
  const int j = (int)(((uint32_t)(t >> 7) - r.fill) % kGroups);  // the group's block of a stage of codes
  const int n = n0 + row;
  RawScale next[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) next[h] = load_raw_scale(p, n, (kb0 + j) * 64 + 32 * h);
  for (int i = j; i < nk + j; i += kGroups) {  // a stage of codes, of which this group takes block j
    RawScale cur[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      cur[h] = next[h];
      next[h] = load_raw_scale(p, n, (kb0 + i + kGroups) * 64 + 32 * h);
    }
    if (!warp_wait(r.cfull0 + 8 * r.cs, r.cphase, abort_flag, p.err, kErrDequant)) return false;
    const uint8_t *crow = r.codes + r.cs * kCodeStageB + row * 128;
    uint4 c[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) c[h] = *reinterpret_cast<const uint4 *>(crow + (((2 * j + h) ^ (row & 7)) << 4));
    const uint32_t cempty = r.cempty0 + 8 * r.cs;
    if (++r.cs == CSTAGES) {
      r.cs = 0;
      r.cphase ^= 1;
    }
    if (i >= nk) {  // the last stage of codes ends before this group's block
      __syncwarp();
      if (lane == 0) mbar_arrive(cempty);
      break;
    }
    const uint32_t f = r.fill + (uint32_t)i;
    const int stage = (int)(f % STAGES);
    if (!warp_wait(r.empty0 + 8 * stage, ((f / STAGES) & 1u) ^ 1u, abort_flag, p.err, kErrDequant)) return false;
    if (row < rows) {
      uint8_t *dst = slot(stage) + row * 128;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const GroupScale<F> g = group_scale<F>(p, cur[h]);
        const uint32_t w[4] = {c[h].x, c[h].y, c[h].z, c[h].w};
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<uint4 *>(dst + (((4 * h + q) ^ (row & 7)) << 4)) =
              p.split_scale ? dequant8<F>(w[q], g, true) : dequant8<F>(w[q], g, false);
      }
    }
    fence_proxy_async_smem();  // the MMA reads through the async proxy
    __syncwarp();
    // The codes are given back only here, after their use: given back right
    // behind the loads, the next copy overwrote some before they were read
    // (wrong rows at K >= 2048).
    if (lane == 0) {
      arrive(stage);
      mbar_arrive(cempty);
    }
  }
  r.fill += (uint32_t)nk;
  return true;
}

// The code-copying warp's side.
struct CodeRing {
  int cs = 0;
  uint32_t phase = 0;
};
template <int CSTAGES>
__device__ __forceinline__ bool copy_codes(const QuantParams &p, CodeRing &r, const CUtensorMap *map,
                                           uint8_t *codes, uint32_t cfull0, uint32_t cempty0, int n0, int kb0,
                                           int nk, volatile int *abort_flag) {
  for (int i = 0; i < nk; i += 4) {
    if (!warp_wait(cempty0 + 8 * r.cs, r.phase ^ 1, abort_flag, p.err, kErrCodes)) return false;
    mbar_expect_tx(cfull0 + 8 * r.cs, kCodeStageB);
    tma_load_2d(smem_u32(codes + r.cs * kCodeStageB), map, cfull0 + 8 * r.cs, (kb0 + i) * 32, n0);
    if (++r.cs == CSTAGES) {
      r.cs = 0;
      r.phase ^= 1;
    }
  }
  return true;
}
template <int CSTAGES>
__device__ __forceinline__ void drain_codes(const QuantParams &p, const CodeRing &r, uint32_t cfull0) {
  for (int s = 0; s < CSTAGES; ++s) {
    const int st = (r.cs + s) % CSTAGES;
    wait_drain(cfull0 + 8 * st, st < r.cs ? r.phase : r.phase ^ 1, p.err, kErrCodes);
  }
}

__device__ __forceinline__ uint32_t pack2(int tc, float lo, float hi) {
  if (tc == MM_BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
  }
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}

// ---------------------------------------------------------------- pair
constexpr uint32_t kPairStageB = 2 * 128 * kRowB;
constexpr int kPairCodeStages = 3;
__host__ __device__ constexpr int pair_stages(int f) { return is_w4(f) ? 5 : 6; }
__host__ __device__ constexpr size_t pair_smem(int f) { return pair_stages(f) * kPairStageB + code_ring(f, kPairCodeStages) + 1024 + 512; }
constexpr int kGroupRows = 8;  // row tiles walked together, so their A and B stay in L2

// Tile of a unit: row tile, first column, width (256, or 128 for the halves
// that the last, partly filled wave's tiles are cut into).
__device__ __forceinline__ void pair_unit(const QuantParams &p, int u, int &tm, int &n0, int &w) {
  int t = u, half = -1;
  if (u >= p.full_units) {
    t = p.full_units + ((u - p.full_units) >> 1);
    half = (u - p.full_units) & 1;
  }
  const int per = kGroupRows * p.tiles_n;
  const int g = t / per, rows = min(kGroupRows, p.tiles_m - g * kGroupRows);
  const int r = t - g * per;
  tm = g * kGroupRows + r % rows;
  n0 = (r / rows) * 256 + (half > 0 ? 128 : 0);
  w = half < 0 ? 256 : 128;
}

template <int F>
__global__ void __launch_bounds__(threads_of(F), 1)
    quant_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                      const __grid_constant__ CUtensorMap tmBh, const QuantParams p) {
  constexpr int STAGES = pair_stages(F), CSTAGES = kPairCodeStages;
  constexpr bool W4 = is_w4(F);
  pdl_launch_dependents();
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  uint8_t *codes = smem + STAGES * kPairStageB;
  uint64_t *bars = reinterpret_cast<uint64_t *>(codes + code_ring(F, CSTAGES));
  const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * STAGES;
  const uint32_t tfull0 = empty0 + 8 * STAGES, tempty0 = tfull0 + 16, drain = tempty0 + 16;
  const uint32_t cfull0 = drain + 8, cempty0 = cfull0 + 8 * CSTAGES;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 2 * STAGES + 5 + 2 * CSTAGES);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t pos = cluster_ctarank();
  const bool leader = pos == 0;
  const int cid = (int)cluster_id_x(), ncl = (int)nclusters_x();

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full0 + 8 * s, W4 ? 1 + 2 * kGroupWarps : 1);  // the arming; both CTAs' weights
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull0 + 8 * a, 1);
      mbar_init(tempty0 + 8 * a, 8);  // four storing warps of both CTAs
    }
    mbar_init(drain, 1);
    for (int s = 0; s < CSTAGES; ++s) {
      mbar_init(cfull0 + 8 * s, 1);
      mbar_init(cempty0 + 8 * s, kDequantWarps);
    }
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmB);
    if (!W4) prefetch_tmap(&tmBh);
    if (cid < p.total_units) {  // the first blocks of this CTA's operands into L2
      int tm, n0, w;
      pair_unit(p, cid, tm, n0, w);
      for (int kb = 0; kb < min(p.num_kb, STAGES); ++kb) {
        tma_prefetch_2d(&tmA, kb * (W4 ? 64 : 128), tm * 256 + (int)pos * 128);
        if (!W4) tma_prefetch_2d(&tmB, kb * 128, n0 + (int)pos * (w / 2));
      }
      if (W4)
        for (int c = 0; c < min((p.num_kb + 3) / 4, CSTAGES); ++c)
          tma_prefetch_2d(&tmB, c * 128, n0 + (int)pos * (w / 2));
    }
  }
  if (warp == 1) tmem_alloc<2>(smem_u32(tmem_slot), 512);
  fence_before();
  cluster_sync_all();
  fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const uint32_t leader_full0 = map_to_rank(full0, 0), leader_tempty0 = map_to_rank(tempty0, 0);
  pdl_wait();

  if (warp == 0) {
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int u = cid; u < p.total_units && ok; u += ncl) {
      int tm, n0, w;
      pair_unit(p, u, tm, n0, w);
      const int nh = w / 2, m0 = tm * 256 + (int)pos * 128;
      const uint32_t bytes = 2 * (128 + (W4 ? 0 : nh)) * kRowB;  // of both CTAs
      for (int kb = 0; kb < p.num_kb; ++kb) {
        if (!warp_wait(empty0 + 8 * stage, phase ^ 1, abort_flag, p.err, kErrCopy)) {
          ok = false;
          break;
        }
        const uint32_t sa = smem_u32(smem + stage * kPairStageB), sb = sa + 128 * kRowB;
        const uint32_t lfb = leader_full0 + 8 * stage;
        if (leader) mbar_expect_tx(full0 + 8 * stage, bytes);
        tma_load_2d_pair(sa, &tmA, lfb, kb * (W4 ? 64 : 128), m0);
        if constexpr (!W4)
          tma_load_2d_pair(sb, w == 256 ? &tmB : &tmBh, lfb, kb * 128, n0 + (int)pos * nh);
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    if (leader)  // both CTAs' copies have landed
      for (int s = 0; s < STAGES; ++s) {
        const int st = (stage + s) % STAGES;
        wait_drain(full0 + 8 * st, st < stage ? phase : phase ^ 1, p.err, kErrCopy);
      }
    __syncwarp();
  } else if (warp == 1) {
    if (leader) {
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int u = cid; u < p.total_units && ok; u += ncl) {
        int tm, n0, w;
        pair_unit(p, u, tm, n0, w);
        const uint32_t idesc = instr_desc(F == FMT_W4_BF16 ? 1 : 0, 256, (uint32_t)w);
        if (!warp_wait(tempty0 + 8 * acc, acc_phase ^ 1, abort_flag, p.err, kErrMma)) break;
        fence_after();
        const uint32_t d = tmem_base + (uint32_t)(acc * 256);
        for (int kb = 0; kb < p.num_kb; ++kb) {
          if (!warp_wait<W4>(full0 + 8 * stage, phase, abort_flag, p.err, kErrMma)) {
            ok = false;
            break;
          }
          fence_after();
          const uint32_t sa = smem_u32(smem + stage * kPairStageB);
          const uint64_t ad = desc_at(sa), bd = desc_at(sa + 128 * kRowB);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma<2, !W4>(d, ad + 2 * kk, bd + 2 * kk, idesc, (kb > 0 || kk > 0) ? 1u : 0u);
          mma_commit_pair(empty0 + 8 * stage);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
        mma_commit_pair(tfull0 + 8 * acc);
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1;
        }
      }
      mma_commit<2>(drain);
      wait_drain(drain, 0, p.err, kErrDrain);
    }
    __syncwarp();
  } else if (W4 && warp >= 6) {
    if constexpr (W4) {
      if (warp == 6 + kDequantWarps) {
        CodeRing r;
        for (int u = cid; u < p.total_units; u += ncl) {
          int tm, n0, w;
          pair_unit(p, u, tm, n0, w);
          if (!copy_codes<CSTAGES>(p, r, &tmB, codes, cfull0, cempty0, n0 + (int)pos * (w / 2), 0, p.num_kb, abort_flag))
            break;
        }
        drain_codes<CSTAGES>(p, r, cfull0);
        __syncwarp();
      } else {
        DequantRing r{codes, cfull0, cempty0, empty0};
        for (int u = cid; u < p.total_units; u += ncl) {
          int tm, n0, w;
          pair_unit(p, u, tm, n0, w);
          if (!dequant_blocks<F, STAGES, CSTAGES>(
                  p, r, n0 + (int)pos * (w / 2), w / 2, 0, p.num_kb, abort_flag,
                  [&](int st) { return smem + st * kPairStageB + 128 * kRowB; },
                  [&](int st) { mbar_arrive_cluster(leader_full0 + 8 * st); }))
            break;
        }
      }
    }
  } else {
    const int q = warp & 3;  // the TMEM lanes this warp may read
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int u = cid; u < p.total_units; u += ncl) {
      int tm, n0, w;
      pair_unit(p, u, tm, n0, w);
      if (!warp_wait(tfull0 + 8 * acc, acc_phase, abort_flag, p.err, kErrStore)) break;
      fence_after();
      const int row = tm * 256 + (int)pos * 128 + q * 32 + lane;
      const float sa = p.sa && row < p.M ? p.sa[row] : 1.f;
      const uint32_t tbase = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * 256);
#pragma unroll 1
      for (int c = 0; c < w && n0 + c < p.N; c += 32) {
        uint32_t r[32];
        tmem_ld_32cols(tbase + (uint32_t)c, r);
        tmem_ld_wait();
        if (row >= p.M) continue;
        const int col = n0 + c;
        const int64_t at = (int64_t)row * p.ldc + col;
        if (p.vec && col + 32 <= p.N) {
          float v[32];
#pragma unroll
          for (int i = 0; i < 32; ++i)
            v[i] = __uint_as_float(r[i]) * sa * (p.sb ? __ldg(p.sb + col + i) : 1.f);
          if (p.tc == MM_F32) {
            float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              dst[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          } else {
            uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.out) + at);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              dst[i] = make_uint4(pack2(p.tc, v[8 * i], v[8 * i + 1]), pack2(p.tc, v[8 * i + 2], v[8 * i + 3]),
                                  pack2(p.tc, v[8 * i + 4], v[8 * i + 5]), pack2(p.tc, v[8 * i + 6], v[8 * i + 7]));
          }
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (col + i < p.N)
              store_value(p.out, p.tc, at + i, __uint_as_float(r[i]) * sa * (p.sb ? __ldg(p.sb + col + i) : 1.f));
        }
      }
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(leader_tempty0 + 8 * acc);
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1;
      }
    }
  }
  fence_before();
  __syncthreads();
  if (*abort_flag) {  // the other CTA's copies into this one may still be landing
    const uint64_t t0 = global_ns();
    while (global_ns() - t0 < 100000ull) __nanosleep(1000);
  }
  cluster_sync_all();  // the leader's MMAs read both CTAs' memory
  fence_after();
  if (warp == 1) tmem_dealloc<2>(tmem_base, 512);
}

// ---------------------------------------------------------------- swap
template <int F, int BN>
struct Swap {
  static constexpr uint32_t kStageB = (128 + BN) * kRowB;
  static constexpr int kCodeStages = BN == 256 ? 2 : 3;
  static constexpr int kStages = is_w4(F) ? (BN <= 64 ? 6 : BN == 128 ? 5 : 4)
                                          : (BN == 32 ? 10 : BN == 64 ? 8 : BN == 128 ? 6 : 4);
  static constexpr size_t kTileB = (size_t)BN * 128 * 4;  // the fp32 tile, over the ring
  static constexpr size_t kSmem = kStages * kStageB + code_ring(F, kCodeStages) + 1024 + 512;
  static constexpr uint32_t kCols = BN;  // TMEM columns, a power of two of at least 32
  static_assert(kTileB <= kStages * kStageB, "the fp32 tile fits the ring");
};

template <int F, int BN>
__global__ void __launch_bounds__(threads_of(F), 1)
    quant_swap_kernel(const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmA,
                      const QuantParams p) {
  using S = Swap<F, BN>;
  constexpr bool W4 = is_w4(F);
  pdl_launch_dependents();
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  uint8_t *codes = smem + S::kStages * S::kStageB;
  uint64_t *bars = reinterpret_cast<uint64_t *>(codes + code_ring(F, S::kCodeStages));
  const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * S::kStages;
  const uint32_t done = empty0 + 8 * S::kStages;
  const uint32_t cfull0 = done + 8, cempty0 = cfull0 + 8 * S::kCodeStages;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 2 * S::kStages + 1 + 2 * S::kCodeStages);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ranks = (int)gridDim.x, rank = (int)blockIdx.x;  // a cluster along x splits K
  const int n0 = (int)blockIdx.y * 128, m0 = (int)blockIdx.z * BN;
  const int kb0 = rank * p.kb_per_rank, nk = max(0, min(p.kb_per_rank, p.num_kb - kb0));

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(full0 + 8 * s, W4 ? 1 + kGroupWarps : 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    mbar_init(done, 1);
    for (int s = 0; s < S::kCodeStages; ++s) {
      mbar_init(cfull0 + 8 * s, 1);
      mbar_init(cempty0 + 8 * s, kDequantWarps);
    }
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmB);
    for (int i = 0; i < min(W4 ? (nk + 3) / 4 : nk, 16); ++i)  // weights into L2
      tma_prefetch_2d(&tmB, kb0 * (W4 ? 32 : 128) + i * 128, n0);
  }
  if (warp == 1) tmem_alloc<1>(smem_u32(tmem_slot), S::kCols);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait();

  if (warp == 0) {
    int i = 0;
    for (; i < nk; ++i) {
      const int st = i % S::kStages;
      if (!warp_wait(empty0 + 8 * st, ((uint32_t)(i / S::kStages) & 1u) ^ 1u, abort_flag, p.err, kErrCopy)) break;
      const uint32_t sb = smem_u32(smem + st * S::kStageB);
      mbar_expect_tx(full0 + 8 * st, W4 ? BN * kRowB : S::kStageB);
      if constexpr (!W4) tma_load_2d(sb, &tmB, full0 + 8 * st, (kb0 + i) * 128, n0);
      tma_load_2d(sb + 128 * kRowB, &tmA, full0 + 8 * st, (kb0 + i) * (W4 ? 64 : 128), m0);
    }
    for (int f = max(0, i - S::kStages); f < i; ++f)
      wait_drain(full0 + 8 * (f % S::kStages), (uint32_t)(f / S::kStages) & 1u, p.err, kErrCopy);
    __syncwarp();
  } else if (warp == 1) {
    constexpr uint32_t idesc = instr_desc(F == FMT_W4_BF16 ? 1 : 0, 128, BN);
    for (int i = 0; i < nk; ++i) {
      const int st = i % S::kStages;
      if (!warp_wait(full0 + 8 * st, (uint32_t)(i / S::kStages) & 1u, abort_flag, p.err, kErrMma)) break;
      fence_after();
      const uint32_t sb = smem_u32(smem + st * S::kStageB);
      const uint64_t bd = desc_at(sb), ad = desc_at(sb + 128 * kRowB);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        mma<1, !W4>(tmem_base, bd + 2 * kk, ad + 2 * kk, idesc, (i > 0 || kk > 0) ? 1u : 0u);
      mma_commit<1>(empty0 + 8 * st);
    }
    mma_commit<1>(done);
    wait_drain(done, 0, p.err, kErrDrain);
    __syncwarp();
  } else if (W4 && warp >= 6) {
    if constexpr (W4) {
      if (warp == 6 + kDequantWarps) {
        CodeRing r;
        copy_codes<S::kCodeStages>(p, r, &tmB, codes, cfull0, cempty0, n0, kb0, nk, abort_flag);
        drain_codes<S::kCodeStages>(p, r, cfull0);
        __syncwarp();
      } else {
        DequantRing r{codes, cfull0, cempty0, empty0};
        dequant_blocks<F, S::kStages, S::kCodeStages>(
            p, r, n0, 128, kb0, nk, abort_flag, [&](int st) { return smem + st * S::kStageB; },
            [&](int st) { mbar_arrive(full0 + 8 * st); });
      }
    }
  }
  // When the MMAs are complete the ring is idle and the accumulator can be read.
  const bool stores = warp >= 2 && warp < 6;
  const int q = warp & 3;
  bool ok = true;
  if (stores) {
    ok = warp_wait(done, 0, abort_flag, p.err, kErrStore);
    fence_after();
  }
  const int cols = min(BN, p.M - m0);  // rows of A in the tile
  const int n = n0 + q * 32 + lane;
  const float sb = p.sb && n < p.N ? p.sb[n] : 1.f;
  const uint32_t tbase = tmem_base + ((uint32_t)(q * 32) << 16);
  if (ranks == 1) {
    if (stores && ok) {
#pragma unroll 1
      for (int c = 0; c < cols; c += 32) {
        uint32_t r[32];
        tmem_ld_32cols(tbase + (uint32_t)c, r);
        tmem_ld_wait();
        if (n < p.N) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (c + i < cols) {
              const int m = m0 + c + i;
              store_value(p.out, p.tc, (int64_t)m * p.ldc + n,
                          __uint_as_float(r[i]) * (p.sa ? __ldg(p.sa + m) : 1.f) * sb);
            }
        }
      }
    }
  } else {
    float *tile = reinterpret_cast<float *>(smem);  // [BN][128]
    if (stores) {
#pragma unroll 1
      for (int c = 0; c < cols; c += 32) {
        uint32_t r[32];
        tmem_ld_32cols(tbase + (uint32_t)c, r);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i) tile[(c + i) * 128 + q * 32 + lane] = nk > 0 ? __uint_as_float(r[i]) : 0.f;
      }
    }
    cluster_sync_all();
    // rank r adds the rows r, r + ranks, ... of the tile, over the ranks in order
    if (stores && n < p.N) {
      const uint32_t mine = smem_u32(tile + q * 32 + lane);
      for (int m = rank; m < cols; m += ranks) {
        float part[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k < ranks) part[k] = ld_cluster_f32(map_to_rank(mine + (uint32_t)m * 512u, (uint32_t)k));
        float v = part[0];
#pragma unroll
        for (int k = 1; k < 8; ++k)
          if (k < ranks) v += part[k];
        store_value(p.out, p.tc, (int64_t)(m0 + m) * p.ldc + n, v * (p.sa ? __ldg(p.sa + m0 + m) : 1.f) * sb);
      }
    }
    cluster_sync_all();  // no CTA leaves while another reads its tile
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == 1) tmem_dealloc<1>(tmem_base, S::kCols);
}

// ---------------------------------------------------------------- host side
// What a product's kernels read: 16-byte aligned rows of bytes.
struct Operands {
  const void *a, *b;          // A; the weights (e4m3, or codes)
  int64_t lda, ldb;           // bytes
  int M, N;
  int64_t a_bytes, b_bytes;   // of a row
};

// A K-major map of e4m3 or 16-bit rows in boxes of 128 bytes x box_rows (4-bit
// weights: of codes, as bytes).
template <int F, bool WEIGHTS>
mm_status rows_map(CUtensorMap *map, const Operands &o, int box_rows) {
  constexpr bool bytes = !is_w4(F) || WEIGHTS;
  const int64_t row = WEIGHTS ? o.b_bytes : o.a_bytes;
  const int rows = WEIGHTS ? o.N : o.M;
  const int64_t ld = rows == 1 ? (row + 15) / 16 * 16 : WEIGHTS ? o.ldb : o.lda;
  const CUtensorMapDataType type = bytes             ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : F == FMT_W4_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                      : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  return encode_map_2d(map, type, WEIGHTS ? o.b : o.a, (uint64_t)(bytes ? row : row / 2), (uint64_t)rows,
                       (uint64_t)ld, bytes ? 128 : 64, (uint32_t)box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int F>
mm_status pair_capacity(int *clusters) {
  static std::once_flag once;
  static cudaError_t err = cudaSuccess;
  static int n = 0;
  std::call_once(once, [] {
    err = cudaFuncSetAttribute(quant_pair_kernel<F>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)pair_smem(F));
    if (err != cudaSuccess) return;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = 2;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(2);
    lc.blockDim = dim3(threads_of(F));
    lc.dynamicSmemBytes = pair_smem(F);
    lc.attrs = &at;
    lc.numAttrs = 1;
    err = cudaOccupancyMaxActiveClusters(&n, quant_pair_kernel<F>, &lc);
  });
  if (err != cudaSuccess) return cuda_error(err, "quantised product set-up");
  if (n < 1) return set_error(MM_ERR_UNSUPPORTED, "no pair of CTAs fits on this device");
  *clusters = n;
  return MM_OK;
}

template <int F>
mm_status run_pair(const Operands &o, QuantParams p, LaunchCtx &ctx) {
  int clusters = 0;
  CUtensorMap ma, mb, mbh;
  mm_status st;
  if ((st = pair_capacity<F>(&clusters)) != MM_OK) return st;
  if ((st = rows_map<F, false>(&ma, o, 128)) != MM_OK) return st;
  if ((st = rows_map<F, true>(&mb, o, 128)) != MM_OK) return st;
  if ((st = rows_map<F, true>(&mbh, o, 64)) != MM_OK) return st;
  p.tiles_m = (p.M + 255) / 256;
  p.tiles_n = (p.N + 255) / 256;
  const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n;
  if (tiles >= (1LL << 30)) return set_error(MM_ERR_UNSUPPORTED, "too many tiles");
  // a last wave that fills at most half the pairs is cut into half tiles
  const int64_t rem = tiles % clusters;
  const bool halve = tiles > clusters && rem > 0 && 2 * rem <= clusters;
  p.full_units = (int)(halve ? tiles - rem : tiles);
  p.total_units = (int)(halve ? tiles + rem : tiles);
  const int grid = 2 * (int)std::min<int64_t>(p.total_units, clusters);
  cudaError_t e = launch_pdl(quant_pair_kernel<F>, dim3((unsigned)grid), dim3(threads_of(F)), pair_smem(F),
                             ctx.stream, dim3(2), ma, mb, mbh, p);
  return e == cudaSuccess ? MM_OK : cuda_error(e, "quantised product launch (pair)");
}

template <int F, int BN>
mm_status run_swap_bn(const Operands &o, QuantParams p, int ranks, LaunchCtx &ctx) {
  static std::once_flag once;
  static cudaError_t err = cudaSuccess;
  std::call_once(once, [] {
    err = cudaFuncSetAttribute(quant_swap_kernel<F, BN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)Swap<F, BN>::kSmem);
  });
  if (err != cudaSuccess) return cuda_error(err, "quantised product set-up");
  CUtensorMap ma, mb;
  mm_status st;
  if ((st = rows_map<F, true>(&mb, o, 128)) != MM_OK) return st;
  if ((st = rows_map<F, false>(&ma, o, BN)) != MM_OK) return st;
  p.kb_per_rank = (p.num_kb + ranks - 1) / ranks;
  if (is_w4(F)) p.kb_per_rank = (p.kb_per_rank + 3) / 4 * 4;  // whole stages of codes
  const int gy = (p.N + 127) / 128, gz = (p.M + BN - 1) / BN;
  if (gy > 65535 || gz > 65535) return set_error(MM_ERR_UNSUPPORTED, "too many tiles");
  cudaError_t e = launch_pdl(quant_swap_kernel<F, BN>, dim3((unsigned)ranks, (unsigned)gy, (unsigned)gz),
                             dim3(threads_of(F)), Swap<F, BN>::kSmem, ctx.stream, dim3((unsigned)ranks), mb, ma,
                             p);
  return e == cudaSuccess ? MM_OK : cuda_error(e, "quantised product launch (swap)");
}

template <int F>
mm_status run_product(const Operands &o, const QuantParams &p, LaunchCtx &ctx) {
  if (p.M > 256) return run_pair<F>(o, p, ctx);
  const int bn = p.M <= 32 ? 32 : p.M <= 64 ? 64 : p.M <= 128 ? 128 : 256;
  const int64_t tiles = ((int64_t)p.N + 127) / 128;
  int ranks = 1;
  while (ranks < 8 && tiles * ranks * 2 <= ctx.dev->info.sms && p.num_kb >= 4 * ranks) ranks *= 2;
  return bn == 32    ? run_swap_bn<F, 32>(o, p, ranks, ctx)
         : bn == 64  ? run_swap_bn<F, 64>(o, p, ranks, ctx)
         : bn == 128 ? run_swap_bn<F, 128>(o, p, ranks, ctx)
                     : run_swap_bn<F, 256>(o, p, ranks, ctx);
}

// Copies of the operands whose rows TMA cannot address (a base or a distance
// between rows that is not a multiple of 16 bytes), in the stream's scratch.
mm_status align_operands(Operands &o, LaunchCtx &ctx) {
  auto fine = [](const void *p, int64_t rows, int64_t ld) {
    return (uintptr_t)p % 16 == 0 && (rows == 1 || (ld % 16 == 0 && ld < (1LL << 40)));
  };
  const bool pack_a = !fine(o.a, o.M, o.lda), pack_b = !fine(o.b, o.N, o.ldb);
  if (!pack_a && !pack_b) return MM_OK;
  const int64_t la = (o.a_bytes + 15) / 16 * 16, lb = (o.b_bytes + 15) / 16 * 16;
  const size_t na = pack_a ? (size_t)la * o.M : 0, nb = pack_b ? (size_t)lb * o.N : 0;
  void *w = nullptr;
  mm_status st = get_scratch(*ctx.dev, ctx.stream, SCRATCH_REPACK, na + nb, &w);
  if (st != MM_OK) return st;
  if (pack_a) {
    if ((st = launch_pack_rows(o.a, o.lda, o.M, o.a_bytes, w, la, ctx)) != MM_OK) return st;
    o.a = w;
    o.lda = la;
  }
  if (pack_b) {
    uint8_t *dst = static_cast<uint8_t *>(w) + na;
    if ((st = launch_pack_rows(o.b, o.ldb, o.N, o.b_bytes, dst, lb, ctx)) != MM_OK) return st;
    o.b = dst;
    o.ldb = lb;
  }
  return MM_OK;
}

mm_status write_zeros(void *out, int64_t ldc, int M, int N, int tc, cudaStream_t s) {
  const size_t es = (size_t)dtype_bytes(tc);
  MM_CUDA_TRY(cudaMemset2DAsync(out, (size_t)ldc * es, 0, (size_t)N * es, (size_t)M, s));
  return MM_OK;
}

QuantParams params_of(void *out, int64_t ldc, int M, int N, int tc, LaunchCtx &ctx) {
  QuantParams p;
  std::memset(&p, 0, sizeof p);
  p.out = out;
  p.ldc = ldc;
  p.tc = tc;
  p.M = M;
  p.N = N;
  p.vec = (uintptr_t)out % 16 == 0 && (ldc * dtype_bytes(tc)) % 16 == 0;
  p.err = ctx.dev->d_err + kOperatorErrorWord;
  return p;
}

}  // namespace

mm_status launch_gemm_q8(const Q8Args &a, LaunchCtx &ctx) {
  if (a.K == 0) return write_zeros(a.out, a.ldc, a.M, a.N, a.tc, ctx.stream);
  Operands o{a.A, a.B, a.lda, a.ldb, a.M, a.N, a.K, a.K};
  mm_status st = align_operands(o, ctx);
  if (st != MM_OK) return st;
  QuantParams p = params_of(a.out, a.ldc, a.M, a.N, a.tc, ctx);
  p.sa = a.scale_a;
  p.sb = a.scale_b;
  p.num_kb = (int)(((int64_t)a.K + 127) / 128);
  if ((st = run_product<FMT_E4M3>(o, p, ctx)) != MM_OK) return st;
  count_operator_launch();
  return MM_OK;
}

mm_status launch_gemm_w4_tiles(const W4Args &a, LaunchCtx &ctx) {
  Operands o{a.A, a.codes, a.lda * 2, a.ldw / 2, a.M, a.N, (int64_t)a.K * 2, ((int64_t)a.K + 1) / 2};
  mm_status st = align_operands(o, ctx);
  if (st != MM_OK) return st;
  QuantParams p = params_of(a.out, a.ldc, a.M, a.N, a.tc, ctx);
  p.num_kb = (int)(((int64_t)a.K + 63) / 64);
  p.scales = a.scales;
  p.zeros = a.zeros;
  p.lds = a.lds;
  p.ts = a.ts;
  p.group_shift = a.group == 32 ? 5 : a.group == 64 ? 6 : 7;
  p.groups = (a.K + a.group - 1) / a.group;
  p.split_scale = a.ts != a.ta;
  st = a.ta == MM_BF16 ? run_product<FMT_W4_BF16>(o, p, ctx) : run_product<FMT_W4_F16>(o, p, ctx);
  if (st != MM_OK) return st;
  count_operator_launch();
  return MM_OK;
}

}  // namespace mm
