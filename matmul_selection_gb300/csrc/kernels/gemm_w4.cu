// Product with weights held in 4 bits and group scales:
//   out[m, n] = sum_k A[m, k] s[n, k / group] (q[n, k] - z[n, k / group])
//
// For more than 16 rows of A (fewer: gemv_quant.cu), on tcgen05 (kind::f16), as
// out^T = W A^T: 128 rows of the weights are
// the MMA's A side, BN rows of A its other side.  The scales change along K, so
// the weights are made on the way in: sixteen warps turn codes into 16-bit
// weights (q - z is exact, its product with the scale is rounded once to A's
// type) and write them into TMEM, from where the MMA takes its A operand.
// Through shared memory the writes would have to be fenced to the async proxy
// stage by stage, which took longer than the MMA of the stage.  Codes and
// rows of A come by TMA through a ring each; a stage holds 64 of K.  With f16 A and
// scales of a wider type a small kernel ahead finds a power of two for each row of
// weights that keeps them in f16's range.  CTAs are
// persistent; where there are few tiles K is split over the CTAs of a cluster,
// whose fp32 tiles meet in distributed shared memory and are added in rank
// order.
// Measured (bf16, groups of 128): 4096^3 100 us (1.37 PFLOP/s), 1000 x 4096 x
// 4096 27.3, bound by the tensor cores and the ends of the waves; 128 x 19456 x
// 16384 68 us and 32 x 19456 x 16384 65 (2.5 TB/s), bound by the weight-making
// warps (58 % of the integer pipe, 61 % of the issue slots).
#include <algorithm>

#include "../operators.h"
#include "tcgen05.cuh"
#include "values.cuh"
#include "w4.cuh"

namespace mm {

namespace {

using namespace tc;

// ---------------------------------------------------------------- tiles
constexpr int kErrCopy = 0x901, kErrMma = 0x902, kErrStore = 0x903, kErrDrain = 0x904, kErrCodes = 0x905,
              kErrDequant = 0x906;

// Warp 0 copies A, warp 1 issues MMAs, warp 2 copies codes, warps 4-11 store
// (two for each quarter of the 128 lanes), warps 12-27 make weights: four
// groups of four, each on every fourth stage, so that a stage's chain (two
// waits, the codes, the arithmetic, the write to TMEM) may take four stages'
// time.
constexpr int kStoreWarp = 4, kStoreWarps = 8, kDequantWarp = 12;
constexpr int kGroups = 4, kGroupWarps = 4, kDequantWarps = kGroups * kGroupWarps;
constexpr int kTileThreads = 32 * (kDequantWarp + kDequantWarps);
constexpr uint32_t kCodeStageB = 128 * 128;  // 256 codes (four blocks of 64) of 128 rows

template <int BN>
struct Tile {
  // Blocks of 64 of K a stage: two, which halves what a stage costs the warps
  // that hand it on, but for 256 rows, where the MMA of one takes longer.
  static constexpr int kBlocks = BN == 256 ? 1 : 2;
  static constexpr uint32_t kPanelB = BN * 128, kStageB = kBlocks * kPanelB;
  static constexpr int kStages = BN >= 128 ? 5 : 6;
  static constexpr int kCodeStages = BN >= 128 ? 3 : 4;
  // the fp32 tile where K is split: beside the rings, or over them
  static constexpr bool kOver = BN >= 128;
  static constexpr uint32_t kTileB = kOver ? 0 : BN * 512;
  static constexpr size_t kSmem = kStages * kStageB + kCodeStages * kCodeStageB + kTileB + 1024 + 512;
  // TMEM: the accumulator, then the stages' weights, 32 columns a block
  static constexpr uint32_t kUsed = BN + 32 * kBlocks * kStages, kCols = kUsed <= 256 ? 256 : 512;
  static_assert(kUsed <= 512, "TMEM");
  static_assert(kStages >= kGroups && kStages <= 4 / kBlocks * (kCodeStages - 1) + 1, "see dequant_blocks");
  static_assert(!kOver || (size_t)BN * 512 <= kStages * kStageB, "the fp32 tile fits the ring");
};

struct TileParams {
  void *out;
  int64_t ldc;
  int tc;
  int M, N;
  int num_kb, kb_per_rank;  // blocks of 64 of K, multiples of 4
  int tiles_n, tiles;
  Waits wait;
  W4Scales w;
  int split_scale;  // the scales' type is not A's
  // f16 A and wider scales, else null: for each row of weights a power of two that
  // its scales are divided by and its column of the output is multiplied with
  const float *row_factor;
  bool vec;         // out's rows are 16-byte aligned
};

// The largest finite scale of a row of weights is brought to [2^11, 2^12): 15 times
// that is still an f16, and the two parts of a scale (see group_scale) keep f16's
// whole precision down to 2^-14 of it, one rounding's to 2^-25.  A warp a row; 2.5 us
// of a call (100 x 4096 x 4096 14.1, with f16 scales 11.0).
__global__ void __launch_bounds__(256) w4_row_factor_kernel(const W4Scales w, float *factor) {
  pdl_launch_dependents();
  pdl_wait();
  const int n = (int)blockIdx.x * 8 + (int)(threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (n >= w.N) return;
  uint32_t big = 0;
  for (int g = lane; g < w.groups; g += 32) {
    const uint32_t s = __float_as_uint(load_value(w.s, w.ts, (int64_t)n * w.lds + g)) & 0x7fffffffu;
    if (s < 0x7f800000u) big = max(big, s);
  }
  big = __reduce_max_sync(0xffffffffu, big);
  // 2^(e - 11) for big in [2^e, 2^(e + 1)), no smaller than 2^-126
  const int e = (int)(big >> 23) - 11;
  if (lane == 0) factor[n] = big == 0 ? 1.f : __uint_as_float((uint32_t)max(e, 1) << 23);
}

// The scale and zero point of 32 codes of a row.  A scale of another type than
// A's is taken as a sum of two of A's type, hi + lo, so that a weight is still
// rounded once (to within 2^-8 of a rounding).
template <int TA>
struct GroupScale {
  typename Pair16<TA>::T hi, lo, zero;
};
template <int TA>
__device__ __forceinline__ GroupScale<TA> group_scale(const TileParams &p, const RawScale &r, float per_factor) {
  using T = typename Pair16<TA>::T;
  GroupScale<TA> g;
  if (!p.split_scale) {
    g.hi = g.lo = bits_as<T>(r.s * 0x00010001u);
  } else {
    float s = raw_scale_value(p.w, r);
    if (TA == MM_F16) s *= per_factor;  // (exact)
    g.hi = Pair16<TA>::both(s);
    const float rest = s - __low2float(g.hi);
    g.lo = Pair16<TA>::both(isfinite(rest) ? rest : 0.f);
  }
  // the bias that the codes are read with, and the zero point
  g.zero = bits_as<T>((TA == MM_BF16 ? 0x43004300u : 0x64006400u) + (r.z & 15u) * 0x00010001u);
  return g;
}

// Eight codes of a word into eight weights in k order.  A code in the low
// mantissa bits of 128 (bf16) or 1024 (f16) is the number 128 + q or 1024 + q;
// the difference with 128 + z or 1024 + z is exact.  A byte of the word holds
// two neighbours: one permute of the word and the word shifted by a nibble
// puts both into the low nibbles of two halves.
template <int TA>
__device__ __forceinline__ void dequant8(uint32_t w, const GroupScale<TA> &g, bool split, uint32_t *out) {
  using T = typename Pair16<TA>::T;
  constexpr uint32_t kBias = TA == MM_BF16 ? 0x43004300u : 0x64006400u;
  const uint32_t w4 = w >> 4;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t pair = __byte_perm(w, w4, 0x0400 + 0x0101 * i);  // bytes i of w, of w4 (from 16 bits up)
    const T d = __hsub2(bits_as<T>((pair & 0x000f000fu) | kBias), g.zero);
    out[i] = as_bits(split ? __hfma2(d, g.hi, __hmul2(d, g.lo)) : __hmul2(d, g.hi));
  }
}

// The weight-making warps' side of the rings.
struct DequantRing {
  const uint8_t *codes;
  uint32_t cfull0, cempty0;  // the code stages' barriers
  uint32_t empty0, full0;    // a stage is free; its weights (and A's rows) are there
  uint32_t weights;          // TMEM address of stage 0's weights
  int group;                 // of this warp
  int stage;                 // of the group's next fill
  uint32_t phase = 0;
  uint32_t fills = 0;        // stages filled before this tile
};

// The weights past K of the stage that reaches past it, `left` of whose are below:
// zeros.  A code there is arbitrary, and the weight that it makes may be infinite,
// which A's zeros would make a NaN.  The stage has been written: what is 32 weights
// from `c` on is read back, masked and written again (rare, so out of the way).
template <int BLOCKS>
__device__ __noinline__ void clear_past_k(uint32_t dst, int left) {
  tmem_st_wait();
#pragma unroll 1
  for (int c = 0; c < BLOCKS * 64; c += 32) {
    if (c + 32 <= left) continue;
    uint32_t v[16];
    tmem_ld_16cols(dst + (uint32_t)(c / 2), v);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int n = left - (c + 2 * i);
      v[i] &= n >= 2 ? 0xffffffffu : n == 1 ? 0x0000ffffu : 0u;
    }
    tmem_st_16cols(dst + (uint32_t)(c / 2), v);
  }
}

// The weights of 128 rows from row n0, blocks [kb0, kb0 + nk) (whole stages of
// codes), into TMEM: each thread a row (its lane) of the stages whose place in
// the ring is its group's modulo 4.
// A parity wait tells only adjacent phases apart.  Operand ring: when a group
// waits for the consumption of fill f - STAGES, its previous fill f - 4 needed
// that of f - 4 - STAGES, which covers f - 2 STAGES as STAGES >= 4.  Codes: the
// wait for a stage of codes follows that consumption, and the fill STAGES back
// used the codes CSTAGES back, or later ones: those had landed.
template <int TA, typename S>
__device__ __forceinline__ bool dequant_blocks(const TileParams &p, DequantRing &r, int n0, int kb0, int nk,
                                               volatile int *abort_flag) {
  constexpr int B = S::kBlocks, PER = 4 / B;  // stages a stage of codes makes
  const int warp = (int)threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = (warp & 3) * 32 + lane;  // the TMEM lanes this warp may write
  const int j = (int)(((uint32_t)r.group - r.fills) % kGroups), part = j % PER;
  const uint32_t dst0 = r.weights + ((uint32_t)((warp & 3) * 32) << 16);
  const ScaleRow srow = scale_row(p.w, n0 + row);
  float per_factor = 1.f;
  if (TA == MM_F16 && p.row_factor && n0 + row < p.N) per_factor = 1.f / p.row_factor[n0 + row];
  const bool two = p.w.group_shift == 5;  // a block of 64 spans two groups
  const uint8_t *crow = r.codes + row * 128;
  const int ns = nk / B;
  RawScale next[B][2];
  auto load_scales = [&](int i) {
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const int k = (kb0 + i * B + b) * 64;
      next[b][0] = load_raw_scale(p.w, srow, k);
      next[b][1] = two ? load_raw_scale(p.w, srow, k + 32) : next[b][0];
    }
  };
  load_scales(j);
  uint32_t c = (r.fills + (uint32_t)j) / PER;  // the stage of codes, over all tiles
  for (int i = j; i < ns; i += kGroups, c += kGroups / PER) {
    RawScale cur[B][2];
#pragma unroll
    for (int b = 0; b < B; ++b) cur[b][0] = next[b][0], cur[b][1] = next[b][1];
    load_scales(i + kGroups);
    const int stage = r.stage;
    if (!warp_wait(r.empty0 + 8 * stage, r.phase ^ 1, abort_flag, p.wait, kErrDequant)) return false;
    if ((r.stage += kGroups) >= S::kStages) {
      r.stage -= S::kStages;
      r.phase ^= 1;
    }
    const uint32_t cs = c % S::kCodeStages;
    if (!warp_wait(r.cfull0 + 8 * cs, (c / S::kCodeStages) & 1u, abort_flag, p.wait, kErrDequant)) return false;
    uint4 q[2 * B];
#pragma unroll
    for (int h = 0; h < 2 * B; ++h)
      q[h] = *reinterpret_cast<const uint4 *>(crow + cs * kCodeStageB +
                                              ((uint32_t)((part * 2 * B + h) ^ (row & 7)) << 4));
    fence_after();
#pragma unroll
    for (int b = 0; b < B; ++b) {
      GroupScale<TA> g = group_scale<TA>(p, cur[b][0], per_factor);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h && two) g = group_scale<TA>(p, cur[b][1], per_factor);
        const uint4 w = q[2 * b + h];
        uint32_t v[16];
        if (p.split_scale) {
          dequant8<TA>(w.x, g, true, v);
          dequant8<TA>(w.y, g, true, v + 4);
          dequant8<TA>(w.z, g, true, v + 8);
          dequant8<TA>(w.w, g, true, v + 12);
        } else {
          dequant8<TA>(w.x, g, false, v);
          dequant8<TA>(w.y, g, false, v + 4);
          dequant8<TA>(w.z, g, false, v + 8);
          dequant8<TA>(w.w, g, false, v + 12);
        }
        tmem_st_16cols(dst0 + (uint32_t)((stage * B + b) * 32 + h * 16), v);
      }
    }
    const int left = p.w.K - (kb0 + i * B) * 64;
    if (left < B * 64) clear_past_k<B>(dst0 + (uint32_t)(stage * B * 32), left);
    tmem_st_wait();
    fence_before();
    __syncwarp();
    // The codes are given back only here, after their use: given back right
    // behind the loads, the next copy overwrote some before they were read
    // (wrong rows at K >= 2048).
    if (lane == 0) {
      mbar_arrive(r.full0 + 8 * stage);
      mbar_arrive(r.cempty0 + 8 * cs);
    }
  }
  r.fills += (uint32_t)ns;
  return true;
}

template <int TA, int BN>
__global__ void __launch_bounds__(kTileThreads, 1)
    w4_tile_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmA,
                   const TileParams p) {
  using S = Tile<BN>;
  constexpr int STAGES = S::kStages, CSTAGES = S::kCodeStages;
  pdl_launch_dependents();
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  uint8_t *codes = smem + STAGES * S::kStageB;
  float *tile = reinterpret_cast<float *>(S::kOver ? smem : codes + CSTAGES * kCodeStageB);
  uint64_t *bars = reinterpret_cast<uint64_t *>(codes + CSTAGES * kCodeStageB + S::kTileB);
  const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * STAGES;
  const uint32_t cfull0 = empty0 + 8 * STAGES, cempty0 = cfull0 + 8 * CSTAGES;
  const uint32_t tfull = cempty0 + 8 * CSTAGES, tempty = tfull + 8, drain = tempty + 8, stall = drain + 8;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 2 * STAGES + 2 * CSTAGES + 4);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ranks = (int)gridDim.x, rank = (int)blockIdx.x;  // a cluster along x splits K
  const int kb0 = rank * p.kb_per_rank, nk = max(0, min(p.kb_per_rank, p.num_kb - kb0));  // multiples of 4
  constexpr int B = S::kBlocks;
  const int first = (int)blockIdx.y, step = (int)gridDim.y;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full0 + 8 * s, 1 + kGroupWarps);  // A's arming; the weights' four warps
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int s = 0; s < CSTAGES; ++s) {
      mbar_init(cfull0 + 8 * s, 1);
      mbar_init(cempty0 + 8 * s, 4 / B * kGroupWarps);
    }
    mbar_init(tfull, 1);
    mbar_init(tempty, kStoreWarps);
    mbar_init(drain, 1);
    mbar_init(stall, 1);
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == 2 && lane == 0) {
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmW);
    for (int i = 0; i < min((nk + 3) / 4, 16); ++i)  // the first tile's codes into L2
      tma_prefetch_2d(&tmW, kb0 * 32 + i * 128, (first % p.tiles_n) * 128);
  }
  if (warp == 1) tmem_alloc<1>(smem_u32(tmem_slot), S::kCols);
  fence_before();
  if (ranks > 1) cluster_sync_all();  // the others run: their memory may be written
  else __syncthreads();
  fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();

  if (warp == 0) {
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int u = first; u < p.tiles && ok; u += step)
      for (int i = 0; i < nk; i += B) {
        if (!warp_wait(empty0 + 8 * stage, phase ^ 1, abort_flag, p.wait, kErrCopy)) {
          ok = false;
          break;
        }
        mbar_expect_tx(full0 + 8 * stage, S::kStageB);
#pragma unroll
        for (int b = 0; b < B; ++b)
          tma_load_2d(smem_u32(smem + stage * S::kStageB + b * S::kPanelB), &tmA, full0 + 8 * stage,
                      (kb0 + i + b) * 64, u / p.tiles_n * BN);
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1;
        }
      }
    for (int s = 0; s < STAGES; ++s) {
      const int st = (stage + s) % STAGES;
      wait_drain(full0 + 8 * st, st < stage ? phase : phase ^ 1, p.wait, kErrCopy);
    }
    __syncwarp();
  } else if (warp == 1) {
    constexpr uint32_t idesc = instr_desc(TA == MM_BF16 ? 1 : 0, 128, BN);
    int stage = 0;
    uint32_t phase = 0, tphase = 0;
    bool ok = !p.wait.stall || warp_wait(stall, 0, abort_flag, p.wait, kErrMma);
    for (int u = first; u < p.tiles && ok; u += step) {
      if (!warp_wait(tempty, tphase ^ 1, abort_flag, p.wait, kErrMma)) break;
      for (int i = 0; i < nk; i += B) {
        if (!warp_wait(full0 + 8 * stage, phase, abort_flag, p.wait, kErrMma)) {
          ok = false;
          break;
        }
        fence_after();
#pragma unroll
        for (int b = 0; b < B; ++b) {
          const uint64_t bd = desc_at(smem_u32(smem + stage * S::kStageB + b * S::kPanelB));
          const uint32_t w = tmem + BN + (uint32_t)((stage * B + b) * 32);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_ts(tmem, w + 8 * kk, bd + 2 * kk, idesc, (i > 0 || b > 0 || kk > 0) ? 1u : 0u);
        }
        mma_commit<1>(empty0 + 8 * stage);
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1;
        }
      }
      if (!ok) break;
      mma_commit<1>(tfull);
      tphase ^= 1;
    }
    mma_commit<1>(drain);
    wait_drain(drain, 0, p.wait, kErrDrain);
    __syncwarp();
  } else if (warp == 2) {
    int cs = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int u = first; u < p.tiles && ok; u += step)
      for (int i = 0; i < nk; i += 4) {
        if (!warp_wait(cempty0 + 8 * cs, phase ^ 1, abort_flag, p.wait, kErrCodes)) {
          ok = false;
          break;
        }
        mbar_expect_tx(cfull0 + 8 * cs, kCodeStageB);
        tma_load_2d(smem_u32(codes + cs * kCodeStageB), &tmW, cfull0 + 8 * cs, (kb0 + i) * 32,
                    u % p.tiles_n * 128);
        if (++cs == CSTAGES) {
          cs = 0;
          phase ^= 1;
        }
      }
    for (int s = 0; s < CSTAGES; ++s) {
      const int st = (cs + s) % CSTAGES;
      wait_drain(cfull0 + 8 * st, st < cs ? phase : phase ^ 1, p.wait, kErrCodes);
    }
    __syncwarp();
  } else if (warp >= kDequantWarp) {
    DequantRing r{codes, cfull0, cempty0, empty0, full0, tmem + BN};
    r.group = r.stage = (warp - kDequantWarp) / kGroupWarps;
    for (int u = first; u < p.tiles; u += step)
      if (!dequant_blocks<TA, S>(p, r, u % p.tiles_n * 128, kb0, nk, abort_flag)) break;
  }
  const int q = warp & 3, half = (warp - kStoreWarp) >> 2;
  const bool stores = warp >= kStoreWarp && warp < kStoreWarp + kStoreWarps;
  const uint32_t tbase = tmem + ((uint32_t)(q * 32) << 16);
  if (ranks == 1) {
    if (stores) {
      uint32_t tphase = 0;
      for (int u = first; u < p.tiles; u += step) {
        if (!warp_wait(tfull, tphase, abort_flag, p.wait, kErrStore)) break;
        tphase ^= 1;
        fence_after();
        const int m0 = u / p.tiles_n * BN, n = u % p.tiles_n * 128 + q * 32 + lane;
        const float factor = TA == MM_F16 && p.row_factor && n < p.N ? p.row_factor[n] : 1.f;
#pragma unroll 1
        for (int c = half * 32; c < BN && m0 + c < p.M; c += 64) {
          uint32_t r[32];
          tmem_ld_32cols(tbase + (uint32_t)c, r);
          tmem_ld_wait();
          if (n < p.N) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (m0 + c + i < p.M)
                store_value(p.out, p.tc, (int64_t)(m0 + c + i) * p.ldc + n,
                            TA == MM_F16 ? __uint_as_float(r[i]) * factor : __uint_as_float(r[i]));
          }
        }
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(tempty);
      }
    }
  } else {  // one tile a cluster
    const int m0 = first / p.tiles_n * BN, rows = min(BN, p.M - m0), per = BN / ranks;
    if (stores) {
      warp_wait(tfull, 0, abort_flag, p.wait, kErrStore);
      fence_after();
    }
    if (S::kOver) cluster_sync_all();  // every CTA's rings are idle
    if (stores)
      push_tile(tbase, smem_u32(tile), rank, ranks, per, rows, half * 32, 64, q * 32 + lane, nk == 0);
    cluster_sync_all();
    auto store = [&](auto step) {
      constexpr int STEP = decltype(step)::value;
      const int n = first % p.tiles_n * 128 + (STEP == 1 ? 4 * lane : lane);
      float f[4] = {1.f, 1.f, 1.f, 1.f};
      if (TA == MM_F16 && p.row_factor)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (n + i * STEP < p.N) f[i] = p.row_factor[n + i * STEP];
      sum_tile<STEP == 1>(tile, rank, ranks, per, rows, warp, kTileThreads / 32, [&](int m, float4 v) {
        if (TA == MM_F16) v = make_float4(v.x * f[0], v.y * f[1], v.z * f[2], v.w * f[3]);
        store_four<STEP>(p.out, p.tc, (int64_t)(m0 + m) * p.ldc + n, v, p.N - n);
      });
    };
    if (p.vec) store(std::integral_constant<int, 1>());
    else store(std::integral_constant<int, 32>());
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == 1) tmem_dealloc<1>(tmem, S::kCols);
}

template <int TA, int BN>
mm_status run_tiles(const W4Args &a, const TmaRows &ra, const TmaRows &rw, TileParams p, LaunchCtx &ctx) {
  static PerDevice<int> set_up;
  auto kern = w4_tile_kernel<TA, BN>;
  int done;
  const cudaError_t err = set_up.get(ctx.dev->info.ordinal, &done, [&](int *) {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Tile<BN>::kSmem);
  });
  if (err != cudaSuccess) return cuda_error(err, "gemm_w4 set-up");
  CUtensorMap mw, ma;
  mm_status st = encode_map_2d(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, rw.p, (uint64_t)rw.bytes, (uint64_t)rw.rows,
                               (uint64_t)rw.ld, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B);
  if (st != MM_OK) return st;
  st = encode_map_2d(&ma, TA == MM_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, ra.p,
                     (uint64_t)a.K, (uint64_t)ra.rows, (uint64_t)ra.ld, 64, BN, CU_TENSOR_MAP_SWIZZLE_128B);
  if (st != MM_OK) return st;
  p.tiles_n = (a.N + 127) / 128;
  const int64_t tiles = (int64_t)p.tiles_n * ((a.M + BN - 1) / BN);
  if (tiles >= (1LL << 31)) return set_error(MM_ERR_UNSUPPORTED, "too many tiles");
  p.tiles = (int)tiles;
  int ranks = 1;
  while (ranks < 8 && tiles * ranks * 2 <= ctx.dev->info.sms && p.num_kb >= 8 * ranks) ranks *= 2;
  p.kb_per_rank = (p.num_kb / 4 + ranks - 1) / ranks * 4;
  const int grid = ranks > 1 ? p.tiles : std::min(p.tiles, ctx.dev->info.sms);
  cudaError_t e = launch_pdl(kern, dim3((unsigned)ranks, (unsigned)grid), dim3(kTileThreads), Tile<BN>::kSmem,
                             ctx.stream, dim3((unsigned)ranks), mw, ma, p);
  return e == cudaSuccess ? MM_OK : cuda_error(e, "gemm_w4 launch (tiles)");
}

// The narrowest tile that holds A's rows: the codes are unpacked once, and the
// narrower the tile, the deeper its rings (19456 x 16384, 32 rows 65 us, 128 rows
// 68).
template <int TA>
mm_status launch_tiles(const W4Args &a, const TmaRows &ra, const TmaRows &rw, const TileParams &p, LaunchCtx &ctx) {
  return a.M <= 32    ? run_tiles<TA, 32>(a, ra, rw, p, ctx)
         : a.M <= 64  ? run_tiles<TA, 64>(a, ra, rw, p, ctx)
         : a.M <= 128 ? run_tiles<TA, 128>(a, ra, rw, p, ctx)
                      : run_tiles<TA, 256>(a, ra, rw, p, ctx);
}

}  // namespace

mm_status launch_gemm_w4(const W4Args &a, LaunchCtx &ctx) {
  if (a.K == 0) return write_zeros(a.out, a.ldc, a.M, a.N, a.tc, ctx);
  // Up to 16 rows the GEMV form, exact in the codes (16 x 19456 x 16384 55 us; the
  // narrowest tiles, of 32 rows, 65).
  if (a.M <= 16) return launch_gemv_w4(a, ctx);
  mm_status st;
  // (all scratch before the first launch: a call that is refused has launched nothing)
  void *factor = nullptr;
  if (a.ta == MM_F16 && a.ts != a.ta &&
      (st = get_scratch(ctx, SCRATCH_WORKSPACE, (size_t)a.N * sizeof(float), &factor)) != MM_OK)
    return st;
  TmaRows ra{a.A, a.lda * 2, a.M, (int64_t)a.K * 2}, rw{a.codes, a.ldw / 2, a.N, ((int64_t)a.K + 1) / 2};
  if ((st = align_rows(ra, rw, ctx)) != MM_OK) return st;
  TileParams p;
  std::memset(&p, 0, sizeof p);
  p.out = a.out;
  p.ldc = a.ldc;
  p.tc = a.tc;
  p.M = a.M;
  p.N = a.N;
  // blocks of 64 of K, up to whole stages of codes (what is past K multiplies zeros)
  p.num_kb = (int)(((int64_t)a.K + 255) / 256 * 4);
  p.wait = operator_waits(ctx);
  p.w = w4_scales(a);
  p.split_scale = a.ts != a.ta;
  if (factor) {
    cudaError_t e = launch_pdl(w4_row_factor_kernel, dim3((unsigned)((a.N + 7) / 8)), dim3(256), 0, ctx.stream, dim3(1),
                               p.w, static_cast<float *>(factor));
    if (e != cudaSuccess) return cuda_error(e, "gemm_w4 launch (row factors)");
    count_operator_launch();
    p.row_factor = static_cast<const float *>(factor);
  }
  p.vec = (uintptr_t)a.out % 16 == 0 && (a.ldc * dtype_bytes(a.tc)) % 16 == 0;
  st = a.ta == MM_BF16 ? launch_tiles<MM_BF16>(a, ra, rw, p, ctx) : launch_tiles<MM_F16>(a, ra, rw, p, ctx);
  if (st == MM_OK) count_operator_launch();
  return st;
}

}  // namespace mm
