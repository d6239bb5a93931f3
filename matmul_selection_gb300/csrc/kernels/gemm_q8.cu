// Product of e4m3 operands with row scales, on tcgen05 (kind::f8f6f4):
//   out[m, n] = scale_a[m] scale_b[n] sum_k A[m, k] B[n, k]
// The scales are factors of a whole row or column of the output, so they stay
// out of the sum: the tensor core adds e4m3 products in fp32 and the epilogue
// multiplies once.  Both operands are K-major; a stage of the ring holds 128
// bytes of K (four MMAs of 32), laid out by TMA with the 128-byte swizzle.
//
//   pair   many rows: 256 x 256 output tiles on pairs of SMs
//          (cta_group::2), each SM loading 128 rows of A and 128 of B a stage;
//          persistent, two accumulators in TMEM, so that a tile's epilogue
//          runs under the next tile's main loop.
//   swap   few rows: out^T = B A^T, 128 rows of B (the weights) on the MMA's
//          128-lane side and BN rows of A on the other, so that a short A is
//          not padded to 128 rows.  K is split over the CTAs of a cluster;
//          their fp32 tiles meet in distributed shared memory and are added
//          in rank order, which is one launch, no workspace and the same bits
//          every time.
// Measured: 8192^3 334-349 us under the power cap (279-288 in short runs, 3.9 PFLOP/s);
// 1000 x 4096 x 4096 17.5 us, 300 x 4096 x 4096 13.4, 32 x 19456 x 16384 49 us (6.5
// TB/s, HBM-bound), 127 x 4097 x 4100 10.3 (prologue, split and meeting).
// Every mbarrier wait is bounded (see tcgen05.cuh); a wait that gives up
// records a code in the operators' error word.
#include <algorithm>

#include "../operators.h"
#include "../q8_choice.h"
#include "tcgen05.cuh"
#include "tile_out.cuh"
#include "values.cuh"

namespace mm {

namespace {

using namespace tc;

constexpr int kThreads = 192;  // warp 0 copies, warp 1 issues MMAs, warps 2-5 store
constexpr uint32_t kRowB = 128;  // bytes of K a stage
constexpr int kErrCopy = 0x801, kErrMma = 0x802, kErrStore = 0x803, kErrDrain = 0x804;

struct Q8Params {
  void *out;
  int64_t ldc;
  const float *sa, *sb;
  int tc;
  int M, N;
  int num_kb;       // 128-byte blocks of K
  int tiles_m, tiles_n;
  int full_units;   // pair: units of whole tiles; those after are half tiles
  int total_units;
  int kb_per_rank;  // swap
  int vec;          // out's rows are 16-byte aligned (pair: and whole pieces of 16 bytes)
  Waits wait;
};

// Whether `ok` holds in all of the 128 threads of the storing warps (barrier 1).
__device__ __forceinline__ bool all_of_128(bool ok) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.and.aligned.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(all)
      : "r"((uint32_t)ok)
      : "memory");
  return all != 0;
}

// ---------------------------------------------------------------- pair
constexpr int kPairStages = 6;
constexpr uint32_t kPairStageB = 2 * 128 * kRowB;
constexpr uint32_t kPairBoxesB = 4 * 2 * kBoxB;      // two for each storing warp
constexpr size_t kPairSmem = kPairStages * kPairStageB + kPairBoxesB + 1024 /* column scales */ + 1024 + 256;
constexpr int kGroupRows = 8;  // row tiles walked together, so their A and B stay in L2

// Tile of a unit: row tile, first column, width (256, or 128 for the halves
// that the last, partly filled wave's tiles are cut into).
__device__ __forceinline__ void pair_unit(const Q8Params &p, int u, int &tm, int &n0, int &w) {
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

__global__ void __launch_bounds__(kThreads, 1)
    q8_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const __grid_constant__ CUtensorMap tmBh, const __grid_constant__ CUtensorMap tmC,
                   const Q8Params p) {
  pdl_launch_dependents();
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  uint8_t *boxes = smem + kPairStages * kPairStageB;
  float *col_scale = reinterpret_cast<float *>(boxes + kPairBoxesB);  // of the tile being stored
  uint64_t *bars = reinterpret_cast<uint64_t *>(boxes + kPairBoxesB + 1024);
  const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * kPairStages;
  const uint32_t tfull0 = empty0 + 8 * kPairStages, tempty0 = tfull0 + 16, drain = tempty0 + 16, stall = drain + 8;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 2 * kPairStages + 6);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t pos = cluster_ctarank();
  const bool leader = pos == 0;
  const int cid = (int)cluster_id_x(), ncl = (int)nclusters_x();

  if (threadIdx.x == 0) {
    for (int s = 0; s < kPairStages; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull0 + 8 * a, 1);
      mbar_init(tempty0 + 8 * a, 8);  // four storing warps of both CTAs
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
    if (p.vec) prefetch_tmap(&tmC);
    if (cid < p.total_units) {  // the first blocks of this CTA's operands into L2
      int tm, n0, w;
      pair_unit(p, cid, tm, n0, w);
      for (int kb = 0; kb < min(p.num_kb, kPairStages); ++kb) {
        tma_prefetch_2d(&tmA, kb * (int)kRowB, tm * 256 + (int)pos * 128);
        tma_prefetch_2d(&tmB, kb * (int)kRowB, n0 + (int)pos * (w / 2));
      }
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
      const uint32_t bytes = 2 * (128 + nh) * kRowB;  // of both CTAs
      for (int kb = 0; kb < p.num_kb; ++kb) {
        if (!warp_wait(empty0 + 8 * stage, phase ^ 1, abort_flag, p.wait, kErrCopy)) {
          ok = false;
          break;
        }
        const uint32_t sa = smem_u32(smem + stage * kPairStageB), sb = sa + 128 * kRowB;
        const uint32_t lfb = leader_full0 + 8 * stage;
        if (leader) mbar_expect_tx(full0 + 8 * stage, bytes);
        tma_load_2d_pair(sa, &tmA, lfb, kb * (int)kRowB, m0);
        tma_load_2d_pair(sb, w == 256 ? &tmB : &tmBh, lfb, kb * (int)kRowB, n0 + (int)pos * nh);
        if (++stage == kPairStages) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    if (leader)  // both CTAs' copies have landed
      for (int s = 0; s < kPairStages; ++s) {
        const int st = (stage + s) % kPairStages;
        wait_drain(full0 + 8 * st, st < stage ? phase : phase ^ 1, p.wait, kErrCopy);
      }
    __syncwarp();
  } else if (warp == 1) {
    if (leader) {
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      // (test hook: a wait that only its limit ends; in the other kernels likewise)
      bool ok = !p.wait.stall || warp_wait(stall, 0, abort_flag, p.wait, kErrMma);
      for (int u = cid; u < p.total_units && ok; u += ncl) {
        int tm, n0, w;
        pair_unit(p, u, tm, n0, w);
        const uint32_t idesc = instr_desc(0, 256, (uint32_t)w);
        if (!warp_wait(tempty0 + 8 * acc, acc_phase ^ 1, abort_flag, p.wait, kErrMma)) break;
        fence_after();
        const uint32_t d = tmem_base + (uint32_t)(acc * 256);
        for (int kb = 0; kb < p.num_kb; ++kb) {
          if (!warp_wait(full0 + 8 * stage, phase, abort_flag, p.wait, kErrMma)) {
            ok = false;
            break;
          }
          fence_after();
          const uint32_t sa = smem_u32(smem + stage * kPairStageB);
          const uint64_t ad = desc_at(sa), bd = desc_at(sa + 128 * kRowB);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_f8<2>(d, ad + 2 * kk, bd + 2 * kk, idesc, (kb > 0 || kk > 0) ? 1u : 0u);
          mma_commit_pair(empty0 + 8 * stage);
          if (++stage == kPairStages) {
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
      wait_drain(drain, 0, p.wait, kErrDrain);
    }
    __syncwarp();
  } else {
    const int q = warp & 3;  // the TMEM lanes this warp may read
    uint8_t *mine = boxes + (warp - 2) * 2 * kBoxB;
    const bool f32 = p.tc == MM_F32;
    const int step = f32 ? 32 : 64;  // columns a box
    int acc = 0, side = 0;
    uint32_t acc_phase = 0;
    for (int u = cid; u < p.total_units; u += ncl) {
      int tm, n0, w;
      pair_unit(p, u, tm, n0, w);
      // the four warps go on or give up together (and are all done with the last
      // tile's column scales)
      if (!all_of_128(warp_wait(tfull0 + 8 * acc, acc_phase, abort_flag, p.wait, kErrStore))) break;
      fence_after();
      const int row0 = tm * 256 + (int)pos * 128 + q * 32, row = row0 + lane;
      const float sa = p.sa && row < p.M ? p.sa[row] : 1.f;
      const uint32_t tbase = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * 256);
      // Rows through a swizzled box in shared memory and TMA, which clips what
      // is past M and N.  (Stored by the lanes, 64 bytes of a row each, a
      // product with K = 64 took 19.0 us at 1865 x 5056.)  Rows that TMA cannot
      // address are read back from the box and stored by the warp, a row at a
      // time: 330 us at 8000 x 16001 x 64.  (Stored by the lanes, a row each, 1298 us.)
      for (int i = (int)threadIdx.x - 64; i < 256; i += 128)
        col_scale[i] = p.sb && n0 + i < p.N ? p.sb[n0 + i] : 1.f;
      asm volatile("bar.sync 1, 128;" ::: "memory");
#pragma unroll 1
      for (int c = 0; c < w && n0 + c < p.N && row0 < p.M; c += step) {
        uint32_t r0[32], r1[32];
        tmem_ld_32cols(tbase + (uint32_t)c, r0);
        if (!f32) tmem_ld_32cols(tbase + (uint32_t)(c + 32), r1);
        tmem_ld_wait();
        if (lane == 0) tma_store_wait_read<1>();  // this box's previous store has read it
        __syncwarp();
        uint8_t *box = mine + side * kBoxB;
        const float4 *s4 = reinterpret_cast<const float4 *>(col_scale + c);
        auto put = [&](int j, uint32_t a, uint32_t b, uint32_t c2, uint32_t d) {  // 16-byte chunk j of the row
          *reinterpret_cast<uint4 *>(box + lane * 128 + ((j ^ (lane & 7)) << 4)) = make_uint4(a, b, c2, d);
        };
        if (f32) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float4 s = s4[j];
            put(j, __float_as_uint(__uint_as_float(r0[4 * j]) * sa * s.x),
                __float_as_uint(__uint_as_float(r0[4 * j + 1]) * sa * s.y),
                __float_as_uint(__uint_as_float(r0[4 * j + 2]) * sa * s.z),
                __float_as_uint(__uint_as_float(r0[4 * j + 3]) * sa * s.w));
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint32_t *r = j < 4 ? r0 + 8 * j : r1 + 8 * (j - 4);
            const float4 s = s4[2 * j], q4 = s4[2 * j + 1];
            put(j, pack2(p.tc, __uint_as_float(r[0]) * sa * s.x, __uint_as_float(r[1]) * sa * s.y),
                pack2(p.tc, __uint_as_float(r[2]) * sa * s.z, __uint_as_float(r[3]) * sa * s.w),
                pack2(p.tc, __uint_as_float(r[4]) * sa * q4.x, __uint_as_float(r[5]) * sa * q4.y),
                pack2(p.tc, __uint_as_float(r[6]) * sa * q4.z, __uint_as_float(r[7]) * sa * q4.w));
          }
        }
        if (p.vec) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) tma_store_2d(&tmC, smem_u32(box), n0 + c, row0);
        } else {
          __syncwarp();
          const int left = min(step, p.N - n0 - c), rows = min(32, p.M - row0);  // (the box holds 32)
          if (f32) store_box<4>(box, p.out, (int64_t)row0 * p.ldc + n0 + c, p.ldc, rows, left);
          else store_box<2>(box, p.out, (int64_t)row0 * p.ldc + n0 + c, p.ldc, rows, left);
        }
        side ^= 1;
      }
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(leader_tempty0 + 8 * acc);
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1;
      }
    }
    if (lane == 0) tma_store_wait_all();
    __syncwarp();
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
// Warps 0 and 3 copy B and A, warp 1 issues MMAs, warps 4-11 take the tile out
// of TMEM (two for each quarter of the lanes); all of them store it.
constexpr int kSwapThreads = 384, kSwapStore = 4;

template <int BN>
struct Swap {
  static constexpr uint32_t kStageB = (128 + BN) * kRowB;
  static constexpr int kStages = BN == 32 ? 9 : BN == 64 ? 7 : 5;
  static constexpr uint32_t kTileB = BN * 128 * 4;  // the fp32 tile, beside the ring: others write it early
  static constexpr size_t kSmem = kStages * kStageB + kTileB + 1024 + 256;
  static constexpr uint32_t kCols = BN;  // TMEM columns, a power of two of at least 32
};

template <int BN>
__global__ void __launch_bounds__(kSwapThreads, 1)
    q8_swap_kernel(const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmA,
                   const Q8Params p) {
  using S = Swap<BN>;
  pdl_launch_dependents();
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  float *tile = reinterpret_cast<float *>(smem + S::kStages * S::kStageB);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + S::kStages * S::kStageB + S::kTileB);
  const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * S::kStages;
  const uint32_t done = empty0 + 8 * S::kStages, stall = done + 8;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 2 * S::kStages + 2);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ranks = (int)gridDim.y, rank = (int)blockIdx.y;  // a cluster along y splits K
  const int n0 = (int)blockIdx.x * 128, m0 = (int)blockIdx.z * BN;
  const int kb0 = rank * p.kb_per_rank, nk = max(0, min(p.kb_per_rank, p.num_kb - kb0));

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(full0 + 8 * s, 2);  // both copying warps arm their bytes
      mbar_init(empty0 + 8 * s, 1);
    }
    mbar_init(done, 1);
    mbar_init(stall, 1);
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == 3 && lane == 0) prefetch_tmap(&tmA);
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmB);
    for (int i = 0; i < min(nk, 16); ++i) tma_prefetch_2d(&tmB, (kb0 + i) * (int)kRowB, n0);
  }
  if (warp == 1) tmem_alloc<1>(smem_u32(tmem_slot), S::kCols);
  fence_before();
  if (ranks > 1) cluster_sync_all();  // the others run: their memory may be written
  else __syncthreads();
  fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();

  if (warp == 0 || warp == 3) {
    const CUtensorMap *map = warp == 0 ? &tmB : &tmA;
    const uint32_t offset = warp == 0 ? 0u : 128 * kRowB, bytes = (warp == 0 ? 128 : BN) * kRowB;
    const int y = warp == 0 ? n0 : m0;
    int i = 0;
    for (; i < nk; ++i) {
      const int st = i % S::kStages;
      if (!warp_wait(empty0 + 8 * st, ((uint32_t)(i / S::kStages) & 1u) ^ 1u, abort_flag, p.wait, kErrCopy)) break;
      mbar_expect_tx(full0 + 8 * st, bytes);
      tma_load_2d(smem_u32(smem + st * S::kStageB + offset), map, full0 + 8 * st, (kb0 + i) * (int)kRowB, y);
    }
    for (int f = max(0, i - S::kStages); f < i; ++f)
      wait_drain(full0 + 8 * (f % S::kStages), (uint32_t)(f / S::kStages) & 1u, p.wait, kErrCopy);
    __syncwarp();
  } else if (warp == 1) {
    constexpr uint32_t idesc = instr_desc(0, 128, BN);
    const bool ok = !p.wait.stall || warp_wait(stall, 0, abort_flag, p.wait, kErrMma);
    for (int i = 0; i < nk && ok; ++i) {
      const int st = i % S::kStages;
      if (!warp_wait(full0 + 8 * st, (uint32_t)(i / S::kStages) & 1u, abort_flag, p.wait, kErrMma)) break;
      fence_after();
      const uint32_t sb = smem_u32(smem + st * S::kStageB);
      const uint64_t bd = desc_at(sb), ad = desc_at(sb + 128 * kRowB);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        mma_f8<1>(tmem, bd + 2 * kk, ad + 2 * kk, idesc, (i > 0 || kk > 0) ? 1u : 0u);
      mma_commit<1>(empty0 + 8 * st);
    }
    mma_commit<1>(done);
    wait_drain(done, 0, p.wait, kErrDrain);
    __syncwarp();
  }
  const int rows = min(BN, p.M - m0), per = BN / ranks;
  if (warp >= kSwapStore) {
    warp_wait(done, 0, abort_flag, p.wait, kErrStore);
    fence_after();
    const int q = warp & 3;
    push_tile(tmem + ((uint32_t)(q * 32) << 16), smem_u32(tile), rank, ranks, per, rows,
              ((warp - kSwapStore) >> 2) * 32, 64, q * 32 + lane, nk == 0);
    fence_before();
  }
  if (ranks > 1) cluster_sync_all();
  else __syncthreads();
  fence_after();
  if (warp == 1) tmem_dealloc<1>(tmem, S::kCols);
  auto store = [&](auto step) {
    constexpr int STEP = decltype(step)::value;
    const int n = n0 + (STEP == 1 ? 4 * lane : lane), left = p.N - n;
    float sb[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) sb[i] = p.sb && i * STEP < left ? p.sb[n + i * STEP] : 1.f;
    sum_tile<STEP == 1>(tile, rank, ranks, per, rows, warp, kSwapThreads / 32, [&](int m, float4 v) {
      const float sa = p.sa ? p.sa[m0 + m] : 1.f;
      store_four<STEP>(p.out, p.tc, (int64_t)(m0 + m) * p.ldc + n,
                       make_float4(v.x * sa * sb[0], v.y * sa * sb[1], v.z * sa * sb[2], v.w * sa * sb[3]), left);
    });
  };
  if (p.vec) store(std::integral_constant<int, 1>());
  else store(std::integral_constant<int, 32>());
}

// ---------------------------------------------------------------- host side
// A K-major map in boxes of 128 bytes of K x box_rows.
mm_status rows_map(CUtensorMap *map, const uint8_t *p, int rows, int K, int64_t ld, int box_rows) {
  if (rows == 1) ld = ((int64_t)K + 15) / 16 * 16;
  return encode_map_2d(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, p, (uint64_t)K, (uint64_t)rows, (uint64_t)ld,
                       kRowB, (uint32_t)box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

mm_status pair_capacity(int device, int *clusters) {
  static PerDevice<int> fits;
  const cudaError_t err = fits.get(device, clusters, [](int *n) -> cudaError_t {
    cudaError_t e = cudaFuncSetAttribute(q8_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kPairSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = 2;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(2);
    lc.blockDim = dim3(kThreads);
    lc.dynamicSmemBytes = kPairSmem;
    lc.attrs = &at;
    lc.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(n, q8_pair_kernel, &lc);
  });
  if (err != cudaSuccess) return cuda_error(err, "gemm_q8 set-up");
  if (*clusters < 1) return set_error(MM_ERR_UNSUPPORTED, "no pair of CTAs fits on this device");
  return MM_OK;
}

mm_status run_pair(const Q8Args &a, Q8Params p, int clusters, LaunchCtx &ctx) {
  CUtensorMap ma, mb, mbh, mc;
  mm_status st;
  if ((st = rows_map(&ma, a.A, a.M, a.K, a.lda, 128)) != MM_OK) return st;
  if ((st = rows_map(&mb, a.B, a.N, a.K, a.ldb, 128)) != MM_OK) return st;
  if ((st = rows_map(&mbh, a.B, a.N, a.K, a.ldb, 64)) != MM_OK) return st;
  mc = ma;
  // TMA clips a row's end to 16 bytes, not to an element (at N = 2046 of 16 bits
  // in rows of 2048 it wrote the two elements behind the row).
  const int es = dtype_bytes(p.tc);
  p.vec = p.vec && (int64_t)p.N * es % 16 == 0;
  if (p.vec) {
    st = encode_map_2d(&mc,
                       p.tc == MM_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                       : p.tc == MM_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                         : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                       p.out, (uint64_t)p.N, (uint64_t)p.M, (uint64_t)p.ldc * es, 128 / es, 32,
                       CU_TENSOR_MAP_SWIZZLE_128B);
    if (st != MM_OK) return st;
  }
  p.tiles_m = (a.M + 255) / 256;
  p.tiles_n = (a.N + 255) / 256;
  const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n;
  if (tiles >= (1LL << 30)) return set_error(MM_ERR_UNSUPPORTED, "too many tiles");
  // a last wave that fills at most half the pairs is cut into half tiles
  const int64_t rem = tiles % clusters;
  const bool halve = tiles > clusters && rem > 0 && 2 * rem <= clusters;
  p.full_units = (int)(halve ? tiles - rem : tiles);
  p.total_units = (int)(halve ? tiles + rem : tiles);
  const int grid = 2 * (int)std::min<int64_t>(p.total_units, clusters);
  cudaError_t e = launch_pdl(q8_pair_kernel, dim3((unsigned)grid), dim3(kThreads), kPairSmem, ctx.stream,
                             dim3(2), ma, mb, mbh, mc, p);
  return e == cudaSuccess ? MM_OK : cuda_error(e, "gemm_q8 launch (pair)");
}

template <int BN>
mm_status run_swap(const Q8Args &a, Q8Params p, int ranks, LaunchCtx &ctx) {
  static PerDevice<int> set_up;
  int done;
  const cudaError_t err = set_up.get(ctx.dev->info.ordinal, &done, [](int *) {
    return cudaFuncSetAttribute(q8_swap_kernel<BN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)Swap<BN>::kSmem);
  });
  if (err != cudaSuccess) return cuda_error(err, "gemm_q8 set-up");
  CUtensorMap ma, mb;
  mm_status st;
  if ((st = rows_map(&mb, a.B, a.N, a.K, a.ldb, 128)) != MM_OK) return st;
  if ((st = rows_map(&ma, a.A, a.M, a.K, a.lda, BN)) != MM_OK) return st;
  p.kb_per_rank = (p.num_kb + ranks - 1) / ranks;
  const int gx = (a.N + 127) / 128, gz = (a.M + BN - 1) / BN;  // at most kQ8SwapRowTiles
  cudaError_t e = launch_pdl(q8_swap_kernel<BN>, dim3((unsigned)gx, (unsigned)ranks, (unsigned)gz),
                             dim3(kSwapThreads), Swap<BN>::kSmem, ctx.stream, dim3(1, (unsigned)ranks), mb, ma, p);
  return e == cudaSuccess ? MM_OK : cuda_error(e, "gemm_q8 launch (swap)");
}

}  // namespace

mm_status launch_gemm_q8(const Q8Args &in, LaunchCtx &ctx) {
  Q8Args a = in;
  mm_status st;
  if (a.K == 0) return write_zeros(a.out, a.ldc, a.M, a.N, a.tc, ctx);
  int clusters = 0;
  if ((st = pair_capacity(ctx.dev->info.ordinal, &clusters)) != MM_OK) return st;
  const Q8Choice form = choose_q8(a.M, a.N, ((int64_t)a.K + kRowB - 1) / kRowB, ctx.dev->info.sms, clusters);
  if (form.form == Q8_GEMV) return launch_gemv_q8(a, ctx);
  TmaRows ra{a.A, a.lda, a.M, a.K}, rb{a.B, a.ldb, a.N, a.K};
  if ((st = align_rows(ra, rb, ctx)) != MM_OK) return st;
  a.A = static_cast<const uint8_t *>(ra.p);
  a.lda = ra.ld;
  a.B = static_cast<const uint8_t *>(rb.p);
  a.ldb = rb.ld;
  Q8Params p;
  std::memset(&p, 0, sizeof p);
  p.out = a.out;
  p.ldc = a.ldc;
  p.sa = a.scale_a;
  p.sb = a.scale_b;
  p.tc = a.tc;
  p.M = a.M;
  p.N = a.N;
  p.num_kb = (int)(((int64_t)a.K + kRowB - 1) / kRowB);
  p.vec = (uintptr_t)a.out % 16 == 0 && (a.ldc * dtype_bytes(a.tc)) % 16 == 0 && a.ldc < (1LL << 37);
  p.wait = operator_waits(ctx);
  st = form.form == Q8_PAIR ? run_pair(a, p, clusters, ctx)
       : form.bn == 32      ? run_swap<32>(a, p, form.ranks, ctx)
       : form.bn == 64      ? run_swap<64>(a, p, form.ranks, ctx)
                            : run_swap<128>(a, p, form.ranks, ctx);
  if (st != MM_OK) return st;
  count_operator_launch();
  return MM_OK;
}

}  // namespace mm
