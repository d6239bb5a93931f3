// PTX wrappers for the operator kernels that run on tcgen05: mbarriers with
// bounded waits, TMA, TMEM, the MMA forms they issue.  (The GEMM family of
// tc_gemm.cu keeps its own, with the variants only it needs.)
//
// "Warp-collective" wrappers are executed by all 32 lanes, so that a role's
// loop state stays warp-uniform; elect.sync picks the lane that performs the
// operation.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include <cstdint>

#include "../operators.h"

namespace mm {
namespace tc {

constexpr uint64_t kDrainLimitNs = 20000000ull;   // waits for what is in flight after an abort

__device__ __forceinline__ uint32_t smem_u32(const void *p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}

// ---------------------------------------------------------------- mbarriers
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_init_fence() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}
// Warp-collective.
__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar), "r"(bytes)
      : "memory");
}
// By one thread.
__device__ __forceinline__ void mbar_expect_tx_one(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
               : "memory");
}
__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// The same, suspended for up to `ns` before it answers no: a waiting warp then
// takes few issue slots from the working ones.
__device__ __forceinline__ bool mbar_try_wait_for(uint32_t bar, uint32_t parity, uint32_t ns) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(ns)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ uint64_t global_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

// Wait for the phase of `parity`, by a whole warp.  Gives up (false, in every
// lane) when the CTA's abort flag is up, or after the limit (Waits): then it raises
// the flag and records `code` in the error word.
static __device__ __noinline__ bool warp_wait_slow(uint32_t bar, uint32_t parity, volatile int *abort_flag,
                                            int *err, uint64_t limit_ns, int code) {
  const uint64_t t0 = global_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 4; ++i)
      if (__all_sync(0xffffffffu, mbar_try_wait_for(bar, parity, 20000u))) return true;
    int stop = 0;
    if ((threadIdx.x & 31) == 0) {
      if (*abort_flag) {
        stop = 1;
      } else if (global_ns() - t0 > limit_ns) {
        *abort_flag = 1;
        atomicCAS(err, 0, code);
        stop = 1;
      }
    }
    if (__shfl_sync(0xffffffffu, stop, 0)) return false;
  }
}
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *abort_flag,
                                          const Waits &w, int code) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return warp_wait_slow(bar, parity, abort_flag, w.err, w.limit_ns, code);
}
// A bounded wait that ignores the abort flag, for copies and MMAs in flight.
static __device__ __noinline__ void wait_drain_slow(uint32_t bar, uint32_t parity, int *err, int code) {
  const uint64_t t0 = global_ns();
  while (!mbar_try_wait(bar, parity))
    if (global_ns() - t0 > kDrainLimitNs) {
      atomicCAS(err, 0, code);
      return;
    }
}
__device__ __forceinline__ void wait_drain(uint32_t bar, uint32_t parity, const Waits &w, int code) {
  if (!mbar_try_wait(bar, parity)) wait_drain_slow(bar, parity, w.err, code);
}

// Wait by one thread on its own; false after the limit (recorded).
__device__ __forceinline__ bool thread_wait(uint32_t bar, uint32_t parity, const Waits &w, int code) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_ns();
  while (!mbar_try_wait_for(bar, parity, 20000u))
    if (global_ns() - t0 > w.limit_ns) {
      atomicCAS(w.err, 0, code);
      return false;
    }
  return true;
}

// ---------------------------------------------------------------- clusters
__device__ __forceinline__ uint32_t cluster_ctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_id_x() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%clusterid.x;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t nclusters_x() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%nclusterid.x;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t map_to_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ void st_cluster_f32(uint32_t cluster_addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(cluster_addr), "f"(v) : "memory");
}

// ---------------------------------------------------------------- TMA
__device__ __forceinline__ void prefetch_tmap(const CUtensorMap *map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
// L2 prefetch of a box: nothing returns to the SM, so it may run before the
// grid dependency wait.
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap *map, int x, int y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y)
               : "memory");
}
// `bytes` (a multiple of 16) between 16-byte aligned addresses, by one thread.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}
// Warp-collective.
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap *map, uint32_t bar,
                                            int x, int y) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
      : "memory");
}
// The same by every active lane on its own.
__device__ __forceinline__ void tma_load_2d_lane(uint32_t dst, const CUtensorMap *map, uint32_t bar, int x,
                                                 int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
      : "memory");
}
// For a CTA pair: the bytes complete on the leader's barrier
// (a shared::cluster address).  Warp-collective.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap *map,
                                                 uint32_t leader_bar, int x, int y) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%3, %4}], [%2];\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(leader_bar), "r"(x), "r"(y)
      : "memory");
}

// Store of a box from shared memory by one thread, as a group of its own.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap *map, uint32_t src, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];\n\t"
      "cp.async.bulk.commit_group;" ::"l"(reinterpret_cast<uint64_t>(map)),
      "r"(src), "r"(x), "r"(y)
      : "memory");
}
// This thread's stores, all but the newest N, have read their boxes.
template <int N>
__device__ __forceinline__ void tma_store_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void tma_store_wait_all() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}
// This thread's writes to shared memory, visible to the async proxy.
__device__ __forceinline__ void fence_proxy_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// ---------------------------------------------------------------- TMEM and MMA
__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
template <int CG>  // CTAs of the group: 1, or 2 for a pair.  Whole warp.
__device__ __forceinline__ void tmem_alloc(uint32_t dst_smem, uint32_t ncols) {
  if constexpr (CG == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n\t"
                 "tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::"r"(dst_smem),
                 "r"(ncols)
                 : "memory");
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;\n\t"
                 "tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::"r"(dst_smem),
                 "r"(ncols)
                 : "memory");
  }
}
template <int CG>
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  if constexpr (CG == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
                 : "memory");
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
                 : "memory");
}
// D += A B^T of e4m3 operands in shared memory (kind::f8f6f4), 32 of K.  CG:
// CTAs of the group.  Warp-collective.
#define MM_MMA_ASM(CGS, KIND)                                                                     \
  asm volatile(                                                                                   \
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"          \
      "@e tcgen05.mma.cta_group::" CGS ".kind::" KIND " [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem), \
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)                                         \
      : "memory")
template <int CG>
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate) {
  if constexpr (CG == 1)
    MM_MMA_ASM("1", "f8f6f4");
  else
    MM_MMA_ASM("2", "f8f6f4");
}
#undef MM_MMA_ASM
// The same with A in TMEM (16-bit types, two of K a column), one CTA.
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Instruction descriptor: D fp32, A and B of one type (kind::f8f6f4: 0 e4m3;
// kind::f16: 0 f16, 1 bf16), both K-major, m x n.
__host__ __device__ constexpr uint32_t instr_desc(uint32_t type, uint32_t m, uint32_t n) {
  return (1u << 4) | (type << 7) | (type << 10) | ((n >> 3) << 17) | ((m >> 4) << 24);
}
// Arrive on `bar` (this CTA's) when the MMAs issued so far are complete.
// Warp-collective.
template <int CG>
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  if constexpr (CG == 1)
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
        : "memory");
}
// The same on the barriers at this offset in both CTAs of the pair.
__device__ __forceinline__ void mma_commit_pair(uint32_t bar) {
  const uint16_t mask = 3;
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;\n\t}" ::"r"(bar),
      "h"(mask)
      : "memory");
}
// 32 lanes x 32 consecutive columns: thread i gets lane i's 32 columns.
__device__ __forceinline__ void tmem_ld_32cols(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_wait() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// ---------------------------------------------------------------- tiles out of TMEM
// A swapped product's fp32 tile (lane = column n of the output, TMEM column =
// row m) on its way out, where K may be split over the RANKS CTAs of a
// cluster.  Row m belongs to CTA m % RANKS: each storing warp writes its 32
// lanes' values of a row to the owner's shared memory, [rank][m / RANKS][128]
// floats, which costs the sender no wait; after a barrier each owner adds its
// rows' parts in rank order from its own memory, a warp a row, four columns a
// lane, so the stores to global memory are whole rows of 128.  (The owners
// reading the other CTAs' tiles instead, a column at a time, cost 13 us at
// 128 rows; 9 us read 16 bytes a lane.)
// Columns [c0, c0 + step, ...) of 32 of `rows`, by one warp; `tile` is the
// address in this CTA, `lane_col` the lane's column n.
template <int RANKS>
__device__ __forceinline__ void push_tile(uint32_t tmem_addr, uint32_t tile, int rank, int per, int rows,
                                          int c0, int step, int lane_col, bool empty) {
  uint32_t owner[RANKS];
#pragma unroll
  for (int k = 0; k < RANKS; ++k)
    owner[k] = map_to_rank(tile + (uint32_t)(rank * per * 128 + lane_col) * 4u, (uint32_t)k);
#pragma unroll 1
  for (int c = c0; c < rows; c += step) {
    uint32_t r[32];
    tmem_ld_32cols(tmem_addr + (uint32_t)c, r);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (c + i < rows)
        st_cluster_f32(owner[i % RANKS] + (uint32_t)((c + i) / RANKS) * 512u, empty ? 0.f : __uint_as_float(r[i]));
  }
}
__device__ __forceinline__ void push_tile(uint32_t tmem_addr, uint32_t tile, int rank, int ranks, int per,
                                          int rows, int c0, int step, int lane_col, bool empty) {
  switch (ranks) {
  case 1: return push_tile<1>(tmem_addr, tile, rank, per, rows, c0, step, lane_col, empty);
  case 2: return push_tile<2>(tmem_addr, tile, rank, per, rows, c0, step, lane_col, empty);
  case 4: return push_tile<4>(tmem_addr, tile, rank, per, rows, c0, step, lane_col, empty);
  default: return push_tile<8>(tmem_addr, tile, rank, per, rows, c0, step, lane_col, empty);
  }
}
// The owner's side: its rows to out(m, v), a warp a row.  A lane has the
// columns 4 lane .. 4 lane + 3 (VEC, for rows that take 16-byte aligned
// stores), else lane, lane + 32, lane + 64 and lane + 96.
template <bool VEC, typename Out>
__device__ __forceinline__ void sum_tile(const float *tile, int rank, int ranks, int per, int rows, int warp,
                                         int warps, Out &&out) {
  const int lane = threadIdx.x & 31;
  for (int s = warp; s * ranks + rank < rows; s += warps) {
    float4 v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < ranks) {
        const float *part = tile + (k * per + s) * 128;
        v[k] = VEC ? reinterpret_cast<const float4 *>(part)[lane]
                   : make_float4(part[lane], part[lane + 32], part[lane + 64], part[lane + 96]);
      }
#pragma unroll
    for (int k = 1; k < 8; ++k)
      if (k < ranks) v[0].x += v[k].x, v[0].y += v[k].y, v[0].z += v[k].z, v[0].w += v[k].w;
    out(s * ranks + rank, v[0]);
  }
}

// 16 consecutive columns of 32 lanes: thread i writes lane i's.
__device__ __forceinline__ void tmem_st_16cols(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// The same read.
__device__ __forceinline__ void tmem_ld_16cols(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// ---------------------------------------------------------------- host side
// Shared-memory descriptor bits (without the address) of a K-major operand in
// 128-byte rows with the 128-byte swizzle: 8-row groups 1024 bytes apart.
constexpr uint64_t kDescKMajor128 = ((uint64_t)(16 >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
                                    ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
__device__ __forceinline__ uint64_t desc_at(uint32_t smem_addr) {
  return kDescKMajor128 | (uint64_t)((smem_addr >> 4) & 0x3FFFu);
}

// A 2-D tiled map: `inner` elements a row, `outer` rows ld_bytes apart, boxes
// of box_inner x box_outer.
inline mm_status encode_map_2d(CUtensorMap *map, CUtensorMapDataType type, const void *base,
                               uint64_t inner, uint64_t outer, uint64_t ld_bytes,
                               uint32_t box_inner, uint32_t box_outer, CUtensorMapSwizzle swizzle) {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  if (!fn) return set_error(MM_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");
  cuuint64_t dims[2] = {inner, outer};
  cuuint64_t strides[1] = {ld_bytes};
  cuuint32_t box[2] = {box_inner, box_outer};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = fn(map, type, 2, const_cast<void *>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return set_error(MM_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  return MM_OK;
}

}  // namespace tc
}  // namespace mm
