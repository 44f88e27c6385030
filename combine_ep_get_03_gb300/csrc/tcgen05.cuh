// Inline PTX for the fifth-generation tensor cores: tensor-map loads, TMEM,
// MMA issue and completion, shared-memory and instruction descriptors.
#pragma once

#include <cuda.h>

#include "device_common.cuh"

namespace ep {

// ------------------------------------------------------------------ loads

__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
      :
      : "r"(smem_u32(dst)), "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
      :
      : "r"(smem_u32(dst)), "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, const void* src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];"
               :
               : "l"(map), "r"(x), "r"(y), "r"(smem_u32(src))
               : "memory");
}

// A 4-byte asynchronous copy, 0 instead where `on` is false (src is not read),
// and an arrival on `bar` (counted in its expected arrivals) when this
// thread's copies so far have landed.
__device__ __forceinline__ void copy_async4(uint32_t dst, const float* src, bool on) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" : : "r"(dst), "l"(src), "r"(on ? 4 : 0) : "memory");
}
__device__ __forceinline__ void copy_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" : : "r"(smem_u32(bar)) : "memory");
}

// A tensor map over bytes [planes][rows][width] (2-D where planes is 0), box
// 128 x box_rows, 128-byte swizzle.
cudaError_t make_byte_map(CUtensorMap* map, const void* base, int width, long long rows, int planes, int box_rows);
// The same over bf16 [rows][width], box 64 x box_rows.
cudaError_t make_bf16_map(CUtensorMap* map, const void* base, int width, long long rows, int box_rows);

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" : : "l"(map) : "memory");
}

// ------------------------------------------------------------------ pairs of blocks
//
// A cluster of two blocks on neighbouring SMs whose tensor cores work on one
// tile of twice the rows.  Block 0 issues; each block holds its rows of A, half
// of B and its rows of the accumulator.

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" : : : "memory");
}
// An arrival on block 0's barrier at the place of `bar`.  It says that this
// block's tensor core may read what fence_proxy_async_smem ordered before it, or
// may write TMEM that has been read; no thread of block 0 reads memory on its
// account.  (With release at cluster scope each arrival waits some 1000 cycles
// for all of the thread's writes.)
__device__ __forceinline__ void mbar_arrive_first(uint64_t* bar) {
  asm volatile(
      "{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %0, 0;\n"
      " mbarrier.arrive.shared::cluster.b64 _, [a];\n}\n"
      :
      : "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void pair_tmem_alloc(uint32_t* slot, uint32_t columns) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
               :
               : "r"(smem_u32(slot)), "r"(columns)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
}
__device__ __forceinline__ void pair_tmem_free(uint32_t addr, uint32_t columns) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" : : "r"(addr), "r"(columns));
}
__device__ __forceinline__ void pair_mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t desc, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n"
      :
      : "r"(d), "l"(a), "l"(b), "r"(desc), "r"(accumulate ? 1u : 0u)
      : "memory");
}
// An arrival on both blocks' barriers when every MMA that this thread issued
// has finished.
__device__ __forceinline__ void pair_mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
               :
               : "r"(smem_u32(bar)), "h"(static_cast<uint16_t>(3))
               : "memory");
}

// ------------------------------------------------------------------ TMEM

// One warp takes `columns` (a power of two >= 32) TMEM columns; their address
// lands in *slot (shared memory).
__device__ __forceinline__ void tmem_alloc(uint32_t* slot, uint32_t columns) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
               :
               : "r"(smem_u32(slot)), "r"(columns)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t columns) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" : : "r"(addr), "r"(columns));
}
__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" : : : "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" : : : "memory"); }

// 32 consecutive columns of the warp's 32 lanes: register j of lane l is
// element (lane base + l, column + j).
__device__ __forceinline__ void tmem_load32(uint32_t addr, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
        "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
        "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(addr)
      : "memory");
}
// Waits for this thread's loads; `v` are registers that one of them fills, so
// that nothing reads them before.
__device__ __forceinline__ void tmem_load_wait(uint32_t* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]),
                 "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]),
                 "+r"(v[23]), "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]),
                 "+r"(v[30]), "+r"(v[31])
               :
               : "memory");
}

// Moves a warpgroup's register limit (all four warps together).  The limits
// of a block's warpgroups may not add up to more than its launch allocated.
template <int N>
__device__ __forceinline__ void registers_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" : : "n"(N));
}
template <int N>
__device__ __forceinline__ void registers_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" : : "n"(N));
}

// ------------------------------------------------------------------ MMA

// Shared-memory operand descriptor, 128-byte swizzle, tiles at 1024-byte
// boundaries.  `lead` and `stride` are the leading and stride byte offsets.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead, uint32_t stride) {
  return static_cast<uint64_t>((addr & 0x3ffffu) >> 4) | (static_cast<uint64_t>((lead & 0x3ffffu) >> 4) << 16) |
         (static_cast<uint64_t>((stride & 0x3ffffu) >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// Instruction descriptor with fp32 accumulation; operand formats 0 (e4m3 for
// f8f6f4, f16 for f16); `mn_major` for operands whose rows are the long axis
// of the contraction.
__host__ __device__ constexpr uint32_t mma_desc(int M, int N, bool mn_major) {
  return (1u << 4) | (mn_major ? 3u << 15 : 0u) | (static_cast<uint32_t>(N / 8) << 17) |
         (static_cast<uint32_t>(M / 16) << 24);
}

__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t desc, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n"
      :
      : "r"(d), "l"(a), "l"(b), "r"(desc), "r"(accumulate ? 1u : 0u)
      : "memory");
}
// One lane of a converged warp, the same one every time.  Code that only this
// lane runs keeps its operands in uniform registers; behind a test of the lane
// number the same MMAs cost about three times the issue time.
__device__ __forceinline__ bool elect_one() {
  uint32_t yes;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(yes));
  return yes != 0;
}

// An arrival on `bar` when every MMA that this thread issued has finished.
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
               :
               : "r"(smem_u32(bar))
               : "memory");
}

}  // namespace ep
