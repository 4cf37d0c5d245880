// sda_pipe.cuh -- bounded mbarrier waits and tensor-map encoding shared by the
// paged-cache kernels (chunk attention and attention mass).
#pragma once

#include <cuda.h>

#include "sda_internal.cuh"
#include "umma_ptx.cuh"

namespace sda {

#ifdef __CUDACC__
// How long a try of a wait may sleep: warps that poll more often slow the others
// down (attention of a 2048-token chunk over 8192 positions: 1.43 ms without the
// hint, 1.37 with it).
constexpr uint32_t kWaitHintNs = 10000000;

// Where a bounded wait reports a timeout, and after how long.
struct PipeWait {
  volatile int* abort_flag;  // shared: set once any role of the CTA gave up
  int* error;                // global error word (1 = a wait timed out)
  uint64_t timeout_ns;
};

// try_wait that may sleep for up to `ns` before it answers.
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

// Bounded wait.  Returns false (and raises the abort flags) on timeout; once
// any role has aborted, every later wait returns false at once, so all roles
// run to the end of their loops quickly and the CTA exits.
__device__ __forceinline__ bool pipe_wait(uint32_t bar, uint32_t parity, const PipeWait& w) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  if (*w.abort_flag) return false;
  const uint64_t t0 = ptx::globaltimer_ns();
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait_for(bar, parity, kWaitHintNs)) return true;
    if ((it & 15u) == 0) {
      if (*w.abort_flag) return false;
      if (ptx::globaltimer_ns() - t0 > w.timeout_ns) {
        *w.abort_flag = 1;
        atomicExch(w.error, 1);
        return false;
      }
    }
  }
}

// pipe_wait for a converged warp.  All lanes poll: a lane polling alone for its
// warp was slower (a prompt chunk of attention 1.34 to 1.75 ms).
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const PipeWait& w) {
  return __all_sync(0xffffffffu, pipe_wait(bar, parity, w));
}

// Wait used only while draining copies / MMAs this CTA started: bounded by
// the timeout, but not cut short by the abort flag.
__device__ __forceinline__ void pipe_drain(uint32_t bar, uint32_t parity, const PipeWait& w) {
  const uint64_t t0 = ptx::globaltimer_ns();
  while (!ptx::mbar_try_wait(bar, parity)) {
    if (ptx::globaltimer_ns() - t0 > w.timeout_ns) {
      atomicExch(w.error, 1);
      return;
    }
  }
}

// True in one lane of the (converged) warp.  Code that issues MMAs keeps its
// control flow warp-uniform and guards only the instruction with this, so that
// descriptors stay in uniform registers: 33 cycles per M64 N64 K16 MMA, the
// shared-memory bound, against 47 from inside an `if (lane == 0)`.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// 4-D tiled load of one box into shared memory, completing on `bar`.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* tmap, int x, int y, int z, int w,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}

// Arrive on `bar` once this thread's earlier cp.async have landed (counted in
// the barrier's arrivals).
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile(
      "barrier.cluster.arrive.release.aligned;\n\t"
      "barrier.cluster.wait.acquire.aligned;" ::
          : "memory");
}

// Pairs of CTAs (cta_group::2).
// Both CTAs' warps together.
__device__ __forceinline__ void tmem_alloc_pair(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem),
               "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// Arrive on `bar` of both CTAs once this thread's earlier pair MMAs are done.
__device__ __forceinline__ void commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}
__device__ __forceinline__ uint32_t map_cta(uint32_t addr, uint32_t cta) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(cta));
  return r;
}
// (A release at cluster scope costs its thread about 1000 cycles, an acquire in a wait
// about 400.  What goes to the other CTA on every tile is an arrival alone, after reads
// of TMEM or after stores to the CTA's own shared memory that the MMAs read; stores to
// the other CTA are rare and have a fence_cluster() of their own on both sides.)
__device__ __forceinline__ void arrive_cluster(uint32_t mapped) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(mapped) : "memory");
}
__device__ __forceinline__ void store_cluster(uint32_t mapped, uint32_t v) {
  asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(mapped), "r"(v) : "memory");
}
// Stores to the other CTA's shared memory, and counts the 4 bytes on its barrier.
__device__ __forceinline__ void store_async(uint32_t mapped, uint32_t v, uint32_t mapped_bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(mapped),
               "r"(v), "r"(mapped_bar)
               : "memory");
}
__device__ __forceinline__ void fence_cluster() { asm volatile("fence.acq_rel.cluster;" ::: "memory"); }
// Tiled loads into this CTA that complete on a barrier of the pair's CTA 0.
__device__ __forceinline__ void tma_pair_4d(uint32_t dst, const void* tmap, int x, int y, int z, int w,
                                            uint32_t bar0) {
  asm volatile(
      "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar0)
      : "memory");
}
__device__ __forceinline__ void tma_pair_2d(uint32_t dst, const void* tmap, int x, int y, uint32_t bar0) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(bar0)
      : "memory");
}

// 16 lanes x 8 columns of TMEM (16x256b, one repetition).
__device__ __forceinline__ void tmem_ld_16x256b_x1(uint32_t taddr, uint32_t (&r)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(taddr));
}
// Two 8x8 b16 matrices, and one, stored as they are held.
__device__ __forceinline__ void stmatrix_x2(uint32_t addr, uint32_t r0, uint32_t r1) {
  asm volatile("stmatrix.sync.aligned.m8n8.x2.shared.b16 [%0], {%1, %2};" ::"r"(addr), "r"(r0),
               "r"(r1)
               : "memory");
}
__device__ __forceinline__ void stmatrix_x1(uint32_t addr, uint32_t r0) {
  asm volatile("stmatrix.sync.aligned.m8n8.x1.shared.b16 [%0], {%1};" ::"r"(addr), "r"(r0)
               : "memory");
}
#endif

// launch_pdl with clusters of `cluster` CTAs.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl_cluster(void (*kernel)(KArgs...), dim3 grid, dim3 block, unsigned cluster,
                               size_t smem, cudaStream_t st, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// A 2-D bf16 tensor map over [rows, cols] (row stride cols) with boxes of
// box_rows x box_cols, 128-byte swizzle; out-of-range elements read as zero.
bool pipe_map_2d(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows, uint32_t box_cols,
                 uint32_t box_rows);

// Pool rows from `base` on seen as [groups of 8 rows][D / 64 panels][8 rows]
// [64 columns], with boxes of box_groups groups x `panels` panels: each group of
// a box lands as `panels` swizzle atoms of 1 KB.
bool pipe_map_pool(CUtensorMap* m, const void* base, uint64_t D, uint64_t groups, uint32_t panels,
                   uint32_t box_groups);

}  // namespace sda
