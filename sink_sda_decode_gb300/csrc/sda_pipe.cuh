// sda_pipe.cuh -- bounded mbarrier waits and tensor-map encoding shared by the
// paged-cache kernels (chunk attention and attention mass).
#pragma once

#include <cuda.h>

#include "sda_internal.cuh"
#include "umma_ptx.cuh"

namespace sda {

#ifdef __CUDACC__
// Where a bounded wait reports a timeout, and after how long.
struct PipeWait {
  volatile int* abort_flag;  // shared: set once any role of the CTA gave up
  int* error;                // global error word (1 = a wait timed out)
  uint64_t timeout_ns;
};

// Bounded wait.  Returns false (and raises the abort flags) on timeout; once
// any role has aborted, every later wait returns false at once, so all roles
// run to the end of their loops quickly and the CTA exits.
__device__ __forceinline__ bool pipe_wait(uint32_t bar, uint32_t parity, const PipeWait& w) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  if (*w.abort_flag) return false;
  const uint64_t t0 = ptx::globaltimer_ns();
  for (uint32_t it = 1;; ++it) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    if ((it & 63u) == 0) {
      if (*w.abort_flag) return false;
      if (ptx::globaltimer_ns() - t0 > w.timeout_ns) {
        *w.abort_flag = 1;
        atomicExch(w.error, 1);
        return false;
      }
    }
  }
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
#endif

// A 2-D bf16 tensor map over [rows, cols] (row stride cols) with boxes of
// box_rows x box_cols, 128-byte swizzle; out-of-range elements read as zero.
bool pipe_map_2d(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows, uint32_t box_cols,
                 uint32_t box_rows);

}  // namespace sda
