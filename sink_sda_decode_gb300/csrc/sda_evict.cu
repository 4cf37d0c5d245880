// sda_evict.cu -- eviction from a cache held as a table of single slots: which
// positions of each sequence to keep by their accumulated attention weight,
// with tables and weights compacted and the freed slots listed.
//
// A sequence of n positions and a budget k < n keeps its first `first` and
// last `recent` positions and, of those between, the k - first - recent with
// the largest weight (-0 equal to +0, NaN below -inf, equal weights by
// increasing position).  Weights map to 32-bit keys that preserve that order,
// so the k-th key is found by an exact radix select (digits of 11, 11 and 10
// bits, stopping once the digit's bin is kept whole); one ordered pass then
// gives every position its rank among the kept or the freed ones.
//
// In-place calls are safe: a position is read before anything is written at
// or before it, because a kept position's rank is at most its own index.
#include <cuda_runtime.h>

#include <cstdint>

#include "sda_evict.cuh"

namespace sda {

namespace {

constexpr int kThreads = 1024;
constexpr int kBins = 2048;
static_assert(kBins == 2 * kThreads, "two histogram bins per thread");

__device__ __forceinline__ uint32_t weight_key(float f) {
  uint32_t u = __float_as_uint(f);
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0u;  // NaN: below every number
  if (u == 0x80000000u) u = 0u;                    // -0 ranks as +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ int checked_len(const int32_t* kv_len, int b, int64_t S) {
  const int n = kv_len[b];
  return n < 0 || n > S ? 0 : n;
}

// Exclusive scan over the block; *total receives the block's sum.
__device__ __forceinline__ uint32_t scan_exclusive(uint32_t v, uint32_t* warp_sums, uint32_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    uint32_t w = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  const uint32_t before = warp == 0 ? 0u : warp_sums[warp - 1];
  *total = warp_sums[kThreads / 32 - 1];
  __syncthreads();
  return before + x - v;
}

// freed_indptr = prefix sums of max(n_b - budget, 0); status bit 1 for a bad
// length.  A kernel of its own because out_len may be kv_len itself.
__global__ void __launch_bounds__(kThreads) evict_indptr_kernel(const EvictArgs a) {
  pdl_wait();
  pdl_trigger();
  __shared__ uint32_t warp_sums[kThreads / 32];
  uint32_t run = 0;
  int bad = 0;
  if (threadIdx.x == 0) a.freed_indptr[0] = 0;
  for (int b0 = 0; b0 < a.B; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    uint32_t c = 0;
    if (b < a.B) {
      const int n = a.kv_len[b];
      bad |= n < 0 || n > a.S;
      c = (uint32_t)max(checked_len(a.kv_len, b, a.S) - a.budget, 0);
    }
    uint32_t tot;
    const uint32_t ex = scan_exclusive(c, warp_sums, &tot);
    if (b < a.B) a.freed_indptr[b + 1] = (int32_t)(run + ex + c);
    run += tot;
  }
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) *a.status = bad ? 1 : 0;
}

__global__ void __launch_bounds__(kThreads) evict_kernel(const EvictArgs a) {
  pdl_wait();
  pdl_trigger();
  __shared__ uint32_t hist[kBins];
  __shared__ uint32_t warp_sums[kThreads / 32];
  __shared__ uint32_t s_digit, s_above, s_count;
  const int b = blockIdx.x, tid = threadIdx.x;
  const int n = checked_len(a.kv_len, b, a.S);
  const int k = min(n, a.budget);
  const int foff = a.freed_indptr[b];
  const float* row = a.scores + (int64_t)b * a.S;
  const int32_t* slots = a.slots + (int64_t)b * a.S;
  float* orow = a.out_scores + (int64_t)b * a.out_S;
  int32_t* oslots = a.out_slots + (int64_t)b * a.out_S;
  // positions [m0, m1) compete for `need` places; the others are kept
  const int m0 = n > k ? a.first : n, m1 = n > k ? n - a.recent : n;
  uint32_t need = n > k ? (uint32_t)(k - a.first - a.recent) : 0u;
  uint32_t prefix = 0, mask = 0;
  bool nan_seen = false;
  // NaN is reported wherever it competes, also when nothing has to be ranked
  if (need == 0) {
    for (int p = m0 + tid; p < m1; p += kThreads) nan_seen |= weight_key(row[p]) == 0u;
    prefix = 0xffffffffu;  // no key reaches it (NaN keys are 0, +inf maps to 0xff800000)
    mask = 0xffffffffu;
  } else {
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
      const uint32_t dmask = pass == 2 ? 0x3ffu : 0x7ffu;
      for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
      __syncthreads();
      for (int p = m0 + tid; p < m1; p += kThreads) {
        const uint32_t key = weight_key(row[p]);
        nan_seen |= key == 0u;
        if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & dmask], 1u);
      }
      __syncthreads();
      // bins 2047 - 2i and 2046 - 2i belong to thread i: suffix sums
      const uint32_t hi = hist[kBins - 1 - 2 * tid], lo = hist[kBins - 2 - 2 * tid];
      uint32_t total;
      const uint32_t above = scan_exclusive(hi + lo, warp_sums, &total);
      if (above < need && above + hi >= need) {
        s_digit = kBins - 1 - 2 * tid;
        s_above = above;
        s_count = hi;
      } else if (above + hi < need && above + hi + lo >= need) {
        s_digit = kBins - 2 - 2 * tid;
        s_above = above + hi;
        s_count = lo;
      }
      __syncthreads();
      prefix |= s_digit << shift;
      mask |= dmask << shift;
      need -= s_above;
      const bool whole = need == s_count;
      __syncthreads();
      if (whole) break;
    }
  }
  // kept: every key whose leading bits exceed prefix, and the first `need`
  // that equal it
  uint32_t kept = 0, ties = 0;
  for (int g0 = 0; g0 < n; g0 += kThreads) {
    const int p = g0 + tid;
    float s = 0.f;
    int32_t slot = 0;
    bool gt = false, eq = false;
    if (p < n) {
      s = row[p];
      slot = slots[p];
      if (p < m0 || p >= m1) {
        gt = true;
      } else {
        const uint32_t m = weight_key(s) & mask;
        gt = m > prefix;
        eq = m == prefix;
      }
    }
    uint32_t tot;
    const uint32_t ex = scan_exclusive((eq ? 1u << 16 : 0u) | (gt ? 1u : 0u), warp_sums, &tot);
    const uint32_t room = need > ties ? need - ties : 0u;
    const uint32_t rank = kept + (ex & 0xffffu) + min(ex >> 16, room);
    if (p < n) {
      if (gt || (eq && (ex >> 16) < room)) {
        orow[rank] = s;
        oslots[rank] = slot;
      } else {
        a.freed[foff + p - (int)rank] = slot;
      }
    }
    kept += (tot & 0xffffu) + min(tot >> 16, room);
    ties += tot >> 16;
  }
  for (int64_t p = k + tid; p < a.out_S; p += kThreads) {
    orow[p] = 0.f;
    oslots[p] = -1;
  }
  // the freed list's unused tail
  const int64_t total = a.freed_indptr[a.B];
  for (int64_t e = total + (int64_t)b * kThreads + tid; e < a.freed_capacity;
       e += (int64_t)a.B * kThreads)
    a.freed[e] = -1;
  if (tid == 0) a.out_len[b] = k;
  if (__syncthreads_or(nan_seen) && tid == 0) atomicOr(a.status, 8);
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t st) {
  cudaError_t e = launch_pdl(evict_indptr_kernel, dim3(1), dim3(kThreads), 0, st, a);
  if (e != cudaSuccess || a.B == 0) return e;
  return launch_pdl(evict_kernel, dim3(a.B), dim3(kThreads), 0, st, a);
}

}  // namespace sda
