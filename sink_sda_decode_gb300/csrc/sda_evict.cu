// sda_evict.cu -- eviction from a cache held as a table of single slots: which
// positions of each sequence to keep by their accumulated attention weight,
// with tables and weights compacted and the freed slots listed.
//
// A sequence of n positions and a budget k < n keeps its first `first` and
// last `recent` positions and, of those between, the k - first - recent with
// the largest weight (-0 equal to +0, NaN below -inf, equal weights by
// increasing position).  Weights map to 32-bit keys that preserve that order,
// so the k-th key is found by an exact radix select (stopping once the digit's
// bin is kept whole); one ordered pass then gives every position its rank among
// the kept or the freed ones.
//
// evict_cluster_kernel: one CTA (tables of up to 4096 columns) or a cluster of 8
// or 6 a sequence, each CTA with its share of the positions in shared memory, so that
// scores and slots are read once; the digits' histograms and the kept counts of
// the CTAs are put together through distributed shared memory, and each warp
// writes the kept and the freed of 32 positions in a row at a time.  16 sequences
// of up to 131072 positions cut to 4096 take 37 us, against 179 with one CTA a
// sequence that reads its row again for every digit (evict_stream_kernel, left for
// tables whose share does not fit).  The bytes would take 2 us; what bounds it is the
// chain of the longest sequence: its share's load, three digits (each a histogram and
// two cluster barriers with the sums between them), the counts, the writes.
//
// In-place calls are safe: everything is read before anything is written (the
// cluster kernel), or a position before anything at or before it (the stream
// kernel: a kept position's rank is at most its own index).
#include <cuda_runtime.h>

#include <cstdint>

#include "sda_evict.cuh"
#include "sda_pipe.cuh"

namespace sda {

namespace {

constexpr int kThreads = 1024;
constexpr int kBins = 4096;       // of the widest digit (12 bits)
static_assert(kBins == 4 * kThreads, "four histogram bins per thread");
constexpr int kStreamBins = 2048;  // evict_stream_kernel: digits of 11, 11 and 10 bits

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

// Rows of up to kOneCta columns take one CTA, longer ones a cluster of 8 or 6: 14
// clusters of 8 run at once on a GB300, or 24 of 6, so that more than 14 sequences
// take clusters of 6 where their share fits (16 sequences of up to 131072, replayed
// from a graph: 36.6 us in clusters of 6, 39.2 us in two waves of clusters of 8).
constexpr int kOneCta = 4096, kFused = 4096, kClusters8 = 14;
constexpr size_t kMaxSmem = 200 * 1024;
static_assert(kMaxSmem / 8 / 32 <= kBins / 2, "the bits of a share's rows of 32 fit the histogram");
// Positions of a CTA's share of n positions: a multiple of 32.
__host__ __device__ inline int64_t share_of(int64_t n, int ctas) {
  return ((n + ctas - 1) / ctas + 31) / 32 * 32;
}

__device__ __forceinline__ uint32_t map_cta(const void* p, uint32_t cta) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(cta));
  return r;
}
__device__ __forceinline__ uint32_t load_cta(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint4 load4_cta(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
template <int CS>
__device__ __forceinline__ void all_sync() {
  if constexpr (CS > 1)
    asm volatile(
        "barrier.cluster.arrive.release.aligned;\n\t"
        "barrier.cluster.wait.acquire.aligned;" ::
            : "memory");
  else
    __syncthreads();
}

// FUSED: every CTA sums the freed counts before its sequence itself (at most
// kFused sequences, and out_len is not kv_len); otherwise evict_indptr_kernel has.
template <int CS, bool FUSED>
__global__ void __launch_bounds__(kThreads) evict_cluster_kernel(const EvictArgs a) {
  extern __shared__ uint32_t s_pos[];  // [share] scores, then [share] slots
  __shared__ __align__(16) uint32_t hist[kBins];
  __shared__ uint32_t warp_sums[kThreads / 32];
  __shared__ uint32_t s_digit, s_above, s_count, s_before, s_all;
  __shared__ uint2 s_tot;                     // this CTA's (certainly kept, tied) positions
  __shared__ uint2 s_warp[kThreads / 32];     // and its warps'
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x / CS, rank = blockIdx.x % CS;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = checked_len(a.kv_len, b, a.S);
  const int k = min(n, a.budget);
  int foff, ftotal;
  if constexpr (FUSED) {
    uint32_t before = 0, all = 0;
    int bad = 0;
    for (int x = tid; x < a.B; x += kThreads) {
      const int nx = a.kv_len[x];
      bad |= nx < 0 || nx > a.S;
      const uint32_t c = (uint32_t)max(checked_len(a.kv_len, x, a.S) - a.budget, 0);
      all += c;
      if (x < b) before += c;
    }
    before = __reduce_add_sync(0xffffffffu, before);
    all = __reduce_add_sync(0xffffffffu, all);
    if (lane == 0) s_warp[warp] = make_uint2(before, all);
    bad = __syncthreads_or(bad);
    if (warp == 0) {
      const uint32_t x = __reduce_add_sync(0xffffffffu, s_warp[lane].x);
      const uint32_t y = __reduce_add_sync(0xffffffffu, s_warp[lane].y);
      if (lane == 0) {
        s_before = x;
        s_all = y;
      }
    }
    __syncthreads();
    foff = (int)s_before;
    ftotal = (int)s_all;
    if (rank == 0 && tid == 0) {
      a.freed_indptr[b + 1] = foff + max(n - a.budget, 0);
      if (b == 0) a.freed_indptr[0] = 0;
      if (b == 0 && bad) atomicOr(a.status, 1);
    }
  } else {
    foff = a.freed_indptr[b];
    ftotal = a.freed_indptr[a.B];
  }
  const int64_t cap = share_of(a.S, CS);
  float* sc = reinterpret_cast<float*>(s_pos);
  int32_t* sl = reinterpret_cast<int32_t*>(s_pos + cap);
  // this CTA's positions [p0, p0 + cnt)
  const int share = (int)share_of(n, CS);
  const int p0 = min(n, rank * share), cnt = min(n - p0, share);
  {
    const float* row = a.scores + (int64_t)b * a.S + p0;
    const int32_t* slots = a.slots + (int64_t)b * a.S + p0;
#pragma unroll 4
    for (int x = tid; x < cnt; x += kThreads) {
      sc[x] = row[x];
      sl[x] = slots[x];
    }
  }
  // positions [m0, m1) compete for `need` places; the others are kept
  const int m0 = n > k ? a.first : n, m1 = n > k ? n - a.recent : n;
  const int c0 = min(max(m0 - p0, 0), cnt), c1 = max(min(m1 - p0, cnt), c0);  // of this CTA's
  uint32_t need = n > k ? (uint32_t)(k - a.first - a.recent) : 0u;
  uint32_t prefix = 0, mask = 0;
  bool nan_seen = false;
  for (int x = tid; x < kBins; x += kThreads) hist[x] = 0;
  __syncthreads();
  if (need == 0) {
    for (int x = c0 + tid; x < c1; x += kThreads) nan_seen |= weight_key(sc[x]) == 0u;
    prefix = 0xffffffffu;  // no key reaches it (+inf is 0xff800000)
    mask = 0xffffffffu;
  } else {
    // Digits: sign and exponent (9 bits, a few values among many keys: four
    // histograms, lanes take turns), then 11 and 12 bits of the mantissa.
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 23 : (pass == 1 ? 12 : 0);
      const int bins = pass == 0 ? 512 : (pass == 1 ? 2048 : 4096);
      const uint32_t copy = pass == 0 ? (uint32_t)(lane & 3) * 512u : 0u;
      for (int x = c0 + tid; x < c1; x += 8 * kThreads) {
        uint32_t key[8];  // all eight loads before the first of the atomics
#pragma unroll
        for (int e = 0; e < 8; ++e) key[e] = weight_key(sc[min(x + e * kThreads, c1 - 1)]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (x + e * kThreads < c1) {
            if (pass == 0) nan_seen |= key[e] == 0u;
            if ((key[e] & mask) == prefix) atomicAdd(&hist[copy + ((key[e] >> shift) & (bins - 1))], 1u);
          }
        }
      }
      if (pass == 0) {
        __syncthreads();
        if (tid < 512) hist[tid] += hist[512 + tid] + hist[1024 + tid] + hist[1536 + tid];
      }
      all_sync<CS>();
      // sums over the CTAs, 4 bins a thread
      uint4 sum = make_uint4(0, 0, 0, 0);
      if (4 * tid < bins) {
        if constexpr (CS > 1) {
          uint4 v[CS];
#pragma unroll
          for (int c = 0; c < CS; ++c) v[c] = load4_cta(map_cta(&hist[4 * tid], c));
#pragma unroll
          for (int c = 0; c < CS; ++c)
            sum.x += v[c].x, sum.y += v[c].y, sum.z += v[c].z, sum.w += v[c].w;
        } else {
          sum = *reinterpret_cast<const uint4*>(&hist[4 * tid]);
        }
      }
      // keys in the threads before this one, and so (from the total) in those behind
      const uint32_t mine = sum.x + sum.y + sum.z + sum.w;
      uint32_t total;
      const uint32_t before = scan_exclusive(mine, warp_sums, &total);
      uint32_t above = total - before - mine;  // keys in higher bins
      const uint32_t q[4] = {sum.w, sum.z, sum.y, sum.x};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (above < need && above + q[e] >= need) {
          s_digit = 4 * tid + 3 - e;
          s_above = above;
          s_count = q[e];
        }
        above += q[e];
      }
      all_sync<CS>();  // (every CTA has read the histograms, too)
      prefix |= s_digit << shift;
      mask |= (uint32_t)(bins - 1) << shift;
      need -= s_above;
      const bool whole = need == s_count;  // the same in every CTA
      for (int x = tid; x < kBins; x += kThreads) hist[x] = 0;
      __syncthreads();
      if (whole) break;
    }
  }
  // Warp w takes the positions [32 rows w, 32 rows (w + 1)), a row of 32 at a time:
  // which are kept for certain, and which are tied, as bits (where the histograms were).
  const int rows = (cnt + kThreads - 1) / kThreads;
  const int w0 = warp * rows * 32;
  uint2* bits = reinterpret_cast<uint2*>(hist) + warp * rows;
  uint32_t gt = 0, eq = 0;
#pragma unroll 8
  for (int r = 0; r < rows; ++r) {
    const int x = w0 + r * 32 + lane;
    const uint32_t m = weight_key(sc[min(x, max(cnt - 1, 0))]) & mask;
    const bool race = x >= c0 && x < c1;
    const uint32_t gb = __ballot_sync(0xffffffffu, x < cnt && (!race || m > prefix));
    const uint32_t eb = __ballot_sync(0xffffffffu, race && m == prefix);
    if (lane == 0) bits[r] = make_uint2(gb, eb);
    gt += __popc(gb);
    eq += __popc(eb);
  }
  if (lane == 0) s_warp[warp] = make_uint2(gt, eq);
  __syncthreads();
  const uint2 of = s_warp[lane];  // lane w: warp w's
  uint2 pre;
  pre.x = __reduce_add_sync(0xffffffffu, lane < warp ? of.x : 0u);
  pre.y = __reduce_add_sync(0xffffffffu, lane < warp ? of.y : 0u);
  if constexpr (CS > 1) {
    if (tid == kThreads - 1) s_tot = make_uint2(pre.x + of.x, pre.y + of.y);  // lane 31 of warp 31
    all_sync<CS>();
    uint2 v = make_uint2(0, 0);
    if (lane < rank) {  // lane c: CTA c's
      v.x = load_cta(map_cta(&s_tot.x, lane));
      v.y = load_cta(map_cta(&s_tot.y, lane));
    }
    pre.x += __reduce_add_sync(0xffffffffu, v.x);
    pre.y += __reduce_add_sync(0xffffffffu, v.y);
  }
  // in place: every CTA of the sequence holds its positions by now, so writes may begin
  float* orow = a.out_scores + (int64_t)b * a.out_S;
  int32_t* oslots = a.out_slots + (int64_t)b * a.out_S;
  uint32_t g_before = pre.x, e_before = pre.y;
  const uint32_t lt = (1u << lane) - 1;
#pragma unroll 4
  for (int r = 0; r < rows; ++r) {
    const int x = w0 + r * 32 + lane;
    const uint32_t gb = bits[r].x, eb = bits[r].y;
    const bool sure = (gb >> lane) & 1u, tied = (eb >> lane) & 1u;
    const uint32_t e = e_before + __popc(eb & lt);          // tied positions before this one
    const uint32_t rk = g_before + __popc(gb & lt) + min(e, need);  // its rank among the kept
    if (sure || (tied && e < need)) {
      orow[rk] = sc[x];
      oslots[rk] = sl[x];
    } else if (x < cnt) {
      a.freed[foff + p0 + x - (int)rk] = sl[x];
    }
    g_before += __popc(gb);
    e_before += __popc(eb);
  }
  for (int64_t p = k + rank * kThreads + tid; p < a.out_S; p += CS * kThreads) {
    orow[p] = 0.f;
    oslots[p] = -1;
  }
  // the freed list's unused tail
  for (int64_t e = ftotal + (int64_t)blockIdx.x * kThreads + tid; e < a.freed_capacity;
       e += (int64_t)gridDim.x * kThreads)
    a.freed[e] = -1;
  if (rank == 0 && tid == 0) a.out_len[b] = k;
  if (__syncthreads_or(nan_seen) && tid == 0) atomicOr(a.status, 8);
  all_sync<CS>();  // no CTA leaves while another may still read its shared memory
}

__global__ void __launch_bounds__(kThreads) evict_stream_kernel(const EvictArgs a) {
  pdl_wait();
  pdl_trigger();
  __shared__ uint32_t hist[kStreamBins];
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
      for (int i = tid; i < kStreamBins; i += kThreads) hist[i] = 0;
      __syncthreads();
      for (int p = m0 + tid; p < m1; p += kThreads) {
        const uint32_t key = weight_key(row[p]);
        nan_seen |= key == 0u;
        if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & dmask], 1u);
      }
      __syncthreads();
      // bins 2047 - 2i and 2046 - 2i belong to thread i: suffix sums
      const uint32_t hi = hist[kStreamBins - 1 - 2 * tid], lo = hist[kStreamBins - 2 - 2 * tid];
      uint32_t total;
      const uint32_t above = scan_exclusive(hi + lo, warp_sums, &total);
      if (above < need && above + hi >= need) {
        s_digit = kStreamBins - 1 - 2 * tid;
        s_above = above;
        s_count = hi;
      } else if (above + hi < need && above + hi + lo >= need) {
        s_digit = kStreamBins - 2 - 2 * tid;
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

cudaError_t evict_prepare() {
  const void* kernels[] = {
      reinterpret_cast<const void*>(evict_cluster_kernel<1, true>),
      reinterpret_cast<const void*>(evict_cluster_kernel<1, false>),
      reinterpret_cast<const void*>(evict_cluster_kernel<6, true>),
      reinterpret_cast<const void*>(evict_cluster_kernel<6, false>),
      reinterpret_cast<const void*>(evict_cluster_kernel<8, true>),
      reinterpret_cast<const void*>(evict_cluster_kernel<8, false>)};
  for (const void* k : kernels) {
    const cudaError_t e =
        cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxSmem);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t st) {
  const int cs = a.S <= kOneCta ? 1 : (a.B > kClusters8 && share_of(a.S, 6) * 8 <= (int64_t)kMaxSmem ? 6 : 8);
  const size_t smem = (size_t)share_of(a.S, cs) * 8;
  const bool staged = smem <= kMaxSmem;
  const bool fused = staged && a.B > 0 && a.B <= kFused && a.out_len != a.kv_len;
  if (!fused) {
    const cudaError_t e = launch_pdl(evict_indptr_kernel, dim3(1), dim3(kThreads), 0, st, a);
    if (e != cudaSuccess) return e;
    if (a.B == 0)  // nothing was freed: the whole list is its unused tail (-1 is all ones)
      return a.freed_capacity > 0
                 ? cudaMemsetAsync(a.freed, 0xff, (size_t)a.freed_capacity * sizeof(int32_t), st)
                 : cudaSuccess;
  } else {
    const cudaError_t e = cudaMemsetAsync(a.status, 0, sizeof(int32_t), st);
    if (e != cudaSuccess) return e;
  }
  if (!staged) return launch_pdl(evict_stream_kernel, dim3(a.B), dim3(kThreads), 0, st, a);
  auto go = [&](auto kernel) {
    return launch_pdl_cluster(kernel, dim3(a.B * cs), dim3(kThreads), cs, smem, st, a);
  };
  if (cs == 1) return fused ? go(evict_cluster_kernel<1, true>) : go(evict_cluster_kernel<1, false>);
  if (cs == 6) return fused ? go(evict_cluster_kernel<6, true>) : go(evict_cluster_kernel<6, false>);
  return fused ? go(evict_cluster_kernel<8, true>) : go(evict_cluster_kernel<8, false>);
}

}  // namespace sda
