// sda_chunk_dev.cuh -- what the chunk attention's two kernels share: their
// parameters and the walk over a CTA's tiles.
#pragma once

#include <cuda_bf16.h>

#include "sda_chunk.cuh"
#include "sda_pipe.cuh"

namespace sda {

// The lowest n bits, n up to 10.
__device__ __forceinline__ uint32_t low_bits(int n) { return (1u << min(max(n, 0), 10)) - 1u; }
// Which of the positions j .. j + 9 a row at position pos sees, as bits: a few operations
// a row, where comparing element by element took about ten an element.  (With this and
// div_h, replayed prompts with a window of 128 take 156 us where they took 187, ragged
// prompts 392 to 399 where they took 416; a prompt without masks 1.35 ms, 1.34 before.)
__device__ __forceinline__ uint32_t seen_bits(int pos, int j, int window, int first) {
  const int d = max(pos - j + 1, 0);
  const uint32_t causal = low_bits(d);
  return window == 0 ? causal : causal & (~low_bits(d - window) | low_bits(first - j));
}

constexpr float kHeadroom = 8.0f;  // log2: the running reference is raised when a score exceeds it by this

// The running reference of a row that has no score yet, finite so that a score of -inf
// (an overflow, say) has weight 2^-inf = 0 against it too, not 2^(-inf + inf) = NaN.  What
// is stored of it, or goes into lse, is -inf.
constexpr float kNoScore = -3.402823466e38f;

struct ChunkParams {
  const __nv_bfloat16* kv;
  const float* attn_sink;
  __nv_bfloat16* out;
  float* lse;
  ChunkHeader* hdr;
  ChunkStart* starts;
  ChunkUnit* recs;  // recs[k]: the unit that worker k begins in, for the combine
  int mode, workers;
  float2* part_ml;
  float* part_o;
  ChunkGeom g;
  float qk_scale_log2;
  uint64_t wait_timeout_ns;
};

// Walks units from one on.
struct UnitWalk {
  int b, r, nu;  // unit r of sequence b, which has nu
  __device__ __forceinline__ void init(const ChunkGeom& g, int R, const ChunkStart& s) {
    b = s.b;
    r = s.r;
    nu = s.nt > 0 ? units_of(g, R, b) : 0;
  }
  __device__ __forceinline__ void next(const ChunkGeom& g, int R) {
    ++r;
    while (r >= nu) {
      r = 0;
      nu = units_of(g, R, ++b);
    }
  }
};

// Walks a worker's tiles in order; every role walks the same ones.  R: rows of
// a unit.
template <int R, int TILE>
struct Cursor {
  UnitWalk w;
  int i;       // logical tile within the unit
  int left;    // tiles left, this one included
  bool first;  // first tile of this worker's piece of the unit
  int b, lo, hi, nf, ntiles, row0;
  __device__ __forceinline__ void load(const ChunkGeom& g) {
    const ChunkUnit d = chunk_unit(g, R, TILE, w.b, w.r);
    b = w.b;
    lo = d.lo;
    hi = d.hi;
    nf = d.nf;
    ntiles = d.ntiles;
    row0 = d.row0;
  }
  __device__ __forceinline__ void init(const ChunkGeom& g, const ChunkStart& s) {
    w.init(g, R, s);
    left = s.nt;
    first = true;
    i = s.off;
    if (left > 0) load(g);
  }
  __device__ __forceinline__ bool last() const { return left == 1 || i == ntiles - 1; }
  __device__ __forceinline__ int start() const { return chunk_tile_start(i, nf, lo, TILE); }
  __device__ __forceinline__ void next(const ChunkGeom& g) {
    first = false;
    --left;
    if (++i == ntiles && left > 0) {
      w.next(g, R);
      i = 0;
      first = true;
      load(g);
    }
  }
};

// Where worker `worker` begins; called by all THREADS threads of the CTA, which
// then are past a barrier.  `s_seq` (kFusedSeqs + 1 words) and `scratch` (64 words)
// are shared memory that is free until then.  *bad: the lengths broke the contract.
// The merge is launched all the same and goes by the records, so the caller then
// (kCut) records that the worker begins in no unit: the workspace may hold an earlier
// call's record, or anything.
template <int THREADS, int R, int TILE>
__device__ __noinline__ ChunkStart chunk_begin(const ChunkParams& p, int worker, int* s_seq,
                                                  int* scratch, bool* bad) {
  const ChunkGeom& g = p.g;
  ChunkStart st = {0, 0, 0, 0};
  *bad = false;
  if (p.mode == kPlanned) {
    const int4 v = __ldcg(reinterpret_cast<const int4*>(p.starts + worker));
    return ChunkStart{v.x, v.y, v.z, __ldcg(&p.starts[worker + 1].nt) - v.w};
  }
  constexpr int kW = THREADS / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  long long* sums = reinterpret_cast<long long*>(scratch);  // [kW]
  int* found = scratch + 2 * kW;                             // [5]
  // exclusive prefix of one value per thread, and the total
  auto scan = [&](long long v, long long* total) {
    long long x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();  // (sums may be rewritten)
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    long long before = 0, all = 0;
    for (int w = 0; w < kW; ++w) {
      const long long s = sums[w];
      if (w < warp) before += s;
      all += s;
    }
    *total = all;
    return before + x - v;
  };
  // s_seq[b] = units of the sequences before b
  const int each = (g.B + THREADS - 1) / THREADS;
  const int b0 = min(tid * each, g.B), b1 = min(b0 + each, g.B);
  int wrong = 0;
  long long mine = 0, U;
  for (int b = b0; b < b1; ++b) {
    if (lengths_bad(g, b)) wrong = 1;
    else mine += units_of(g, R, b);
  }
  long long at = scan(mine, &U);
  *bad = __syncthreads_or(wrong);
  if (*bad) return st;
  for (int b = b0; b < b1; ++b) {
    s_seq[b] = (int)at;
    at += units_of(g, R, b);
  }
  if (tid == 0) s_seq[g.B] = (int)U;
  __syncthreads();
  if (p.mode == kWhole) {
    const int lo = (int)(U * worker / p.workers), hi = (int)(U * (worker + 1) / p.workers);
    long long nt = 0, tot;
    for (int u = lo + tid; u < hi; u += THREADS) {
      const int b = last_le(s_seq, g.B, u);
      nt += chunk_unit(g, R, TILE, b, u - s_seq[b]).ntiles;
    }
    scan(nt, &tot);
    if (lo < hi) {
      st.b = last_le(s_seq, g.B, lo);
      st.r = lo - s_seq[st.b];
      st.nt = (int)tot;
    }
  } else {
    // each thread a stretch of units
    const int eu = ((int)U + THREADS - 1) / THREADS;
    const int u0 = min(tid * eu, (int)U), u1 = min(u0 + eu, (int)U);
    long long nt = 0, tt;
    UnitWalk w = {};
    auto from = [&]() {
      w.b = last_le(s_seq, g.B, u0);
      w.r = u0 - s_seq[w.b];
      w.nu = units_of(g, R, w.b);
    };
    if (u0 < u1) {
      from();
      for (int u = u0; u < u1; ++u) {
        nt += chunk_unit(g, R, TILE, w.b, w.r).ntiles;
        if (u + 1 < u1) w.next(g, R);
      }
    }
    const long long tiles = scan(nt, &tt);  // of the units before this stretch
    if (tt > 0x7fffffffll) {
      *bad = true;
      return st;
    }
    const long long cost = tt + U * unit_cost(R);
    const long long per = cost > 0 ? (cost + p.workers - 1) / p.workers : 1;
    const long long mine0 = tiles + (long long)u0 * unit_cost(R);
    const long long mine1 = mine0 + nt + (long long)(u1 - u0) * unit_cost(R);
    // this worker's beginning and the next one's, where they lie in this stretch
    for (int e = 0; e < 2; ++e) {
      const long long at_c = (worker + e) * per;
      if (at_c < mine0 || at_c >= mine1) continue;
      from();
      long long t = tiles, c = mine0;
      for (;;) {
        ChunkUnit d = chunk_unit(g, R, TILE, w.b, w.r);
        if (at_c < c + d.ntiles + unit_cost(R)) {
          d.off = (int)max(at_c - c - unit_cost(R), 0ll);
          if (e == 0) {
            found[0] = w.b;
            found[1] = w.r;
            found[2] = d.off;
            p.recs[worker] = d;
          }
          found[3 + e] = (int)(t + d.off);
          break;
        }
        t += d.ntiles;
        c += d.ntiles + unit_cost(R);
        w.next(g, R);
      }
    }
    if (tid == 0 && worker * per >= cost) p.recs[worker] = ChunkUnit{-1};
    __syncthreads();
    if (worker * per < cost) {
      const int end = (worker + 1) * per < cost ? found[4] : (int)tt;
      st = ChunkStart{found[0], found[1], found[2], end - found[3]};
    }
  }
  ptx::fence_proxy_async_smem();  // the tiles will be written here through the async proxy
  __syncthreads();
  return st;
}

// Pool row of position j of sequence b; -1 for a table entry outside the pool
// (which raises the error word).
__device__ __forceinline__ int pool_row_of(const ChunkGeom& g, int* error, int b, int j) {
  const int blk = __ldg(g.block_table + (size_t)b * g.max_blocks + j / g.k_per_block);
  const long long s = g.base + (long long)blk * g.k_per_block + j % g.k_per_block;
  if (blk < 0 || s >= g.total_pages) {
    atomicExch(error, 3);
    return -1;
  }
  return (int)s;
}
// Pool row of position j of the cursor's unit; -1: no row of the unit sees it
// (it is not read: zeros).
template <typename C>
__device__ __forceinline__ int seen_row(const ChunkParams& p, int* error, const C& c, int j) {
  if (j >= c.hi || (j < c.lo && j >= p.g.first)) return -1;
  return pool_row_of(p.g, error, c.b, j);
}
// The box of 16 positions from j on, in groups of 8 pool rows from `base` on:
// 16 positions lie in one block (tiles and blocks start at multiples of 16) and
// so in 16 pool rows in a row.  A box that no row sees is read from behind the
// pool, which fills it with zeros.
// The pool may end in the middle of a box (it holds groups of 8): what lies behind is
// filled with zeros too, and raises the error word if it is seen.  y: the box's group;
// last: the last of its positions that is seen.  (Boxes begin at every other group, so
// the last group is one's first only where its second half does not exist.)
__device__ __forceinline__ bool ends_behind(const ChunkGeom& g, int y, int j, int last) {
  return y == (int)((g.total_pages - g.base) / 8) - 1 && last >= j + 8;
}
template <typename C>
__device__ __forceinline__ int box_group(const ChunkParams& p, int* error, const C& c, int j, bool* over) {
  const int behind = (int)((p.g.total_pages - p.g.base) / 8);
  int x = j;  // the box's first position that is seen, if any, tells its block
  if (x < c.lo && x >= p.g.first) x = c.lo;
  if (x >= j + 16) return behind;
  const int r = seen_row(p, error, c, x);
  if (r < 0) return behind;
  const int y = (int)((r - (x - j) - p.g.base) / 8);
  const int last = min(j + 15, c.hi - 1);
  *over |= ends_behind(p.g, y, j, last < c.lo ? min(last, p.g.first - 1) : last);
  return y;
}

ChunkParams chunk_params(const void* kv, const ChunkGeom& g, const float* attn_sink, float scale,
                         void* out, float* lse, const ChunkLayout& L, void* ws);
cudaError_t pair_prepare();
cudaError_t launch_chunk_pair(const CUtensorMap& tq, const CUtensorMap& tkv, const ChunkParams& p,
                              bool tma, const ChunkLayout& L, cudaStream_t st);

}  // namespace sda
