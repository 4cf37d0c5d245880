// sda_chunk_dev.cuh -- what the chunk attention's two kernels share: their
// parameters and the walk over a CTA's tiles.
#pragma once

#include <cuda_bf16.h>

#include "sda_chunk.cuh"
#include "sda_pipe.cuh"

namespace sda {

constexpr float kHeadroom = 8.0f;  // log2: the running reference is raised when a score exceeds it by this

struct ChunkParams {
  const __nv_bfloat16* kv;
  const float* attn_sink;
  __nv_bfloat16* out;
  float* lse;
  ChunkHeader* hdr;
  const ChunkUnit* units;
  const int* cta_unit;
  float2* part_ml;
  float* part_o;
  ChunkGeom g;
  float qk_scale_log2;
  uint64_t wait_timeout_ns;
};

__device__ __forceinline__ ChunkUnit load_unit(const ChunkUnit* u) {
  ChunkUnit d;
  int4* w = reinterpret_cast<int4*>(&d);
#pragma unroll
  for (int i = 0; i < 3; ++i) w[i] = __ldcg(reinterpret_cast<const int4*>(u) + i);
  return d;
}

// Walks the CTA's tiles in order; every role walks the same ones.
struct Cursor {
  const ChunkUnit* units;
  int u;           // unit
  int i;           // logical tile within the unit
  int left;        // tiles left to this CTA, this one included
  bool first;      // first tile of this CTA's piece of the unit
  int b, lo, hi, nf, ntiles;
  __device__ __forceinline__ void load() {
    const int4 a = __ldcg(reinterpret_cast<const int4*>(units + u) + 1);
    ntiles = __ldcg(&units[u].ntiles);
    b = __ldcg(&units[u].b);
    lo = a.y;
    hi = a.z;
    nf = a.w;
  }
  __device__ __forceinline__ void init(const ChunkUnit* us, int u0, int t0, int n) {
    units = us;
    u = u0;
    left = n;
    first = true;
    if (left > 0) {
      load();
      i = t0 - __ldcg(&units[u].cum);
    }
  }
  __device__ __forceinline__ bool last() const { return left == 1 || i == ntiles - 1; }
  __device__ __forceinline__ void next() {
    first = false;
    --left;
    if (++i == ntiles && left > 0) {
      ++u;
      i = 0;
      first = true;
      load();
    }
  }
};

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
__device__ __forceinline__ int seen_row(const ChunkParams& p, const Cursor& c, int j) {
  if (j >= c.hi || (j < c.lo && j >= p.g.first)) return -1;
  return pool_row_of(p.g, &p.hdr->error, c.b, j);
}
// The box of 16 positions from j on, in groups of 8 pool rows from `base` on:
// 16 positions lie in one block (tiles and blocks start at multiples of 16) and
// so in 16 pool rows in a row.  A box that no row sees is read from behind the
// pool, which fills it with zeros.
__device__ __forceinline__ int box_group(const ChunkParams& p, const Cursor& c, int j) {
  const int behind = (int)((p.g.total_pages - p.g.base) / 8);
  int x = j;  // the box's first position that is seen, if any, tells its block
  if (x < c.lo && x >= p.g.first) x = c.lo;
  if (x >= j + 16) return behind;
  const int r = seen_row(p, c, x);
  return r < 0 ? behind : (int)((r - (x - j) - p.g.base) / 8);
}

ChunkParams chunk_params(const void* kv, const ChunkGeom& g, const float* attn_sink, float scale,
                         void* out, float* lse, const ChunkLayout& L, void* ws);
cudaError_t pair_prepare();
cudaError_t launch_chunk_pair(const CUtensorMap& tq, const CUtensorMap& tkv, const ChunkParams& p,
                              bool tma, const ChunkLayout& L, cudaStream_t st);

}  // namespace sda
