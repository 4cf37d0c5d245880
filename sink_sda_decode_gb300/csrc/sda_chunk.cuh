// sda_chunk.cuh -- geometry shared by the paged-cache operators: which cached
// positions a token of a chunk sees, the work units of the chunk attention,
// and the launchers.
//
// Sequence b has m_b = q_indptr[b + 1] - q_indptr[b] new tokens and
// n_b = kv_len[b] cached positions, of which the new tokens' own rows are the
// last m_b.  Its token i stands at position p = n_b - m_b + i and sees the
// positions j <= p with (window == 0 or j > p - window or j < first).
// Position j's row is pool row base + block_table[b][j / K] * K + j % K.
#pragma once

#include <cstddef>

#include "sda_internal.cuh"

namespace sda {

struct ChunkGeom {
  const int32_t* q_indptr;     // [B + 1]
  const int32_t* kv_len;       // [B]
  const int32_t* block_table;  // [B, max_blocks]
  int B, T, H, D;
  int max_blocks, k_per_block;
  int64_t base, total_pages;
  int window, first;
  uint32_t h_mul;  // n / H = n h_mul >> h_shift for 0 <= n < 2^31 (div_h)
  int h_shift;
  void set_h() {
    int b = 0;
    while ((1 << b) < H) ++b;
    h_shift = 31 + b;
    h_mul = (uint32_t)(((1ull << h_shift) + H - 1) / H);
  }
};

// All heads share the cached rows, so the (token, head) rows of a sequence
// are one matrix of m_b * H rows of q, and a work unit is up to R consecutive
// rows of it: one tile of queries, whatever H.
struct alignas(16) ChunkUnit {
  int row0;     // first row of q (token * H + head)
  int nrows;    // rows of this unit, 1..R
  int b;        // sequence
  int pos0;     // position of row 0's token (negative if n_b < m_b)
  int h0;       // head of row 0; row i: token pos0 + (h0 + i) / H, head (h0 + i) % H
  int lo;       // positions below lo are visible only if they are below `first`
  int hi;       // positions from hi on are visible to no row
  int nf;       // KV tiles of the first positions (those below lo's tile)
  int ntiles;   // KV tiles: tiles 0..nf-1, then from the one that holds lo on (>= 1)
  int off;      // in a worker's record: its first tile of this unit
  int pad0, pad1;
};
static_assert(sizeof(ChunkUnit) == 48, "three 16-byte words");

constexpr float kLn2 = 0.6931471805599453f;

// Most cached positions of a sequence: a tile (up to 256) that holds the last of them
// ends within 32 bits.
constexpr int kMaxLen = 0x7fffffff - 511;

// The position that logical tile i of a unit starts at, with tiles of `tile` positions.
__host__ __device__ inline int chunk_tile_start(int i, int nf, int lo, int tile) {
  return (i < nf ? i : lo / tile + i - nf) * tile;
}

// Header of the workspace (256 bytes), and behind it one error word per CTA.
struct ChunkHeader {
  int n_units;
  int n_tiles;  // KV tiles of all units
  int per;      // attention mass: row tiles per worker
  int ctas;     // attention mass: workers with row tiles
  int error;    // 2 = bad lengths (nothing computed)
  int words;    // error words of this call (1 = a wait timed out, 3 = bad table entry)
  int pad[58];
};
static_assert(sizeof(ChunkHeader) == 256, "header is 256 bytes");
constexpr size_t kErrorWords = 256, kErrorBytes = 4 * kMaxPlanGrid;  // offset and size of the words

// Where a worker (a CTA, or a pair of CTAs) begins, and how far it goes.
struct alignas(16) ChunkStart {
  int b, r;  // sequence, and unit of it
  int off;   // first tile of that unit
  int nt;    // tiles in all (in the plan's list: tiles before it)
};

// The workers' ranges are equal in cost: a unit of R rows costs its tiles and this
// many more for its beginning and end (on a pair about 5500 cycles, at 1650 a tile).
// Equal numbers of tiles left the workers that had many short units far behind: 12
// sequences of 1 to 300 tokens over 300 to 6000 positions took 521 us (the median
// worker was done after 340), and 420 with equal costs.
constexpr int unit_cost(int R) { return R == 128 ? 3 : 1; }

// How the tiles are shared out.
//   kPlanned  ranges of equal cost, by a kernel before
//   kCut      the same, but every CTA finds its own beginning (few units): one launch
//             less (replayed from a graph, against kPlanned: one token of 16 heads over 64
//             caches 28.7 against 29.7 us, of 64 heads over 8 long caches 92.0 against 94.0,
//             drafted tokens 131.1 against 130.0, ragged prompts 421.5 against 420.5)
//   kWhole    whole units, every CTA its share: no merge of pieces is launched (prompts
//             with a window of 128: 188 us, 209 with a plan and a merge)
enum ChunkMode : int { kPlanned = 0, kCut = 1, kWhole = 2 };
constexpr int kFusedSeqs = 2048, kFusedUnits = 4096;  // most that the CTAs look through themselves

struct ChunkLayout {
  size_t start_off, rec_off, seq_off, ml_off, o_off, total;
  int grid, R, tile;  // R: rows per unit; grid: workers that share the tiles
  bool pair;          // units of 128 rows, 64 for each CTA of a cluster of two
  ChunkMode mode;
};
// Positions per KV tile (a multiple of 16).  With 64 rows of q at D = 512 two
// stages of 64 positions fit beside q in one CTA, or three of 48.  A step is bound by
// the time from a stage's load to its release (load, scores, softmax, PV), so three
// in flight win although their MMAs take 7 % more cycles a position: one token of 64
// heads over 8 caches of up to 65536 positions, 87 against 91 us.
constexpr int chunk_tile(int R, int D) { return R == 64 && D == 512 ? 48 : 64; }
// Whether KV tiles can be loaded as boxes of 16 rows: blocks hold a multiple of
// 16 rows, and the pool from `base` on whole groups of 8 (the tensor map counts
// in them).
inline bool chunk_boxes(const ChunkGeom& g) {
  const int64_t rows = g.total_pages - g.base;
  return g.k_per_block % 16 == 0 && rows > 0 && rows % 8 == 0;
}
// The layout of a call (the sizes depend on B, T, H and D alone).
ChunkLayout chunk_layout(const ChunkGeom& g, int num_sms);

// error = the largest of a workspace's error words.
cudaError_t launch_paged_error(const void* ws, int32_t* error, cudaStream_t st);

cudaError_t chunk_prepare();  // one-time kernel attributes on the current device
cudaError_t launch_chunk_plan(const ChunkGeom& g, const ChunkLayout& L, void* ws, cudaStream_t st);
cudaError_t launch_chunk_attn(const void* q, const void* kv, const ChunkGeom& g,
                              const float* attn_sink, float scale, void* out, float* lse,
                              const ChunkLayout& L, void* ws, cudaStream_t st);
cudaError_t launch_chunk_combine(const float* attn_sink, const ChunkGeom& g, void* out, float* lse,
                                 const ChunkLayout& L, void* ws, cudaStream_t st);

inline size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// Attention mass.
struct MassLayout {
  size_t units_off, seq_off, cta_off, part_off, total;
  int u_max, grid;
};
MassLayout mass_layout(int B, int64_t S, int num_sms);
cudaError_t mass_prepare();
cudaError_t launch_mass(const void* q, const void* kv, const ChunkGeom& g, const float* lse,
                        float scale, const float* prev, float decay, float* out,
                        const MassLayout& L, void* ws, cudaStream_t st);

// sda_api.cu: the text that sda_last_cuda_error returns.
void note_cuda_error(cudaError_t e, const char* where);

#ifdef __CUDACC__
// n / H.  With b = ceil(log2 H), h_mul = (2^(31 + b) + e) / H for some 0 <= e < H, so
// n h_mul / 2^(31 + b) = n / H + (n / 2^31) (e / 2^b) / H exceeds n / H by less than 1 / H.
__device__ __forceinline__ int div_h(const ChunkGeom& g, int n) {
  return (int)(((unsigned long long)(unsigned)n * g.h_mul) >> g.h_shift);
}
__device__ __forceinline__ int units_of(const ChunkGeom& g, int R, int b) {
  const int m = __ldg(g.q_indptr + b + 1) - __ldg(g.q_indptr + b);
  return (int)(((long long)m * g.H + R - 1) / R);
}
__device__ __forceinline__ bool lengths_bad(const ChunkGeom& g, int b) {
  const int q0 = __ldg(g.q_indptr + b), q1 = __ldg(g.q_indptr + b + 1), n = __ldg(g.kv_len + b);
  return q0 < 0 || q1 < q0 || q1 > g.T || n < 0 || n > kMaxLen ||
         n > (long long)g.max_blocks * g.k_per_block;
}
// Unit r of sequence b (off is left 0).
__device__ __forceinline__ ChunkUnit chunk_unit(const ChunkGeom& g, int R, int tile, int b, int r) {
  const int q0 = __ldg(g.q_indptr + b), m = __ldg(g.q_indptr + b + 1) - q0, n = __ldg(g.kv_len + b);
  const int r0 = r * R;  // row in the sequence's m * H rows
  ChunkUnit d;
  d.row0 = q0 * g.H + r0;
  d.nrows = min(R, m * g.H - r0);
  d.b = b;
  const int tok = div_h(g, r0);
  d.pos0 = n - m + tok;
  d.h0 = r0 - tok * g.H;
  const int p_hi = d.pos0 + div_h(g, d.h0 + d.nrows - 1);
  d.hi = max(p_hi + 1, 0);
  d.lo = g.window > 0 ? (int)max((long long)d.pos0 - g.window + 1, 0ll) : 0;
  if (d.hi == 0) d.lo = 0;
  const int lot = d.lo / tile;
  d.nf = (min(g.first, lot * tile) + tile - 1) / tile;
  // rows that see nothing: one tile of masked positions
  d.ntiles = max(d.nf + (d.hi + tile - 1) / tile - lot, 1);
  d.off = d.pad0 = d.pad1 = 0;
  return d;
}

// Exclusive scan over a block of 1024 threads; *total (shared) holds the sum.
__device__ inline long long scan_exclusive(long long v, long long* warp_sums, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    const long long w = warp_sums[lane];
    long long s = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    warp_sums[lane] = s - w;
    if (lane == 31) *total = s;
  }
  __syncthreads();
  const long long r = warp_sums[warp] + x - v;
  __syncthreads();  // warp_sums is rewritten by the next call (*total after its first barrier)
  return r;
}

// Last index i in [0, n) with a[i] <= x; a non-decreasing, a[0] <= x.
__device__ __forceinline__ int last_le(const int* a, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}
#endif

}  // namespace sda
