// sda_chunk_plan.cu -- work plan of the chunk attention, and the merge of
// units that the plan cut.
//
// Everything runs on the device because the lengths live there and the call must
// stay capturable.  The units' KV tiles form one sequence, which is cut into ranges
// of equal cost, one per worker ("split-L").  A unit that a range boundary cuts becomes
// pieces, each of which leaves an unnormalised (m, l, acc); the combine kernel
// merges them.  With few units every CTA of the attention kernel finds its own
// range (sda_chunk_dev.cuh); this file's plan kernel does it for many.
#include <cuda_bf16.h>

#include "sda_chunk.cuh"

namespace sda {

namespace {

constexpr int kPlanThreads = 1024;

__global__ void __launch_bounds__(kPlanThreads) chunk_plan_kernel(
    const ChunkGeom g, int R, int tile, int grid, ChunkHeader* __restrict__ hdr,
    ChunkStart* __restrict__ starts, ChunkUnit* __restrict__ recs, int* __restrict__ seq_unit) {
  __shared__ long long warp_sums[32];
  __shared__ long long s_total;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  // seq_unit[b] = units of the sequences before b; lengths that make no sense stop the plan
  int bad = 0;
  long long U = 0;
  for (int b0 = 0; b0 < g.B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    int nu = 0;
    if (b < g.B) {
      if (lengths_bad(g, b)) bad = 1;
      else nu = units_of(g, R, b);
    }
    const long long ex = scan_exclusive(nu, warp_sums, &s_total);
    const long long tot = s_total;
    if (b < g.B) seq_unit[b] = (int)min(U + ex, 0x7fffffffll);
    U += tot;
    __syncthreads();
  }
  bad = __syncthreads_or(bad);
  const int nu = bad ? 0 : (int)U;
  long long tt = 0, cost = 0;  // tiles, and cost, of all units
  long long per = 1;
  // first the sums, then the units that hold the range boundaries
  for (int pass = 0; pass < 2; ++pass) {
    long long run_t = 0, run_c = 0;
    for (int u0 = 0; u0 < nu; u0 += kPlanThreads) {
      const int u = u0 + tid;
      ChunkUnit d = {};
      int b = 0;
      if (u < nu) {
        b = last_le(seq_unit, g.B, u);  // (sequences without tokens share a start)
        d = chunk_unit(g, R, tile, b, u - seq_unit[b]);
      }
      const long long before = run_t + scan_exclusive(d.ntiles, warp_sums, &s_total);
      const long long units = min(kPlanThreads, nu - u0);
      if (pass == 1 && u < nu) {
        const long long c0 = before + (long long)u * unit_cost(R), c1 = c0 + d.ntiles + unit_cost(R);
        for (long long k = (c0 + per - 1) / per; k * per < c1 && k < grid; ++k) {
          d.off = (int)max(k * per - c0 - unit_cost(R), 0ll);
          starts[k] = ChunkStart{b, u - seq_unit[b], d.off, (int)(before + d.off)};
          recs[k] = d;
        }
      }
      run_t += s_total;
      run_c += s_total + units * unit_cost(R);
      __syncthreads();
    }
    if (pass == 0) {
      if (run_t > 0x7fffffffll) bad = 1;  // uniform: every thread has the same sum
      tt = bad ? 0 : run_t;
      cost = bad ? 0 : run_c;
      per = cost > 0 ? (cost + grid - 1) / grid : 1;
      if (tt == 0) break;
    }
  }
  for (int k = tid; k <= grid; k += kPlanThreads) {
    if (k == grid || k * per >= cost) {
      starts[k] = ChunkStart{0, 0, 0, (int)tt};
      if (k < grid) recs[k] = ChunkUnit{-1};
    }
  }
  if (tid == 0) {
    hdr->n_units = nu;
    hdr->n_tiles = (int)tt;
    hdr->error = bad ? 2 : 0;
  }
}

// The largest of a workspace's error words.
__global__ void paged_error_kernel(const ChunkHeader* __restrict__ hdr, int32_t* __restrict__ error) {
  const int* words = reinterpret_cast<const int*>(reinterpret_cast<const char*>(hdr) + kErrorWords);
  int e = threadIdx.x == 0 ? hdr->error : 0;
  for (int i = threadIdx.x; i < min(hdr->words, kMaxPlanGrid); i += 32) e = max(e, words[i]);
  e = __reduce_max_sync(0xffffffffu, e);
  if (threadIdx.x == 0) *error = e;
}

// Merge of the pieces of cut units.  Block (x = k - 1, y): the beginning of worker
// k's range; it acts if that is the first to cut its unit.  A warp takes 128 columns
// (all of D below that) of one row.  Piece 0 lies in slot 2 (k - 1) + 1 (the unit starts
// in worker k - 1's range), piece i in slot 2 (k - 1 + i).
// What bounds it is the chain of dependent loads: after the two records that tell
// whether a block acts, those of the workers behind k and the (m, l) of all pieces that
// there may be are loaded together, then the partials of P pieces at a time.
constexpr int kCombineWarps = 8;
// A pair's units are seldom cut more than once, and with few registers more rows are
// under way (drafted tokens, replayed from a graph: 123.9 us with P = 2, 125.9 with 3,
// 126.7 with 1, 131.3 with 8); a step's few rows are cut into up to 19 pieces (one token
// over 8 long caches: 92.0 us with P = 8, 92.2 with 4, 93.7 with 2).
constexpr int kPiecesPair = 2, kPiecesOne = 8;

template <int D>
struct CombineCfg {
  static constexpr int kWarpsRow = D < 128 ? 1 : D / 128;  // warps of a row
  static constexpr int kRows = kCombineWarps / kWarpsRow;  // rows of a block
  static constexpr int kPer = D < 128 ? 2 : 4;             // columns of a lane
};

// Loads that stay where they are written: the compiler else puts them one by one
// before their uses.
__device__ __forceinline__ void load_here(const float* p, float (&v)[4]) {
  asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
               : "l"(p));
}
__device__ __forceinline__ void load_here(const float* p, float (&v)[2]) {
  asm volatile("ld.global.v2.f32 {%0, %1}, [%2];" : "=f"(v[0]), "=f"(v[1]) : "l"(p));
}

template <int D, int P>
__global__ void __launch_bounds__(kCombineWarps * 32) chunk_combine_kernel(
    const float* __restrict__ attn_sink, int H, int R, __nv_bfloat16* __restrict__ out,
    float* __restrict__ lse, int workers, const ChunkUnit* __restrict__ recs, const float2* __restrict__ part_ml,
    const float* __restrict__ part_o) {
  using C = CombineCfg<D>;
  pdl_wait();
  pdl_trigger();
  const int k = blockIdx.x + 1;
  const ChunkUnit un = recs[k];  // the unit that worker k begins in
  const int row_before = recs[k - 1].row0, off_before = recs[k - 1].off;
  // not cut here, or cut by an earlier beginning already
  if (un.off == 0 || un.row0 < 0 || (row_before == un.row0 && off_before > 0)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.y * C::kRows + warp / C::kWarpsRow;
  const int col = (warp % C::kWarpsRow) * 128 + lane * C::kPer;
  if (row >= un.nrows) return;
  auto slot = [&](int i) { return (size_t)(i == 0 ? 2 * (k - 1) + 1 : 2 * (k - 1 + i)); };
  auto begins_here = [&](int x) { return x < workers && recs[x].row0 == un.row0 && recs[x].off > 0; };
  // lane i: worker k - 1 + i, whose range begins in the unit's piece i if that exists
  float2 ml0 = make_float2(-INFINITY, 0.f);
  if (k - 1 + lane < workers) ml0 = part_ml[slot(lane) * R + row];
  const float sink = attn_sink[(un.h0 + row) % H], ms = sink * kLog2e;
  uint32_t not_in = __ballot_sync(0xffffffffu, lane > 0 && !begins_here(k - 1 + lane));
  int np = not_in ? __ffs(not_in) - 1 : 32;
  for (int x0 = k + 31; not_in == 0; x0 += 32) {
    not_in = ~__ballot_sync(0xffffffffu, begins_here(x0 + lane));
    np += not_in ? __ffs(not_in) - 1 : 32;
  }
  if (lane >= np) ml0 = make_float2(-INFINITY, 0.f);
  auto ml_of = [&](int i) {
    return i < np ? part_ml[slot(i) * R + row] : make_float2(-INFINITY, 0.f);
  };
  float mk = ml0.x;
  for (int i = lane + 32; i < np; i += 32) mk = fmaxf(mk, ml_of(i).x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mk = fmaxf(mk, __shfl_xor_sync(0xffffffffu, mk, o));
  const float M = fmaxf(ms, mk);
  const bool dead = ms == INFINITY || M == -INFINITY;
  float den = 0.f;
  float acc[C::kPer] = {};
  for (int i0 = 0; i0 < np && !dead; i0 += 32) {
    const float2 ml = i0 == 0 ? ml0 : ml_of(i0 + lane);
    // (a piece whose rows are all masked has m = -inf, l = 0 and weight 0)
    const float w = i0 + lane < np ? ex2_approx(ml.x - M) : 0.f;
    den += ml.x == -INFINITY ? ml.y : ml.y * w;
    const int n = min(32, np - i0);
    for (int j0 = 0; j0 < n; j0 += P) {
      float v[P][C::kPer];
#pragma unroll
      for (int j = 0; j < P; ++j)
        load_here(part_o + (slot(i0 + min(j0 + j, n - 1)) * R + row) * D + col, v[j]);
#pragma unroll
      for (int j = 0; j < P; ++j) {
        const float wj = __shfl_sync(0xffffffffu, w, (j0 + j) & 31);
        if (j0 + j < n) {
#pragma unroll
          for (int x = 0; x < C::kPer; ++x) acc[x] += wj * v[j][x];
        }
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
  if (!dead) den += ex2_approx(ms - M);
  const float inv = dead ? 0.f : 1.f / den;
  const size_t orow = (size_t)un.row0 + row;
#pragma unroll
  for (int x = 0; x < C::kPer; x += 2) {
    // "+ 0.f" turns -0 into +0 (a factor of 0 when the sink is +inf)
    const __nv_bfloat162 v = __floats2bfloat162_rn(acc[x] * inv + 0.f, acc[x + 1] * inv + 0.f);
    *reinterpret_cast<__nv_bfloat162*>(out + orow * D + col + x) = v;
  }
  // (the sink alone: as it is; a NaN that was seen: NaN)
  if (col == 0)
    lse[orow] = den != den ? den : mk == -INFINITY ? sink : (dead ? M * kLn2 : (M + log2f(den)) * kLn2);
}

}  // namespace

ChunkLayout chunk_layout(const ChunkGeom& g, int num_sms) {
  ChunkLayout L;
  const int64_t rows = (int64_t)g.T * g.H;
  // 16-row units where a sequence has at most 16 rows on average (a step of
  // few heads): q then takes a quarter of the shared memory and three KV stages
  // of 64 positions fit, and the rows' masks and stores are not padded to 64.
  L.R = rows <= (int64_t)16 * g.B ? 16 : 64;
  L.grid = num_sms < kMaxPlanGrid ? num_sms : kMaxPlanGrid;
  // With more than 128 rows a sequence on average, pairs of CTAs take units of 128 rows.
  L.pair = g.D >= 256 && rows > (int64_t)128 * g.B;
  if (L.pair) {
    L.R = 128;
    L.grid /= 2;
  }
  L.tile = chunk_tile(L.R, g.D);
  // Where no unit can have more than kWholeTiles tiles (short tables, or a window)
  // units are not cut: a merge takes as long as about four tiles.
  constexpr int64_t kWholeTiles = 8;
  const int64_t S = (int64_t)g.max_blocks * g.k_per_block;
  int64_t most = (S + L.tile - 1) / L.tile;
  if (g.window > 0) {
    const int64_t span = (int64_t)g.window + (L.R - 1) / g.H + 1;
    const int64_t w = span / L.tile + 2 + ((int64_t)g.first + L.tile - 1) / L.tile;
    if (w < most) most = w;
  }
  L.mode = kPlanned;
  if (g.B <= kFusedSeqs) {
    if (most <= kWholeTiles) L.mode = kWhole;
    else if (rows / L.R + g.B <= kFusedUnits) L.mode = kCut;
  }
  size_t off = kErrorWords + kErrorBytes;
  L.start_off = off;
  off = align256(off + (size_t)(L.grid + 1) * sizeof(ChunkStart));
  L.rec_off = off;
  off = align256(off + (size_t)L.grid * sizeof(ChunkUnit));
  L.seq_off = off;
  off = align256(off + (size_t)(g.B + 1) * 4);
  L.ml_off = off;
  off = align256(off + (size_t)2 * L.grid * L.R * 8);
  L.o_off = off;
  off = align256(off + (size_t)2 * L.grid * L.R * g.D * 4);
  L.total = off;
  return L;
}

cudaError_t launch_chunk_plan(const ChunkGeom& g, const ChunkLayout& L, void* ws, cudaStream_t st) {
  if (L.mode != kPlanned) return cudaSuccess;
  char* base = static_cast<char*>(ws);
  return launch_pdl(chunk_plan_kernel, dim3(1), dim3(kPlanThreads), 0, st, g, L.R, L.tile, L.grid,
                    reinterpret_cast<ChunkHeader*>(base),
                    reinterpret_cast<ChunkStart*>(base + L.start_off),
                    reinterpret_cast<ChunkUnit*>(base + L.rec_off),
                    reinterpret_cast<int*>(base + L.seq_off));
}

cudaError_t launch_paged_error(const void* ws, int32_t* error, cudaStream_t st) {
  paged_error_kernel<<<1, 32, 0, st>>>(static_cast<const ChunkHeader*>(ws), error);
  return cudaGetLastError();
}

cudaError_t launch_chunk_combine(const float* attn_sink, const ChunkGeom& g, void* out, float* lse,
                                 const ChunkLayout& L, void* ws, cudaStream_t st) {
  char* base = static_cast<char*>(ws);
  if (L.grid < 2 || L.mode == kWhole) return cudaSuccess;
  auto go = [&](auto kernel, int rows) {
    return launch_pdl(kernel, dim3(L.grid - 1, L.R / rows), dim3(kCombineWarps * 32), 0,
                      st, attn_sink, g.H, L.R, static_cast<__nv_bfloat16*>(out), lse,
                      L.grid, reinterpret_cast<const ChunkUnit*>(base + L.rec_off),
                      reinterpret_cast<const float2*>(base + L.ml_off),
                      reinterpret_cast<const float*>(base + L.o_off));
  };
  switch (g.D) {
    case 64: return go(chunk_combine_kernel<64, kPiecesOne>, CombineCfg<64>::kRows);
    case 128: return go(chunk_combine_kernel<128, kPiecesOne>, CombineCfg<128>::kRows);
    case 256:
      return L.pair ? go(chunk_combine_kernel<256, kPiecesPair>, CombineCfg<256>::kRows)
                    : go(chunk_combine_kernel<256, kPiecesOne>, CombineCfg<256>::kRows);
    case 512:
      return L.pair ? go(chunk_combine_kernel<512, kPiecesPair>, CombineCfg<512>::kRows)
                    : go(chunk_combine_kernel<512, kPiecesOne>, CombineCfg<512>::kRows);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace sda
