// sda_spread.cu -- chunk attention over a cache of E4M3 codes for sequences of many units.
//
// A prompt's rows are read by many units of 128 rows of q (2048 tokens of 64 heads: 1024),
// and converting the codes in each of them costs the attention kernel more than the whole
// cache is worth: eight warps beside the softmax, 2 instructions a code.  So one kernel
// converts every sequence's rows that any of its tokens sees once, to bf16 (exactly: codes
// without their scale), side by side in the workspace, and leaves a scale for each
// position; sda_chunk_pair.cu's kernel, which scales scores and weights, does the rest on
// tables of one block a sequence.
// 2048 tokens of 64 heads over 8192 positions, replayed: 1.31 ms against 1.60 without; 12
// prompts of 150 tokens over 3000 positions 527 us against 752, 4 of 850 tokens 839 against 1196.
#include <cuda_bf16.h>

#include <algorithm>

#include "sda_chunk_fp8.cuh"

namespace sda {

namespace {

constexpr int kTile = 64;  // positions of a tile of the attention kernel
constexpr int kCtaRows = 64;

struct SpreadParams {
  ChunkGeom g;
  const uint8_t* codes;
  const float* scale;
  __nv_bfloat16* rows;  // [B, S, D]
  float* pos_scale;     // [B, S]
  int* bad;             // a flag a CTA
  int32_t* table;       // [B]
  int S, k_shift;
  uint32_t k_mul;
};

// Tiles are read whole, so what lies between the last row and the end of its tile is zeros.
// A warp takes 8 rows.  What bounds it: a read and two writes of L2 a code, 12.6 MB for
// the prompt above.
template <int D>
__global__ void __launch_bounds__(256) spread_kernel(const SpreadParams p) {
  constexpr int kL = D / 16, kPer = 32 / kL;  // lanes a row, rows a load
  const ChunkGeom& g = p.g;
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  const bool lens = !lengths_bad(g, b);  // (the attention kernel refuses them)
  const int n = lens ? __ldg(g.kv_len + b) : 0;
  const int m = lens ? __ldg(g.q_indptr + b + 1) - __ldg(g.q_indptr + b) : 0;
  const int j0 = (int)blockIdx.x * kCtaRows + (int)(threadIdx.x >> 5) * 8;
  // Positions that some token sees: from `lo` on, and those below `first`; tiles that hold
  // any: below `front`, and from lo's on.  (Rows that see nothing have a tile of their own.)
  const int lo = g.window > 0 ? (int)max((long long)n - m - g.window + 1, 0ll) : 0;
  const int lot = lo / kTile * kTile, front = (min(g.first, lot) + kTile - 1) / kTile * kTile;
  const bool live = m > 0 && j0 < max((n + kTile - 1) / kTile, 1) * kTile && (j0 < front || j0 >= lot);
  int bad = 0;
  if (live) {
    int row = -1;  // lane i < 8: of position j0 + i
    float sc = 0.f;
    const int j = j0 + lane;
    if (lane < 8 && j < n && (j >= lo || j < g.first)) {
      const int jb = (int)(((unsigned long long)(unsigned)j * p.k_mul) >> p.k_shift);
      const int blk = __ldg(g.block_table + (size_t)b * g.max_blocks + jb);
      const long long r = g.base + (long long)blk * g.k_per_block + (j - jb * g.k_per_block);
      if (blk < 0 || r >= g.total_pages) {
        bad = 1;
      } else {
        row = (int)r;
        sc = __ldg(p.scale + blk);
      }
    }
    const size_t at = (size_t)b * p.S + j0;
    if (lane < 8) p.pos_scale[at + lane] = sc;
    uint4 x[8 / kPer];
#pragma unroll
    for (int i = 0; i < 8 / kPer; ++i) {
      const int from = __shfl_sync(0xffffffffu, row, i * kPer + lane / kL);
      x[i] = make_uint4(0, 0, 0, 0);
      if (from >= 0) x[i] = load_codes(p.codes + (size_t)from * D + lane % kL * 16);
    }
#pragma unroll
    for (int i = 0; i < 8 / kPer; ++i) {
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
      uint32_t h[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t f[2];
        codes_to_f16(w[e], f[0], f[1]);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&f[k]));
          const __nv_bfloat162 r = __floats2bfloat162_rn(v.x, v.y);
          h[2 * e + k] = *reinterpret_cast<const uint32_t*>(&r);
        }
      }
      uint4* to = reinterpret_cast<uint4*>(p.rows + (at + i * kPer + lane / kL) * D + lane % kL * 16);
      to[0] = make_uint4(h[0], h[1], h[2], h[3]);
      to[1] = make_uint4(h[4], h[5], h[6], h[7]);
    }
  }
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) {
    p.bad[blockIdx.y * gridDim.x + blockIdx.x] = bad;
    if (blockIdx.x == 0) p.table[b] = b;
  }
}

}  // namespace

SpreadLayout spread_layout(const ChunkGeom& g, int num_sms, size_t from) {
  SpreadLayout L;
  const int64_t rows = (int64_t)g.T * g.H;
  const int64_t S = ((int64_t)g.max_blocks * g.k_per_block + kCtaRows - 1) / kCtaRows * kCtaRows;
  // Worth it from four units of 128 rows a sequence on (16 sequences of 3000 positions at
  // D = 512: 85.8 us against 84.4 without at 512 rows, 104.9 against 110.0 at 768; 4 of 8000
  // at 512 rows 59.4 against 64.1; 32 of 2500 at 256 rows 92.2 against 83.0), and wherever
  // pairs work if the pair kernel would load the rows one by one (256 rows: 95.4 against
  // 112.7).  At most 2 GB, as tables may be much wider than their sequences.
  const int64_t least = g.k_per_block % 16 == 0 ? 512 : 129;
  L.worth = g.D >= 256 && rows >= least * g.B && S > 0 && S <= kMaxLen && g.B <= 65535 &&
            g.B * S <= ((int64_t)2 << 30) / (2 * g.D + 8);
  if (!L.worth) {
    L.total = from;
    return L;
  }
  L.S = (int)S;
  L.n_bad = (int)(g.B * S / kCtaRows);
  L.rows_off = align256(from);
  L.scale_off = align256(L.rows_off + (size_t)(g.B * S) * g.D * 2);
  L.bad_off = align256(L.scale_off + (size_t)(g.B * S) * 4);
  L.table_off = align256(L.bad_off + (size_t)L.n_bad * 4);
  L.total = align256(L.table_off + (size_t)g.B * 4);
  return L;
}

ChunkGeom spread_geometry(const ChunkGeom& g, const SpreadLayout& L, void* ws) {
  ChunkGeom s = g;
  s.block_table = reinterpret_cast<const int32_t*>(static_cast<char*>(ws) + L.table_off);
  s.max_blocks = 1;
  s.k_per_block = L.S;
  s.spare = (int)(L.S - (int64_t)g.max_blocks * g.k_per_block);
  s.base = 0;
  s.total_pages = (int64_t)g.B * L.S;
  return s;
}

cudaError_t launch_spread(const ChunkGeom& g, const void* codes, const float* scale, const SpreadLayout& L,
                          void* ws, cudaStream_t st) {
  char* const w = static_cast<char*>(ws);
  SpreadParams p{g, static_cast<const uint8_t*>(codes), scale,
                 reinterpret_cast<__nv_bfloat16*>(w + L.rows_off), reinterpret_cast<float*>(w + L.scale_off),
                 reinterpret_cast<int*>(w + L.bad_off), reinterpret_cast<int32_t*>(w + L.table_off), L.S, 0, 0};
  division(g.k_per_block, &p.k_mul, &p.k_shift);
  const dim3 grid((unsigned)(L.S / kCtaRows), (unsigned)g.B);
  return g.D == 256 ? launch_pdl(spread_kernel<256>, grid, dim3(256), 0, st, (const SpreadParams&)p)
                    : launch_pdl(spread_kernel<512>, grid, dim3(256), 0, st, (const SpreadParams&)p);
}

cudaError_t launch_chunk_spread(const void* q, const ChunkGeom& s, const float* attn_sink, float softmax_scale,
                                void* out, float* lse, const ChunkLayout& C, const SpreadLayout& L, void* ws,
                                cudaStream_t st) {
  if (!C.pair) return cudaErrorInvalidValue;  // (more than 128 rows a sequence: spread_layout's rule is above that)
  char* const w = static_cast<char*>(ws);
  ChunkParams p = chunk_params(w + L.rows_off, s, attn_sink, softmax_scale, out, lse, C, ws);
  p.bad = reinterpret_cast<const int*>(w + L.bad_off);
  p.n_bad = L.n_bad;
  CUtensorMap tq, tkv, ts;
  if (!pipe_map_2d(&tq, q, s.D, (uint64_t)s.T * s.H, 64, C.R / 2) ||
      !pipe_map_pool(&tkv, p.kv, s.D, (uint64_t)s.total_pages / 8, s.D / 128, 2) ||
      !pipe_map_f32(&ts, w + L.scale_off, L.S, s.B, kTile))
    return cudaErrorInvalidValue;
  return launch_chunk_pair_scaled(tq, tkv, ts, p, C, st);
}

}  // namespace sda
