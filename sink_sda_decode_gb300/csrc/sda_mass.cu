// sda_mass.cu -- attention mass: the weight that every cached position
// received from the new tokens, summed over tokens and heads and added to
// what it had (tcgen05 / TMEM).
//
//   out_j = decay prev_j + sum over rows (token, head) that see j of
//           e^(scale <q, kv_j> - lse)
//
// with each row's lse from the chunk attention (sink included), so one
// product S^T = K Q^T and no second pass over a row.  With positions on the
// TMEM lanes the sum over rows is a sum within a thread, in a fixed order.
//
// Two kernels.  mass_kernel, for chunks: pairs of CTAs (cta_group::2) take units of
// 256 positions, 128 in the shared memory of each CTA, and the q rows that see any
// of them, cut into tiles of 256 rows and streamed as 64-column panels, of which
// each CTA loads 128 rows.  (M256 N256 K16 runs at the tensor pipe's full rate,
// and a CTA's panels come in at 32 bytes a cycle; with one CTA to 128
// positions and 128 rows they came at 64, the limit of a SM's loads.)  All (unit, row
// tile) pairs form one sequence, cut into equal ranges, one per pair; a unit that a
// range boundary cuts leaves its partial sums per piece, which a last kernel adds up
// in order.
//   warps 0..15   epilogue: warp w reads TMEM lane quadrant w % 4 (positions)
//                 and quarter w / 4 of the row tile's columns
//   warps 16..23  the unit's cached rows, 16-byte cp.async
//   warp 24       q panels by TMA;  warp 25: the MMAs (CTA 0, for both)
// mass_step_kernel, for steps of few rows: see there.
//
// Measured, 2 sequences of 500 to 600 tokens over 6000 to 8192 positions, 64 heads,
// D = 512 (542 GFLOP): 285 to 328 us, 1900 to 1650 TFLOP/s between runs, the tensor
// pipe active 94 % of the cycles.  One CTA to 128 positions took 744 us; pairs
// with 8 epilogue warps 488 (the weights set the pace), with 16 warps 396, and with a
// range of rows per position in place of masks tested per weight 287.
#include <cuda_bf16.h>

#include "sda_chunk_dev.cuh"

namespace sda {

namespace {

using namespace ptx;

constexpr int kKeys = 256;                // positions per unit, 128 a CTA
constexpr int kRowsQ = 256;               // q rows per tile, 128 loaded by each CTA
constexpr int kPanelB = 128 * 128;        // bytes of a panel: 128 rows x 64 columns
constexpr int kEpWarps = 16, kEpThreads = 512;
constexpr int kLoadWarp0 = 16, kLoadWarps = 8;
constexpr int kStepThreads = 256;         // of mass_step_kernel's sums
constexpr int kQWarp = 24, kMmaWarp = 25;
constexpr int kThreads = 832;
constexpr int kPlanThreads = 1024;
constexpr int kSmemUnits = 8192, kSmemSeqs = 2048;

struct alignas(16) MassUnit {
  int b;      // sequence
  int k0;     // first position
  int row0;   // first q row (token * H) that sees any of the positions
  int nrows;  // rows from there to the last that does (0: none)
  int pos0;   // position of row 0's token; row r: token pos0 + r / H
  int n;      // positions from n on do not exist
  int nq;     // row tiles
  int cum;    // row tiles of all earlier units
};
static_assert(sizeof(MassUnit) == 32, "two 16-byte words");

// Rows (token, head) stand in the order of their tokens' positions, so those that see
// position j are a range.  Of the rows [0, nr) of a tile whose row 0 is row r0 of a
// stretch that starts at position pos0: [lo, hi).
struct RowRange {
  int lo, hi;
};
__device__ __forceinline__ RowRange rows_that_see(int j, int n, int pos0, int r0, int nr, int H,
                                                  int window, int first) {
  const long long a = ((long long)j - pos0) * H - r0;           // first row at j or behind
  const long long z = ((long long)j - pos0 + window) * H - r0;  // first row that j has left behind
  RowRange r;
  r.lo = (int)max(0ll, min(a, (long long)nr));
  r.hi = j >= n ? 0 : (window == 0 || j < first ? nr : (int)max(0ll, min(z, (long long)nr)));
  return r;
}

enum Bar : int { kKFull = 0, kKEmpty, kAccFull0, kAccEmpty0 = kAccFull0 + 2, kQFull0 = kAccEmpty0 + 2 };

template <int D>
struct Cfg {
  static constexpr int kPanels = D / 64;
  static constexpr int kRing = D == 512 ? 5 : 8;  // q panels in flight
  static constexpr int kOffK = 0;
  static constexpr int kOffQ = kPanels * kPanelB;
  static constexpr int kOffCol = kOffQ + kRing * kPanelB;  // per row tile: lse2 float[256]; two of them
  static constexpr int kOffPart = kOffCol + 2 * 1024;      // float [3][128]: the other column quarters' sums
  static constexpr int kOffBar = kOffPart + 1536;
  static constexpr int kOffMisc = kOffBar + 256;
  static constexpr int kSmem = kOffMisc + 16 + 1024;
  static constexpr uint32_t kIdesc = idesc_bf16_f32(kKeys, kRowsQ, false, false);
  static_assert((kQFull0 + 2 * kRing) * 8 <= 256, "mbarrier area");
  static_assert(kSmem <= 232448, "shared memory budget");
};

struct Params {
  const __nv_bfloat16* kv;
  const float* lse;
  float* out;
  ChunkHeader* hdr;
  const MassUnit* units;
  const int* cta_unit;
  float* part;
  ChunkGeom g;
  int64_t S;
  float qk_scale_log2;
  uint64_t wait_timeout_ns;
};

// CTA 0 plans; the others write out = decay * prev (0 behind kv_len).
__global__ void __launch_bounds__(kPlanThreads) mass_plan_kernel(
    const ChunkGeom g, int64_t S, int grid, int u_max, const float* prev, float decay, float* out,
    ChunkHeader* __restrict__ hdr, MassUnit* __restrict__ units, int* __restrict__ seq_unit,
    int* __restrict__ cta_unit) {
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  if (blockIdx.x > 0) {
    const int64_t total = (int64_t)g.B * S, step = (int64_t)(gridDim.x - 1) * kPlanThreads;
    for (int64_t e = (int64_t)(blockIdx.x - 1) * kPlanThreads + tid; e < total; e += step) {
      const int b = (int)(e / S);
      const int64_t j = e - (int64_t)b * S;
      out[e] = j < g.kv_len[b] && prev ? decay * prev[e] : 0.f;
    }
    return;
  }
  __shared__ long long warp_sums[32];
  __shared__ long long s_total;
  __shared__ int s_cum[kSmemUnits];
  __shared__ int s_seq[kSmemSeqs];
  int bad = 0;
  long long U = 0;
  for (int b0 = 0; b0 < g.B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    long long nu = 0;
    if (b < g.B) {
      const int q0 = g.q_indptr[b], q1 = g.q_indptr[b + 1], n = g.kv_len[b];
      if (q0 < 0 || q1 < q0 || q1 > g.T || n < 0 || n > S) bad = 1;
      else if (q1 > q0) nu = ((long long)n + kKeys - 1) / kKeys;
    }
    const long long ex = scan_exclusive(nu, warp_sums, &s_total);
    const long long tot = s_total;
    if (b < g.B) {
      const int v = (int)min(U + ex, (long long)u_max);
      if (b < kSmemSeqs) s_seq[b] = v;
      seq_unit[b] = v;
    }
    U += tot;
    __syncthreads();
  }
  if (U > u_max) bad = 1;
  bad = __syncthreads_or(bad);
  const int nu = bad ? 0 : (int)U;
  const int* seq = g.B <= kSmemSeqs ? s_seq : seq_unit;
  long long tt = 0;
  for (int u0 = 0; u0 < nu; u0 += kPlanThreads) {
    const int u = u0 + tid;
    MassUnit d = {};
    if (u < nu) {
      const int b = last_le(seq, g.B, u);
      const int q0 = g.q_indptr[b], m = g.q_indptr[b + 1] - q0, n = g.kv_len[b];
      d.b = b;
      d.n = n;
      d.k0 = (u - seq[b]) * kKeys;
      const int k1 = min(d.k0 + kKeys, n);
      // tokens at positions [k0, ...) see the tile; with a window only those
      // below its last position + window, unless it holds first positions
      const int p0 = n - m;
      const int ta = max(0, d.k0 - p0);
      long long tb = m;
      if (g.window > 0 && d.k0 >= g.first) tb = min(tb, (long long)k1 - 1 + g.window - p0);
      const long long rows = tb > ta ? (tb - ta) * g.H : 0;
      d.row0 = (q0 + ta) * g.H;
      d.nrows = (int)rows;
      d.pos0 = p0 + ta;
      d.nq = (int)((rows + kRowsQ - 1) / kRowsQ);
    }
    const long long ex = scan_exclusive(d.nq, warp_sums, &s_total);
    const long long tot = s_total;
    if (u < nu) {
      d.cum = (int)min(tt + ex, 0x7fffffffll);
      units[u] = d;
      if (u < kSmemUnits) s_cum[u] = d.cum;
    }
    tt += tot;
    __syncthreads();
  }
  if (tt > 0x7fffffffll) bad = 1;
  const int TT = bad ? 0 : (int)tt;
  const int per = TT > 0 ? (int)((TT + (long long)grid - 1) / grid) : 1;
  for (int k = tid; k <= grid; k += kPlanThreads) {
    const long long t = (long long)k * per;
    int u = nu;
    if (t < TT) {
      if (nu <= kSmemUnits) {
        u = last_le(s_cum, nu, (int)t);
      } else {
        int lo = 0, hi = nu;
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (units[mid].cum <= t) lo = mid;
          else hi = mid;
        }
        u = lo;
      }
    }
    cta_unit[k] = u;
  }
  if (tid == 0) {
    hdr->n_units = nu;
    hdr->n_tiles = TT;
    hdr->per = per;
    hdr->ctas = (TT + per - 1) / per;
    hdr->error = bad ? 2 : 0;
    hdr->words = 0;  // (the next kernel's)
  }
}

__device__ __forceinline__ MassUnit load_unit(const MassUnit* u) {
  const int4 a = __ldcg(reinterpret_cast<const int4*>(u));
  const int4 b = __ldcg(reinterpret_cast<const int4*>(u) + 1);
  return MassUnit{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
}

// A CTA's piece of a unit: row tiles [i0, i1).  Pieces come in the plan's
// order; units without rows are passed over.
struct Piece {
  MassUnit un;
  int i0, i1;
};
struct PieceWalk {
  const MassUnit* units;
  int u, t, t1;
  __device__ __forceinline__ bool next(Piece* p) {
    if (t >= t1) return false;
    do {
      p->un = load_unit(units + u);
      ++u;
    } while (p->un.cum + p->un.nq <= t);
    p->i0 = t - p->un.cum;
    p->i1 = min(p->un.nq, t1 - p->un.cum);
    t = p->un.cum + p->i1;
    return true;
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
mass_kernel(const __grid_constant__ CUtensorMap tmap_q, const Params p) {
  using C = Cfg<D>;
  constexpr int NP = C::kPanels;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_addr(smem);
  const uint32_t sK = sbase + C::kOffK, sQ = sbase + C::kOffQ;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  auto bar = [&](int i) { return sbase + C::kOffBar + 8u * (uint32_t)i; };
  auto q_full = [&](int i) { return bar(kQFull0 + 2 * i); };
  auto q_empty = [&](int i) { return bar(kQFull0 + 2 * i + 1); };
  auto bar0 = [&](int i) { return map_cta(bar(i), 0); };  // of the pair's CTA 0
  const int rank = (int)(blockIdx.x & 1), worker = (int)(blockIdx.x >> 1);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(bar(kKFull), 2 * kLoadWarps);  // CTA 0: the loaders of both
    mbar_init(bar(kKEmpty), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kAccFull0 + i), 1);
      mbar_init(bar(kAccEmpty0 + i), 2 * kEpWarps);  // CTA 0: the epilogues of both
    }
    for (int i = 0; i < C::kRing; ++i) {
      mbar_init(q_full(i), 1);
      mbar_init(q_empty(i), 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmap_q);
  }
  if (warp == kMmaWarp) {
    tmem_alloc_pair(smem_addr(tmem_slot), 512);
  }
  tc_fence_before();
  __syncwarp();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_trigger();
  const int per = __ldcg(&p.hdr->per), n_tiles = __ldcg(&p.hdr->n_tiles);
  const int t0 = (int)min((long long)worker * per, (long long)n_tiles);
  const int t1 = (int)min((long long)(worker + 1) * per, (long long)n_tiles);
  PieceWalk walk{p.units, t0 < t1 ? __ldcg(p.cta_unit + worker) : 0, t0, t1};
  int* const error = reinterpret_cast<int*>(reinterpret_cast<char*>(p.hdr) + kErrorWords) + blockIdx.x;
  if (threadIdx.x == 0) {
    *error = 0;
    if (blockIdx.x == 0) p.hdr->words = gridDim.x;
  }
  __syncthreads();
  const PipeWait wc{abort_flag, error, p.wait_timeout_ns};
  Piece pc;

  if (warp >= kLoadWarp0 && warp < kLoadWarp0 + kLoadWarps) {
    // ===================================================== the unit's cached rows
    constexpr int kRows = 128 / kLoadWarps;  // 16 rows per warp: two swizzle atoms
    constexpr int kCh = D / 8 < 32 ? D / 8 : 32;
    constexpr int kRowsPer = 32 / kCh;
    const int v = warp - kLoadWarp0;
    const uint4* kv4 = reinterpret_cast<const uint4*>(p.kv);
    bool ok = true;
    int x = 0;
    for (; ok && walk.next(&pc); ++x) {
      int sl = -1;
      const int j = pc.un.k0 + rank * 128 + v * kRows + lane;
      if (lane < kRows && j < pc.un.n) {
        const int blk = __ldg(p.g.block_table + (size_t)pc.un.b * p.g.max_blocks + j / p.g.k_per_block);
        const long long s = p.g.base + (long long)blk * p.g.k_per_block + j % p.g.k_per_block;
        if (blk < 0 || s >= p.g.total_pages) atomicExch(error, 3);
        else sl = (int)s;
      }
      if (x > 0) {
        ok = warp_wait(bar(kKEmpty), (x - 1) & 1, wc);
        if (!ok) break;
      }
#pragma unroll
      for (int r0 = 0; r0 < kRows; r0 += kRowsPer) {
        const int r = r0 + lane / kCh;
        const int slot = __shfl_sync(0xffffffffu, sl, r);
#pragma unroll
        for (int c0 = 0; c0 < D / 8; c0 += kCh) {
          const int ch = c0 + lane % kCh;
          const uint4* src = slot >= 0 ? kv4 + (size_t)slot * (D / 8) + ch : kv4;
          cp_async16(sK + (ch >> 3) * kPanelB + (2 * v + (r >> 3)) * 1024 + (r & 7) * 128 +
                         (((ch & 7) ^ (r & 7)) << 4),
                     src, slot >= 0 ? 16u : 0u);
        }
      }
      cp_async_commit();
      cp_async_wait_group<0>();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) arrive_cluster(bar0(kKFull));
    }
    // (the last arrival comes in before this CTA's memory goes away)
    if (ok && x > 0) pipe_drain(bar(kKEmpty), (x - 1) & 1, wc);
  } else if (warp == kQWarp) {
    // ===================================================== q panels
    int f = 0;  // panels issued
    bool ok = true;
    while (ok && walk.next(&pc)) {
      for (int i = pc.i0; i < pc.i1 && ok; ++i) {
        for (int x = 0; x < NP; ++x, ++f) {
          const int s = f % C::kRing;
          if (f >= C::kRing) ok = warp_wait(q_empty(s), ((f / C::kRing) - 1) & 1, wc);
          if (!ok) break;
          if (elect_one()) {
            if (rank == 0) mbar_arrive_expect_tx(q_full(s), 2 * kPanelB);
            tma_pair_2d(sQ + s * kPanelB, &tmap_q, x * 64, pc.un.row0 + i * kRowsQ + rank * 128,
                        map_cta(q_full(s), 0));
          }
          __syncwarp();
        }
      }
    }
    // every panel has been read (so it has landed) before the CTA's memory goes away
    for (int x = max(0, f - C::kRing); x < f; ++x)
      pipe_drain(q_empty(x % C::kRing), (x / C::kRing) & 1, wc);
  } else if (warp == kMmaWarp) {
    // ===================================================== MMAs
    if (rank == 0) {
      int f = 0, g = 0;
      bool ok = true;
      const uint64_t a0 = sdesc_sw128(sK, 16, 1024);
      for (int x = 0; ok && walk.next(&pc); ++x) {
        ok = warp_wait(bar(kKFull), x & 1, wc);
        for (int i = pc.i0; i < pc.i1 && ok; ++i, ++g) {
          const int s = g & 1;
          if (g >= 2) ok = warp_wait(bar(kAccEmpty0 + s), ((g >> 1) - 1) & 1, wc);
          for (int y = 0; y < NP && ok; ++y, ++f) {
            const int r = f % C::kRing;
            ok = warp_wait(q_full(r), (f / C::kRing) & 1, wc);
            if (!ok) break;
            fence_proxy_async_smem();  // the cached rows were copied through the generic proxy
            tc_fence_after();
            const uint64_t b0 = sdesc_sw128(sQ + r * kPanelB, 16, 1024);
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_pair(tmem + s * 256, sdesc_advance(a0, y * kPanelB + k * 32),
                         sdesc_advance(b0, k * 32), C::kIdesc, (y || k) ? 1u : 0u);
              commit_pair(q_empty(r));
              if (y == NP - 1) {
                commit_pair(bar(kAccFull0 + s));
                if (i == pc.i1 - 1) commit_pair(bar(kKEmpty));
              }
            }
            __syncwarp();
          }
        }
      }
    }
  } else if (warp < kEpWarps) {
    // ===================================================== weights and sums
    const int q4 = warp & 3, hc = warp >> 2, st = threadIdx.x;
    const uint32_t lane_base = (uint32_t)(q4 * 32) << 16;
    float* s_part = reinterpret_cast<float*>(smem + C::kOffPart);
    const float sc = p.qk_scale_log2;
    const int H = p.g.H, window = p.g.window, nfirst = p.g.first;
    int g = 0;
    while (walk.next(&pc)) {
      const MassUnit& un = pc.un;
      const int j = un.k0 + rank * 128 + q4 * 32 + lane;  // this thread's position
      float sum = 0.f, comp = 0.f;
      auto lse_of = [&](int i) {  // of this thread's column of row tile i
        const int r = i * kRowsQ + st;
        return st < kRowsQ && r < un.nrows ? __ldg(p.lse + un.row0 + r) * kLog2e : 0.f;
      };
      float lse_next = lse_of(pc.i0);
      for (int i = pc.i0; i < pc.i1; ++i, ++g) {
        const int s = g & 1;
        float* lse2 = reinterpret_cast<float*>(smem + C::kOffCol + s * 1024);
        const int r0 = i * kRowsQ, nr = min(kRowsQ, un.nrows - r0);
        if (st < kRowsQ) lse2[st] = lse_next;
        if (i + 1 < pc.i1) lse_next = lse_of(i + 1);
        const RowRange rr = rows_that_see(j, un.n, un.pos0, r0, nr, H, window, nfirst);
        named_bar_sync(1, kEpThreads);  // (also: everyone is past the tile that used this array)
        warp_wait(bar(kAccFull0 + s), (g >> 1) & 1, wc);
        tc_fence_after();
        float part = 0.f;
        // 16 rows at a time; masks only where a lane needs them
#pragma unroll 1
        for (int c0 = hc * 64; c0 < hc * 64 + 64; c0 += 16) {
          if (!__any_sync(0xffffffffu, rr.lo < c0 + 16 && rr.hi > c0 && rr.lo < rr.hi)) continue;
          uint32_t v[16];
          tmem_ld16(tmem + lane_base + s * 256 + c0, v);
          tmem_wait_ld();
          float a[4] = {0.f, 0.f, 0.f, 0.f};
          if (__all_sync(0xffffffffu, rr.lo <= c0 && rr.hi >= c0 + 16)) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
              a[e & 3] += ex2_approx(fmaf(__uint_as_float(v[e]), sc, -lse2[c0 + e]));
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float w = ex2_approx(fmaf(__uint_as_float(v[e]), sc, -lse2[c0 + e]));
              a[e & 3] += c0 + e >= rr.lo && c0 + e < rr.hi ? w : 0.f;
            }
          }
          part += (a[0] + a[1]) + (a[2] + a[3]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_cluster(bar0(kAccEmpty0 + s));
        // compensated: a unit can have a million rows
        const float y = part - comp, t = sum + y;
        comp = (t - sum) - y;
        sum = t;
      }
      if (hc > 0) s_part[(hc - 1) * 128 + q4 * 32 + lane] = sum;
      named_bar_sync(1, kEpThreads);
      if (hc == 0) {
        const float* o = s_part + q4 * 32 + lane;
        sum = (sum + o[0]) + (o[128] + o[256]);
        if (pc.i0 == 0 && pc.i1 == un.nq) {
          if (j < un.n) p.out[(int64_t)un.b * p.S + j] += sum;
        } else {
          p.part[(size_t)(2 * worker + (pc.i0 == 0 ? 1 : 0)) * kKeys + rank * 128 + q4 * 32 + lane] = sum;
        }
      }
      named_bar_sync(1, kEpThreads);  // s_part may be rewritten
    }
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();  // neither CTA leaves while the other may still reach its memory
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc_pair(tmem, 512);
}

// Adds the pieces of cut units in order: block k - 1 acts if boundary k of
// the tile ranges is the first that cuts its unit (see the chunk combine).
__global__ void __launch_bounds__(kKeys) mass_combine_kernel(
    const ChunkHeader* __restrict__ hdr, const MassUnit* __restrict__ units,
    const int* __restrict__ cta_unit, const float* __restrict__ part, int64_t S,
    float* __restrict__ out) {
  pdl_wait();
  pdl_trigger();
  const int k = blockIdx.x + 1;
  if (k >= hdr->ctas) return;
  const int per = hdr->per;
  const MassUnit un = units[cta_unit[k]];
  const long long t0 = (long long)k * per;
  if (un.cum >= t0 || un.cum < t0 - per) return;
  const long long end = (long long)un.cum + un.nq;
  const int np = 1 + (int)((end - t0 + per - 1) / per);
  const int x = threadIdx.x;
  float sum = part[(size_t)(2 * (k - 1) + 1) * kKeys + x];
  for (int i = 1; i < np; ++i) sum += part[(size_t)(2 * (k - 1 + i)) * kKeys + x];
  if (un.k0 + x < un.n) out[(int64_t)un.b * S + un.k0 + x] += sum;
}

// ------------------------------------------------------------------ steps
// mass_step_kernel: sequences with few q rows (a step of one or a few tokens),
// where the cached rows' way from memory is what counts.  One launch, no plan:
// every CTA sums the sequences' tile counts itself and takes its equal, contiguous
// share of the tiles of 64 positions.  The q rows that see a tile (R at a time) stay
// in shared memory from tile to tile of a sequence; S^T = K Q^T with M = 64
// positions, N = R rows; the sums over the rows are final, so out is written at once.
// Measured: one token of 64 heads over 8 caches of 16384 to 65536 positions, D = 512
// (368 MB): 61 us, where a copy of as many bytes takes 55; the kernel for chunks took 131.
//   warps 0..7   weights and sums: warp w reads TMEM lane quadrant w % 4 (16
//                positions) and half w / 4 of the rows' columns
//   warp 8       MMAs, q loads      warp 9   cached rows by TMA (boxes of 16)
//   warps 10, 11 the columns of out that no tile covers
//   warps 12..19 (gather kernel) cached rows one by one, 16-byte cp.async
constexpr int kTileS = 64;
constexpr int kStepSeqs = 2048;  // sequences whose tile counts a CTA sums itself
constexpr int kSMma = 8, kSTma = 9, kSFill = 10, kSLoad0 = 12, kSLoads = 8;
enum StepBar : int {
  kSqFull = 0,
  kSqEmpty,
  kSAccFull0,
  kSAccEmpty0 = kSAccFull0 + 2,
  kSkFull0 = kSAccEmpty0 + 2,
  kSkFree0 = kSkFull0 + 6,
  kSDrain = kSkFree0 + 6,
  kSBars
};

template <int R, int D>
struct StepCfg {
  static constexpr int kPanels = D / 64, kHalves = D >= 256 ? 2 : 1, kPanelsH = kPanels / kHalves;
  static constexpr int kGroup = kPanelsH * 1024, kHalf = kTileS / 8 * kGroup;
  static constexpr int kStage = kHalves * kHalf, kBox = 2 * kGroup;
  static constexpr int kStages = D == 512 ? (R == 16 ? 3 : 2) : (D == 256 ? 4 : 6);
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kPanels * R * 128;
  static constexpr int kOffTiles = kOffK + kStages * kStage;       // int [kStepSeqs + 1]: tiles before sequence b
  static constexpr int kOffCol = kOffTiles + 4 * kStepSeqs + 16;   // lse2 float[64]
  static constexpr int kOffSum = kOffCol + 256;                    // float [2 tiles][64]
  static constexpr int kOffBar = kOffSum + 512;
  static constexpr int kOffMisc = kOffBar + 256;
  static constexpr int kSmem = kOffMisc + 160 + 1024;
  static constexpr uint32_t kIdesc = idesc_bf16_f32(64, R, false, false);
  static_assert(kSBars * 8 <= 256, "mbarrier area");
  static_assert(kSmem <= 232448, "shared memory budget");
};

struct StepParams {
  const __nv_bfloat16* kv;
  const float* lse;
  const float* prev;
  float* out;
  ChunkHeader* hdr;
  ChunkGeom g;
  int64_t S;
  float qk_scale_log2, decay;
  uint64_t wait_timeout_ns;
};

// A tile of positions and the q rows that see any of it.
struct StepTile {
  int b, n, k0;     // sequence, its cached positions, the tile's first
  int row0, nrows;  // q rows [row0, row0 + nrows)
  int pos0;         // position of row0's token
  __device__ __forceinline__ void set(const ChunkGeom& g, int seq, int kt) {
    b = seq;
    k0 = kt * kTileS;
    n = __ldg(g.kv_len + b);
    const int q0 = __ldg(g.q_indptr + b), m = __ldg(g.q_indptr + b + 1) - q0;
    const int p0 = n - m, ta = max(0, k0 - p0);
    long long tb = m;
    if (g.window > 0 && k0 >= g.first) tb = min(tb, (long long)min(k0 + kTileS, n) - 1 + g.window - p0);
    row0 = (q0 + ta) * g.H;
    nrows = tb > ta ? (int)((tb - ta) * g.H) : 0;
    pos0 = p0 + ta;
  }
};

template <int R, int D, bool TMA>
__global__ void __launch_bounds__(TMA ? 384 : 640, 1)
mass_step_kernel(const __grid_constant__ CUtensorMap tmap_q,
                 const __grid_constant__ CUtensorMap tmap_kv, const StepParams p) {
  using C = StepCfg<R, D>;
  constexpr int KS = C::kStages, kThr = TMA ? 384 : 640;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_addr(smem);
  const uint32_t sQ = sbase + C::kOffQ, sK = sbase + C::kOffK;
  int* s_tiles = reinterpret_cast<int*>(smem + C::kOffTiles);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  int* s_warp = reinterpret_cast<int*>(smem + C::kOffMisc + 16);  // [20]
  auto bar = [&](int i) { return sbase + C::kOffBar + 8u * (uint32_t)i; };
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int tid = threadIdx.x;
  if (tid == 0) {
    mbar_init(bar(kSqFull), 1);
    mbar_init(bar(kSqEmpty), 1);
    mbar_init(bar(kSDrain), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kSAccFull0 + i), 1);
      mbar_init(bar(kSAccEmpty0 + i), 8);
    }
    for (int i = 0; i < KS; ++i) {
      mbar_init(bar(kSkFull0 + i), TMA ? 1 : kSLoads * 32);
      mbar_init(bar(kSkFree0 + i), 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmap_q);
    if (TMA) tma_prefetch_desc(&tmap_kv);
  }
  if (warp == kSMma) {
    tmem_alloc(smem_addr(tmem_slot), 128);
    tmem_relinquish();
  }
  pdl_wait();
  pdl_trigger();
  const int B = p.g.B, H = p.g.H;
  // s_tiles[b] = tiles of the sequences before b; lengths that make no sense stop it
  int bad = 0;
  {
    const int each = (B + kThr - 1) / kThr, b0 = min(tid * each, B), b1 = min(b0 + each, B);
    auto tiles_of = [&](int b) {
      const int q0 = __ldg(p.g.q_indptr + b), q1 = __ldg(p.g.q_indptr + b + 1), n = __ldg(p.g.kv_len + b);
      if (q0 < 0 || q1 < q0 || q1 > p.g.T || n < 0 || n > p.S) {
        bad = 1;
        return 0;
      }
      return q1 > q0 ? (n + kTileS - 1) / kTileS : 0;
    };
    int mine = 0;
    for (int b = b0; b < b1; ++b) mine += tiles_of(b);
    int x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_warp[warp] = x;
    bad = __syncthreads_or(bad);
    int run = x - mine;
    for (int w = 0; w < warp; ++w) run += s_warp[w];
    for (int b = b0; b < b1; ++b) {
      s_tiles[b] = bad ? 0 : run;
      run += tiles_of(b);
    }
    if (b1 == B && (b0 < B || tid == 0)) s_tiles[B] = bad ? 0 : run;
  }
  int* const error = reinterpret_cast<int*>(reinterpret_cast<char*>(p.hdr) + kErrorWords) + blockIdx.x;
  if (tid == 0) {
    *error = 0;
    if (blockIdx.x == 0) {
      p.hdr->words = gridDim.x;
      p.hdr->error = bad ? 2 : 0;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int total = s_tiles[B], per = (total + gridDim.x - 1) / (int)gridDim.x;
  const int t0 = min((int)blockIdx.x * per, total), t1 = min(t0 + per, total);
  const PipeWait wc{abort_flag, error, p.wait_timeout_ns};
  const int b_first = t0 < t1 ? last_le(s_tiles, B, t0) : 0;
  // Calls f on every tile of this CTA that has rows or (all) on every tile.
  auto walk = [&](bool all, auto f) {
    int b = b_first;
    StepTile tl;
    for (int t = t0; t < t1; ++t) {
      while (t >= s_tiles[b + 1]) ++b;
      tl.set(p.g, b, t - s_tiles[b]);
      if (all || tl.nrows > 0)
        if (!f(tl)) break;
    }
  };

  if (TMA && warp == kSTma) {
    // ===================================================== cached rows by TMA
    const int behind = (int)((p.g.total_pages - p.g.base) / 8);
    int g = 0;
    walk(false, [&](const StepTile& tl) {
      const int s = g % KS;
      int y = behind;
      const int j = tl.k0 + lane * 16;
      if (lane < 4 && j < tl.n) {
        const int r = pool_row_of(p.g, error, tl.b, j);
        if (r >= 0) {
          y = (int)((r - p.g.base) / 8);
          if (ends_behind(p.g, y, j, tl.n - 1)) atomicExch(error, 3);
        }
      }
      if (g >= KS && !warp_wait(bar(kSkFree0 + s), ((g / KS) - 1) & 1, wc)) return false;
      if (lane == 0) mbar_arrive_expect_tx(bar(kSkFull0 + s), C::kStage);
      __syncwarp();
      if (lane < 4) {
#pragma unroll
        for (int h = 0; h < C::kHalves; ++h)
          tma_load_4d(sK + s * C::kStage + h * C::kHalf + lane * C::kBox, &tmap_kv, 0, 0,
                      h * C::kPanelsH, y, bar(kSkFull0 + s));
      }
      ++g;
      return true;
    });
    for (int x = max(0, g - KS); x < g; ++x) pipe_drain(bar(kSkFull0 + x % KS), (x / KS) & 1, wc);
  } else if (!TMA && warp >= kSLoad0) {
    // ===================================================== cached rows one by one
    constexpr int kCh = D / 8 < 32 ? D / 8 : 32, kRowsPer = 32 / kCh, kRows = kTileS / kSLoads;
    const int v = warp - kSLoad0;
    const uint4* kv4 = reinterpret_cast<const uint4*>(p.kv);
    int g = 0;
    walk(false, [&](const StepTile& tl) {
      const int s = g % KS;
      const int j = tl.k0 + v * kRows + lane;
      const int sl = lane < kRows && j < tl.n ? pool_row_of(p.g, error, tl.b, j) : -1;
      if (g >= KS && !warp_wait(bar(kSkFree0 + s), ((g / KS) - 1) & 1, wc)) return false;
#pragma unroll
      for (int r0 = 0; r0 < kRows; r0 += kRowsPer) {
        const int r = r0 + lane / kCh;  // row of this warp's group of 8
        const int slot = __shfl_sync(0xffffffffu, sl, r);
#pragma unroll
        for (int c0 = 0; c0 < D / 8; c0 += kCh) {
          const int ch = c0 + lane % kCh, pn = ch >> 3;
          const uint4* src = slot >= 0 ? kv4 + (size_t)slot * (D / 8) + ch : kv4;
          cp_async16(sK + s * C::kStage + pn / C::kPanelsH * C::kHalf + v * C::kGroup +
                         pn % C::kPanelsH * 1024 + r * 128 + (((ch & 7) ^ r) << 4),
                     src, slot >= 0 ? 16u : 0u);
        }
      }
      cp_async_arrive(bar(kSkFull0 + s));
      ++g;
      return true;
    });
    cp_async_wait_all();
  } else if (warp == kSMma) {
    // ===================================================== q loads, MMAs
    const uint64_t b0 = sdesc_sw128(sQ, 16, 1024);
    int g = 0, a = 0, q_row = -1, q_loads = 0;
    walk(false, [&](const StepTile& tl) {
      const int ks = g % KS;
      const uint64_t a0 = sdesc_sw128(sK + ks * C::kStage, 16, C::kGroup);
      for (int r0 = 0; r0 < tl.nrows; r0 += R, ++a) {
        const int s = a & 1;
        if (tl.row0 + r0 != q_row) {
          q_row = tl.row0 + r0;
          if (q_loads > 0) {  // the MMAs that read the rows before are done
            if (elect_one()) mma_commit(bar(kSqEmpty));
            __syncwarp();
            if (!warp_wait(bar(kSqEmpty), (q_loads - 1) & 1, wc)) return false;
          }
          if (elect_one()) {
            mbar_arrive_expect_tx(bar(kSqFull), C::kPanels * R * 128);
#pragma unroll
            for (int x = 0; x < C::kPanels; ++x)
              tma_load_2d(sQ + x * R * 128, &tmap_q, x * 64, q_row, bar(kSqFull));
          }
          __syncwarp();
          ++q_loads;
          if (!warp_wait(bar(kSqFull), (q_loads - 1) & 1, wc)) return false;
        }
        if (a >= 2 && !warp_wait(bar(kSAccEmpty0 + s), ((a >> 1) - 1) & 1, wc)) return false;
        if (r0 == 0 && !warp_wait(bar(kSkFull0 + ks), (g / KS) & 1, wc)) return false;
        if (!TMA) fence_proxy_async_smem();
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int pn = 0; pn < C::kPanels; ++pn) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_bf16(tmem + s * 64,
                       sdesc_advance(a0, pn / C::kPanelsH * C::kHalf + pn % C::kPanelsH * 1024 + k * 32),
                       sdesc_advance(b0, pn * R * 128 + k * 32), C::kIdesc, (pn || k) ? 1u : 0u);
          }
          mma_commit(bar(kSAccFull0 + s));
          if (r0 + R >= tl.nrows) mma_commit(bar(kSkFree0 + ks));
        }
        __syncwarp();
      }
      ++g;
      return true;
    });
    // MMAs are done and q has landed before TMEM and shared memory go away, also where a
    // wait gave up in the middle of a tile
    if (elect_one()) {
      mma_commit(bar(kSDrain));
      pipe_drain(bar(kSDrain), 0, wc);
      if (q_loads > 0) pipe_drain(bar(kSqFull), (q_loads - 1) & 1, wc);
    }
    __syncwarp();
  } else if (warp < 8) {
    // ===================================================== weights and sums
    // 16x256b: thread t holds positions hA = 16 q4 + t / 4 and hB = hA + 8 at the rows
    // 32 hc + 8 rep + 2 (t % 4) + {0, 1} (R = 16: hc = 0 alone, rep = 0, 1)
    constexpr int kReps = R == 16 ? 2 : 4;
    const int q4 = warp & 3, hc = warp >> 2, tq = lane & 3;
    const int hA = q4 * 16 + (lane >> 2), hB = hA + 8;
    float* lse2 = reinterpret_cast<float*>(smem + C::kOffCol);
    float* s_sum = reinterpret_cast<float*>(smem + C::kOffSum);
    const float sc = p.qk_scale_log2;
    const int window = p.g.window, nfirst = p.g.first;
    const bool work = R > 16 || hc == 0;
    int a = 0, have = -1, have_n = 0, x = 0;
    walk(true, [&](const StepTile& tl) {
      const int64_t at = (int64_t)tl.b * p.S + tl.k0;
      const int jA = tl.k0 + hA, jB = tl.k0 + hB;
      float before[2] = {0.f, 0.f};
      if (hc == 0 && tq == 0 && p.prev) {
        if (jA < tl.n) before[0] = p.prev[at + hA];
        if (jB < tl.n) before[1] = p.prev[at + hB];
      }
      float sumA = 0.f, sumB = 0.f, compA = 0.f, compB = 0.f;
      for (int r0 = 0; r0 < tl.nrows; r0 += R, ++a) {
        const int s = a & 1, nr = min(R, tl.nrows - r0);
        if (tl.row0 + r0 != have || nr > have_n) {  // these rows' lse
          have = tl.row0 + r0;
          have_n = nr;
          named_bar_sync(1, kStepThreads);
          if (tid < R) lse2[tid] = tid < nr ? __ldg(p.lse + have + tid) * kLog2e : 0.f;
          named_bar_sync(1, kStepThreads);
        }
        const RowRange ra = rows_that_see(jA, tl.n, tl.pos0, r0, nr, H, window, nfirst);
        const RowRange rb = rows_that_see(jB, tl.n, tl.pos0, r0, nr, H, window, nfirst);
        const bool full = __all_sync(0xffffffffu, ra.lo == 0 && ra.hi == R && rb.lo == 0 && rb.hi == R);
        warp_wait(bar(kSAccFull0 + s), (a >> 1) & 1, wc);
        tc_fence_after();
        if (work) {
          uint32_t v[4 * kReps];
          const uint32_t ta = tmem + ((uint32_t)(q4 * 32) << 16) + s * 64 + 32 * hc;
          if constexpr (R == 16) tmem_ld_16x256b_x2(ta, v);
          else tmem_ld_16x256b_x4(ta, v);
          tmem_wait_ld();
          float pA = 0.f, pB = 0.f;
#pragma unroll
          for (int rep = 0; rep < kReps; ++rep) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int c = 32 * hc + 8 * rep + 2 * tq + (k & 1);
              const float w = ex2_approx(fmaf(__uint_as_float(v[4 * rep + k]), sc, -lse2[c]));
              const bool see = full || (k < 2 ? c >= ra.lo && c < ra.hi : c >= rb.lo && c < rb.hi);
              (k < 2 ? pA : pB) += see ? w : 0.f;
            }
          }
          // compensated: a tile can have many row tiles
          float y = pA - compA, t = sumA + y;
          compA = (t - sumA) - y;
          sumA = t;
          y = pB - compB, t = sumB + y;
          compB = (t - sumB) - y;
          sumB = t;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kSAccEmpty0 + s));
      }
      sumA += __shfl_xor_sync(0xffffffffu, sumA, 1);
      sumA += __shfl_xor_sync(0xffffffffu, sumA, 2);
      sumB += __shfl_xor_sync(0xffffffffu, sumB, 1);
      sumB += __shfl_xor_sync(0xffffffffu, sumB, 2);
      float* half = s_sum + (x & 1) * 64;
      ++x;
      if constexpr (R > 16) {
        if (hc == 1 && tq == 0) {
          half[hA] = sumA;
          half[hB] = sumB;
        }
        named_bar_sync(1, kStepThreads);
      }
      if (hc == 0 && tq == 0) {
        if constexpr (R > 16) {
          sumA += half[hA];
          sumB += half[hB];
        }
        if (jA < tl.n) p.out[at + hA] = fmaf(p.decay, before[0], sumA);
        if (jB < tl.n) p.out[at + hB] = fmaf(p.decay, before[1], sumB);
      }
      return true;
    });
  } else if (warp == kSFill || warp == kSFill + 1) {
    // ===================================================== what no tile covers
    constexpr int kCols = 1024;
    const int chunks = (int)((p.S + kCols - 1) / kCols);
    for (long long x = (long long)blockIdx.x * 2 + (warp - kSFill); x < (long long)B * chunks;
         x += 2 * gridDim.x) {
      const int b = (int)(x / chunks), c0 = (int)(x % chunks) * kCols;
      const int n = __ldg(p.g.kv_len + b);
      const int from = max(c0, s_tiles[b + 1] > s_tiles[b] ? n : 0);
      const int to = (int)min((int64_t)c0 + kCols, p.S);
      const int64_t row = (int64_t)b * p.S;
      for (int j = from + lane; j < to; j += 32)
        p.out[row + j] = j < n && p.prev ? p.decay * p.prev[row + j] : 0.f;
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kSMma) tmem_dealloc(tmem, 128);
}

template <typename F>
cudaError_t for_step(int R, int D, bool tma, F&& f) {
#define SDA_CASE(RV, DV)                                                                      \
  if (R == RV && D == DV)                                                                     \
    return tma ? f(mass_step_kernel<RV, DV, true>, (size_t)StepCfg<RV, DV>::kSmem, dim3(384)) \
               : f(mass_step_kernel<RV, DV, false>, (size_t)StepCfg<RV, DV>::kSmem, dim3(640));
  SDA_CASE(16, 64) SDA_CASE(16, 128) SDA_CASE(16, 256) SDA_CASE(16, 512)
  SDA_CASE(64, 64) SDA_CASE(64, 128) SDA_CASE(64, 256) SDA_CASE(64, 512)
#undef SDA_CASE
  return cudaErrorInvalidValue;
}

template <typename F>
cudaError_t for_dim(int D, F&& f) {
  switch (D) {
    case 64: return f(mass_kernel<64>, (size_t)Cfg<64>::kSmem);
    case 128: return f(mass_kernel<128>, (size_t)Cfg<128>::kSmem);
    case 256: return f(mass_kernel<256>, (size_t)Cfg<256>::kSmem);
    case 512: return f(mass_kernel<512>, (size_t)Cfg<512>::kSmem);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

MassLayout mass_layout(int B, int64_t S, int num_sms) {
  MassLayout L;
  L.u_max = (int)((S + kKeys - 1) / kKeys * B);
  L.grid = (num_sms < kMaxPlanGrid ? num_sms : kMaxPlanGrid) / 2;  // pairs
  size_t off = kErrorWords + kErrorBytes;
  L.units_off = off;
  off = align256(off + (size_t)L.u_max * sizeof(MassUnit));
  L.seq_off = off;
  off = align256(off + (size_t)(B + 1) * 4);
  L.cta_off = off;
  off = align256(off + (size_t)(L.grid + 1) * 4);
  L.part_off = off;
  off = align256(off + (size_t)2 * L.grid * kKeys * 4);
  L.total = off;
  return L;
}

cudaError_t mass_prepare() {
  for (int D : {64, 128, 256, 512}) {
    const cudaError_t e = for_dim(D, [&](auto kernel, size_t smem) {
      return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    });
    if (e != cudaSuccess) return e;
    for (int R : {16, 64}) {
      for (bool tma : {false, true}) {
        const cudaError_t r = for_step(R, D, tma, [&](auto kernel, size_t smem, dim3) {
          return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        });
        if (r != cudaSuccess) return r;
      }
    }
  }
  return cudaSuccess;
}

// Few rows a sequence, cached rows streamed past them.
static cudaError_t launch_mass_step(const void* q, const void* kv, const ChunkGeom& g,
                                    const float* lse, float scale, const float* prev, float decay,
                                    float* out, int num_sms, void* ws, cudaStream_t st) {
  const int R = (int64_t)g.T * g.H <= (int64_t)16 * g.B ? 16 : 64;
  const bool tma = chunk_boxes(g);
  StepParams p;
  p.kv = static_cast<const __nv_bfloat16*>(kv);
  p.lse = lse;
  p.prev = prev;
  p.out = out;
  p.hdr = static_cast<ChunkHeader*>(ws);
  p.g = g;
  p.S = (int64_t)g.max_blocks * g.k_per_block;
  p.qk_scale_log2 = scale * kLog2e;
  p.decay = decay;
  p.wait_timeout_ns = current_wait_fault().timeout_ns;
  CUtensorMap tq, tkv = {};
  if (!pipe_map_2d(&tq, q, g.D, (uint64_t)g.T * g.H, 64, R) ||
      (tma && !pipe_map_pool(&tkv, p.kv + g.base * g.D, g.D, (uint64_t)(g.total_pages - g.base) / 8,
                             g.D >= 256 ? g.D / 128 : g.D / 64, 2)))
    return cudaErrorInvalidValue;
  return for_step(R, g.D, tma, [&](auto kernel, size_t smem, dim3 threads) {
    return launch_pdl(kernel, dim3(num_sms), threads, smem, st, tq, tkv, p);
  });
}

cudaError_t launch_mass(const void* q, const void* kv, const ChunkGeom& g, const float* lse,
                        float scale, const float* prev, float decay, float* out,
                        const MassLayout& L, void* ws, cudaStream_t st) {
  char* base = static_cast<char*>(ws);
  ChunkHeader* hdr = reinterpret_cast<ChunkHeader*>(base);
  MassUnit* units = reinterpret_cast<MassUnit*>(base + L.units_off);
  int* cta_unit = reinterpret_cast<int*>(base + L.cta_off);
  float* part = reinterpret_cast<float*>(base + L.part_off);
  const int64_t S = (int64_t)g.max_blocks * g.k_per_block;
  // Up to 64 rows a sequence on average: their scores with a tile of positions are one
  // MMA tile, and the time is that of reading the cache once.  (q_indptr lies on the
  // device, so the rule goes by the average.  A batch whose rows are all in one sequence
  // reloads them, 64 at a time, for every tile of its positions: 64 sequences of 4096
  // positions, 64 heads, 64 tokens in one and none in the others, D = 512, 96 us, where
  // 65 tokens, by the kernel for chunks, take 27; one token in each takes 49.)
  if (g.T > 0 && (int64_t)g.T * g.H <= (int64_t)64 * g.B && g.B <= kStepSeqs)
    return launch_mass_step(q, kv, g, lse, scale, prev, decay, out, 2 * L.grid, ws, st);
  const int64_t fill = (g.B * S + kPlanThreads - 1) / kPlanThreads;
  cudaError_t e = launch_pdl(mass_plan_kernel, dim3(1 + (unsigned)(fill < 2 * L.grid ? fill : 2 * L.grid)),
                             dim3(kPlanThreads), 0, st, g, S, L.grid, L.u_max, prev, decay, out, hdr,
                             units, reinterpret_cast<int*>(base + L.seq_off), cta_unit);
  if (e != cudaSuccess || g.T == 0 || S == 0) return e;
  CUtensorMap tq;
  if (!pipe_map_2d(&tq, q, g.D, (uint64_t)g.T * g.H, 64, 128)) return cudaErrorInvalidValue;
  Params p;
  p.kv = static_cast<const __nv_bfloat16*>(kv);
  p.lse = lse;
  p.out = out;
  p.hdr = hdr;
  p.units = units;
  p.cta_unit = cta_unit;
  p.part = part;
  p.g = g;
  p.S = S;
  p.qk_scale_log2 = scale * kLog2e;
  p.wait_timeout_ns = current_wait_fault().timeout_ns;
  e = for_dim(g.D, [&](auto kernel, size_t smem) {
    return launch_pdl_cluster(kernel, dim3(2 * L.grid), dim3(kThreads), 2, smem, st, tq, p);
  });
  if (e != cudaSuccess || L.grid < 2) return e;
  return launch_pdl(mass_combine_kernel, dim3(L.grid - 1), dim3(kKeys), 0, st,
                    static_cast<const ChunkHeader*>(hdr), static_cast<const MassUnit*>(units),
                    static_cast<const int*>(cta_unit), static_cast<const float*>(part), S, out);
}

}  // namespace sda
