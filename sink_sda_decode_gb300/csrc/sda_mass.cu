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
// A work unit is a tile of 128 positions, which stays in shared memory, with
// the q rows that see any of it; it is cut into tiles of 128 rows, streamed
// as 64-column panels.  All (position tile, row tile) pairs form one
// sequence, cut into equal ranges, one per CTA; a unit that a range boundary
// cuts leaves 128 partial sums per piece, which a last kernel adds up in
// order.
//   warps 0..7    epilogue: warp w reads TMEM lane quadrant w % 4 (positions)
//                 and half w / 4 of the row tile's columns
//   warps 8..23   the unit's cached rows, 16-byte cp.async
//   warp 24       q panels by TMA;  warp 25: the MMAs
#include <cuda_bf16.h>

#include "sda_chunk.cuh"
#include "sda_pipe.cuh"

namespace sda {

namespace {

using namespace ptx;

constexpr int kKeys = 128;                // positions per unit
constexpr int kRowsQ = 128;               // q rows per tile
constexpr int kPanelB = 128 * 128;        // bytes of a panel: 128 rows x 64 columns
constexpr int kEpWarps = 8, kEpThreads = 256;
constexpr int kLoadWarp0 = 8, kLoadWarps = 16;
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

enum Bar : int { kKFull = 0, kKEmpty, kAccFull0, kAccEmpty0 = kAccFull0 + 2, kDrain = kAccEmpty0 + 2, kQFull0 };

template <int D>
struct Cfg {
  static constexpr int kPanels = D / 64;
  static constexpr int kRing = D == 512 ? 5 : 8;  // q panels in flight
  static constexpr int kOffK = 0;
  static constexpr int kOffQ = kPanels * kPanelB;
  static constexpr int kOffCol = kOffQ + kRing * kPanelB;  // per row tile: lse2 float[128], pos int[128]; two of them
  static constexpr int kOffHalf = kOffCol + 2 * 1024;      // float [128]: the second column half's sums
  static constexpr int kOffBar = kOffHalf + 512;
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
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(bar(kKFull), kLoadWarps);
    mbar_init(bar(kKEmpty), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kAccFull0 + i), 1);
      mbar_init(bar(kAccEmpty0 + i), kEpWarps);
    }
    mbar_init(bar(kDrain), 1);
    for (int i = 0; i < C::kRing; ++i) {
      mbar_init(q_full(i), 1);
      mbar_init(q_empty(i), 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmap_q);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_addr(tmem_slot), 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_trigger();
  const int per = __ldcg(&p.hdr->per), n_tiles = __ldcg(&p.hdr->n_tiles);
  const int t0 = (int)min((long long)blockIdx.x * per, (long long)n_tiles);
  const int t1 = (int)min((long long)(blockIdx.x + 1) * per, (long long)n_tiles);
  PieceWalk walk{p.units, t0 < t1 ? __ldcg(p.cta_unit + blockIdx.x) : 0, t0, t1};
  const PipeWait wc{abort_flag, &p.hdr->error, p.wait_timeout_ns};
  Piece pc;

  if (warp >= kLoadWarp0 && warp < kLoadWarp0 + kLoadWarps) {
    // ===================================================== the unit's cached rows
    constexpr int kRows = kKeys / kLoadWarps;  // 8 rows per warp: one swizzle atom
    constexpr int kCh = D / 8 < 32 ? D / 8 : 32;
    constexpr int kRowsPer = 32 / kCh;
    const int v = warp - kLoadWarp0;
    const uint4* kv4 = reinterpret_cast<const uint4*>(p.kv);
    bool ok = true;
    for (int x = 0; ok && walk.next(&pc); ++x) {
      int sl = -1;
      const int j = pc.un.k0 + v * kRows + lane;
      if (lane < kRows && j < pc.un.n) {
        const int blk = __ldg(p.g.block_table + (size_t)pc.un.b * p.g.max_blocks + j / p.g.k_per_block);
        const long long s = p.g.base + (long long)blk * p.g.k_per_block + j % p.g.k_per_block;
        if (blk < 0 || s >= p.g.total_pages) atomicExch(&p.hdr->error, 3);
        else sl = (int)s;
      }
      if (x > 0) {
        if (lane == 0) ok = pipe_wait(bar(kKEmpty), (x - 1) & 1, wc);
        ok = __shfl_sync(0xffffffffu, ok, 0);
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
          cp_async16(sK + (ch >> 3) * kPanelB + v * 1024 + r * 128 + (((ch & 7) ^ r) << 4), src,
                     slot >= 0 ? 16u : 0u);
        }
      }
      cp_async_commit();
      cp_async_wait_group<0>();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kKFull));
    }
  } else if (warp == kQWarp) {
    // ===================================================== q panels
    if (lane == 0) {
      int f = 0;  // panels issued
      bool ok = true;
      while (ok && walk.next(&pc)) {
        for (int i = pc.i0; i < pc.i1 && ok; ++i) {
          for (int x = 0; x < NP; ++x, ++f) {
            const int s = f % C::kRing;
            if (f >= C::kRing) ok = pipe_wait(q_empty(s), ((f / C::kRing) - 1) & 1, wc);
            if (!ok) break;
            mbar_arrive_expect_tx(q_full(s), kPanelB);
            tma_load_2d(sQ + s * kPanelB, &tmap_q, x * 64, pc.un.row0 + i * kRowsQ, q_full(s));
          }
        }
      }
      for (int s = 0; s < C::kRing; ++s)  // copies in flight land before the CTA's memory goes away
        if (f > s) pipe_drain(q_full(s), ((f - 1 - s) / C::kRing) & 1, wc);
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ===================================================== MMAs
    if (lane == 0) {
      int f = 0, g = 0;
      bool ok = true;
      for (int x = 0; ok && walk.next(&pc); ++x) {
        ok = pipe_wait(bar(kKFull), x & 1, wc);
        for (int i = pc.i0; i < pc.i1 && ok; ++i, ++g) {
          const int s = g & 1;
          if (g >= 2) ok = pipe_wait(bar(kAccEmpty0 + s), ((g >> 1) - 1) & 1, wc);
          const uint64_t a0 = sdesc_sw128(sK, 16, 1024);
          for (int y = 0; y < NP && ok; ++y, ++f) {
            const int r = f % C::kRing;
            ok = pipe_wait(q_full(r), (f / C::kRing) & 1, wc);
            if (!ok) break;
            tc_fence_after();
            const uint64_t b0 = sdesc_sw128(sQ + r * kPanelB, 16, 1024);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_bf16(tmem + s * 128, sdesc_advance(a0, y * kPanelB + k * 32),
                       sdesc_advance(b0, k * 32), C::kIdesc, (y || k) ? 1u : 0u);
            mma_commit(q_empty(r));
          }
          if (ok) mma_commit(bar(kAccFull0 + s));
        }
        if (ok) mma_commit(bar(kKEmpty));
      }
      mma_commit(bar(kDrain));
      pipe_drain(bar(kDrain), 0, wc);
    }
    __syncwarp();
  } else if (warp < kEpWarps) {
    // ===================================================== weights and sums
    const int q4 = warp & 3, hc = warp >> 2, st = threadIdx.x;
    const uint32_t lane_base = (uint32_t)(q4 * 32) << 16;
    float* s_half = reinterpret_cast<float*>(smem + C::kOffHalf);
    const float sc = p.qk_scale_log2;
    const int H = p.g.H, window = p.g.window, nfirst = p.g.first;
    int g = 0;
    while (walk.next(&pc)) {
      const MassUnit& un = pc.un;
      const int j = un.k0 + q4 * 32 + lane;  // this thread's position
      const int k_last = min(un.k0 + kKeys, un.n) - 1;
      float sum = 0.f, comp = 0.f;
      for (int i = pc.i0; i < pc.i1; ++i, ++g) {
        const int s = g & 1;
        float* lse2 = reinterpret_cast<float*>(smem + C::kOffCol + s * 1024);
        int* cpos = reinterpret_cast<int*>(smem + C::kOffCol + s * 1024 + 512);
        const int r0 = i * kRowsQ, nr = min(kRowsQ, un.nrows - r0);
        if (st < kRowsQ) {
          const bool in = st < nr;
          lse2[st] = in ? __ldg(p.lse + un.row0 + r0 + st) * kLog2e : 0.f;
          cpos[st] = in ? un.pos0 + (r0 + st) / H : INT_MIN;
        }
        named_bar_sync(1, kEpThreads);  // (also: everyone is past the tile that used these arrays)
        const int p_lo = un.pos0 + r0 / H, p_hi = un.pos0 + (r0 + nr - 1) / H;
        const bool full = nr == kRowsQ && k_last <= p_lo &&
                          (window == 0 || un.k0 > p_hi - window || k_last < nfirst);
        pipe_wait(bar(kAccFull0 + s), (g >> 1) & 1, wc);
        tc_fence_after();
        float part = 0.f;
#pragma unroll 1
        for (int c0 = hc * 64; c0 < hc * 64 + 64 && c0 < nr; c0 += 16) {
          uint32_t v[16];
          tmem_ld16(tmem + lane_base + s * 128 + c0, v);
          tmem_wait_ld();
          float a[4] = {0.f, 0.f, 0.f, 0.f};
          if (full) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
              a[e & 3] += ex2_approx(fmaf(__uint_as_float(v[e]), sc, -lse2[c0 + e]));
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const int pos = cpos[c0 + e];
              const bool see = j <= pos && (window == 0 || j > pos - window || j < nfirst);
              const float w = ex2_approx(fmaf(__uint_as_float(v[e]), sc, -lse2[c0 + e]));
              a[e & 3] += see ? w : 0.f;
            }
          }
          part += (a[0] + a[1]) + (a[2] + a[3]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kAccEmpty0 + s));
        // compensated: a unit can have a million rows
        const float y = part - comp, t = sum + y;
        comp = (t - sum) - y;
        sum = t;
      }
      if (hc == 1) s_half[q4 * 32 + lane] = sum;
      named_bar_sync(1, kEpThreads);
      if (hc == 0) {
        sum += s_half[q4 * 32 + lane];
        if (pc.i0 == 0 && pc.i1 == un.nq) {
          if (j < un.n) p.out[(int64_t)un.b * p.S + j] += sum;
        } else {
          p.part[(size_t)(2 * blockIdx.x + (pc.i0 == 0 ? 1 : 0)) * kKeys + q4 * 32 + lane] = sum;
        }
      }
      named_bar_sync(1, kEpThreads);  // s_half may be rewritten
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 256);
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
  L.grid = num_sms < kMaxPlanGrid ? num_sms : kMaxPlanGrid;
  size_t off = sizeof(ChunkHeader);
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
  }
  return cudaSuccess;
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
  const int64_t fill = (g.B * S + kPlanThreads - 1) / kPlanThreads;
  cudaError_t e = launch_pdl(mass_plan_kernel, dim3(1 + (unsigned)(fill < L.grid ? fill : L.grid)),
                             dim3(kPlanThreads), 0, st, g, S, L.grid, L.u_max, prev, decay, out, hdr,
                             units, reinterpret_cast<int*>(base + L.seq_off), cta_unit);
  if (e != cudaSuccess || g.T == 0 || S == 0) return e;
  CUtensorMap tq;
  if (!pipe_map_2d(&tq, q, g.D, (uint64_t)g.T * g.H, 64, kRowsQ)) return cudaErrorInvalidValue;
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
    return launch_pdl(kernel, dim3(L.grid), dim3(kThreads), smem, st, tq, p);
  });
  if (e != cudaSuccess || L.grid < 2) return e;
  return launch_pdl(mass_combine_kernel, dim3(L.grid - 1), dim3(kKeys), 0, st,
                    static_cast<const ChunkHeader*>(hdr), static_cast<const MassUnit*>(units),
                    static_cast<const int*>(cta_unit), static_cast<const float*>(part), S, out);
}

}  // namespace sda
