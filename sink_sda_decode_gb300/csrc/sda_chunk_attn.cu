// sda_chunk_attn.cu -- attention of a chunk of new tokens of every sequence
// over its cached positions, found through a block table (tcgen05 / TMEM).
//
// For every row (token i of sequence b, head h), over the positions j the
// token sees (sda_chunk.cuh):
//   x_j = scale <q, kv_j>,  lse = log(e^sink_h + sum_j e^(x_j)),
//   out = sum_j e^(x_j - lse) kv_j
// as an online softmax in the log2 domain.  A cached row is key and value of
// every head, so R consecutive (token, head) rows of q form one tile of
// queries whatever H is, and each KV tile is read once per tile of queries.  This
// kernel has R = 16 or 64, for sequences of up to 128 rows on average (steps, drafted
// tokens of few heads) and for D <= 128; sda_chunk_pair.cu takes the others.
//
// One persistent CTA per SM owns a contiguous range of KV tiles, which it finds itself
// or a plan has found (sda_chunk.cuh, ChunkMode).  Roles:
//   warps 0..7   softmax and epilogue
//   warp 8       QK MMAs and the q loads (TMA)
//   warp 9       PV MMAs
//   warp 10      KV tiles by TMA where blocks hold a multiple of 16 rows
//   warps 12..   (gather kernel, other block sizes) 8 warps copy the tile's rows
//                one by one with 16-byte cp.async
// S = Q K^T (M = 64 rows, N = a tile of positions) and O^T += V^T P^T (M = 128
// of D, N = R rows, K = the positions) read the same shared tile, K-major as K
// and MN-major as V.  A tile lies as groups of 8 rows, each group D / 64
// swizzle atoms of 1 KB.
//
// What bounds it at D = 512 and R = 64: with three stages of 48 positions, the way of a
// stage from its load over scores, softmax and PV to its release; neither the tensor
// pipe (active 40 %) nor DRAM (60 %) is full.  One token of 64 heads over 8 caches of
// 16384 to 65536 positions (365 MB): 86 us, where a copy of as many bytes takes 55;
// about 12 of them are the merge of cut units.
#include <cuda_bf16.h>

#include <type_traits>

#include "sda_chunk_dev.cuh"

namespace sda {

namespace {

using namespace ptx;

constexpr int kSmWarps = 8;
constexpr int kSmThreads = kSmWarps * 32;
constexpr int kQkWarp = 8, kPvWarp = 9, kTmaWarp = 10;
constexpr int kLoadWarp0 = 12, kLoadWarps = 8;  // gather kernel only
constexpr int kMaxStages = 6;
// Gather kernel: 640 threads launch with 96 registers each; the softmax warps
// grow to 128 and the loaders shrink to 64 (the MMA warpgroup keeps 96).
constexpr int kGatherThreads = 640, kGatherRegs = 96;
static_assert(kSmThreads * 128 + kLoadWarps * 32 * 64 + 128 * 96 <= kGatherThreads * kGatherRegs,
              "register split exceeds the launch allocation");

enum Bar : int {
  kQFull = 0,
  kQEmpty,
  kSFull0,
  kSEmpty0 = kSFull0 + 2,
  kPReady0 = kSEmpty0 + 2,
  kDrainQk = kPReady0 + 2,
  kDrainPv,
  kKvFull0,                              // + 2 * stage + half of D
  kPvDone0 = kKvFull0 + 2 * kMaxStages,  // + 2 * stage + half of D
  kBars = kPvDone0 + 2 * kMaxStages
};

template <int R, int D>
struct Cfg {
  static constexpr int kTile = chunk_tile(R, D);
  static constexpr int kPanels = D / 64;
  static constexpr int kBlocks = (D + 127) / 128;    // 128-row blocks of O^T
  static constexpr int kHalves = D >= 256 ? 2 : 1;   // a stage is filled and freed in halves of D
  static constexpr int kPanelsH = kPanels / kHalves, kBlocksH = kBlocks / kHalves;
  // a stage: halves of D, each [groups of 8 rows][panels][1 KB atom]
  static constexpr int kGroup = kPanelsH * 1024;
  static constexpr int kHalf = kTile / 8 * kGroup;
  static constexpr int kStage = kHalves * kHalf;
  static constexpr int kBox = 2 * kGroup, kBoxes = kTile / 16;  // a TMA box: 16 rows of a half
  static constexpr int kStages = D == 512 ? 3 : (D == 256 ? 5 : 6);
  static constexpr int kPanelQ = R * 128;
  static constexpr int kPBytes = R * 128;
  static constexpr int kOffQ = 0;
  static constexpr int kOffKV = kPanels * kPanelQ;
  static constexpr int kOffP = kOffKV + kStages * kStage;  // two P buffers; the epilogue's staging
  static constexpr int kOffBar = kOffP + 2 * kPBytes;
  static constexpr int kOffMisc = kOffBar + 8 * kBars;
  static constexpr int kOffLSum = kOffMisc + 16;        // float [2][64]
  static constexpr int kOffAlpha = kOffLSum;            // aliases the first half (used inside a unit)
  static constexpr int kOffFac = kOffLSum + 4 * 64;     // aliases the second half
  static constexpr int kOffHMax = kOffLSum + 4 * 128;   // float [2 tiles][2][64]
  // The QK MMA reads 64 rows of a q panel and the PV MMA 128 columns of D
  // whatever R and D are: what lies behind (other panels and stages, valid
  // shared memory) lands in TMEM lanes that nothing reads.
  static constexpr int kUsed = kOffHMax + 4 * 256;
  static constexpr int kSmem = kUsed + 1024;
  static constexpr int kOCol = 128;
  static constexpr int kTmemCols = kOCol + kBlocks * R <= 256 ? 256 : 512;
  static constexpr uint32_t kIdescQK = idesc_bf16_f32(64, kTile, false, false);
  static constexpr uint32_t kIdescPV = idesc_bf16_f32(128, R, true, false);
  static_assert(kOCol + kBlocks * R <= 512, "TMEM columns");
  static_assert(kOffKV % 1024 == 0 && kOffP % 1024 == 0 && kPBytes % 1024 == 0, "swizzle atoms");
  static_assert((kPanels - 1) * kPanelQ + 64 * 128 <= kOffBar, "padded QK operand inside smem");
  static_assert(D >= 128 || 2 * kPBytes >= 1024, "padded PV operand inside smem");
  static_assert(kTile % 16 == 0 && kTile <= 64, "MMA shapes");
  static_assert(kStages * kStage >= 4 * (kFusedSeqs + 1), "chunk_begin's words");
  static_assert(kSmem <= 232448, "shared memory budget");
};

template <int R, int D, bool TMA>
__global__ void __launch_bounds__(TMA ? 384 : kGatherThreads, 1)
chunk_attn_kernel(const __grid_constant__ CUtensorMap tmap_q,
                  const __grid_constant__ CUtensorMap tmap_kv, const ChunkParams p) {
  using C = Cfg<R, D>;
  constexpr int KS = C::kStages;
  constexpr int HV = C::kHalves;
  constexpr int kTile = C::kTile;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_addr(smem);
  const uint32_t sQ = sbase + C::kOffQ, sKV = sbase + C::kOffKV, sP = sbase + C::kOffP;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  auto bar = [&](int i) { return sbase + C::kOffBar + 8u * (uint32_t)i; };
  auto kv_full = [&](int s, int h) { return bar(kKvFull0 + 2 * s + h); };
  auto pv_done = [&](int s, int h) { return bar(kPvDone0 + 2 * s + h); };

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(bar(kQFull), 1);
    mbar_init(bar(kQEmpty), 1);
    for (int s = 0; s < KS; ++s) {
      for (int h = 0; h < HV; ++h) {
        mbar_init(kv_full(s, h), TMA ? 1 : kLoadWarps * 32);
        mbar_init(pv_done(s, h), 1);
      }
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(kSFull0 + s), 1);
      mbar_init(bar(kSEmpty0 + s), kSmWarps);
      mbar_init(bar(kPReady0 + s), 1);
    }
    mbar_init(bar(kDrainQk), 1);
    mbar_init(bar(kDrainPv), 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmap_q);
    if (TMA) tma_prefetch_desc(&tmap_kv);
  }
  if (warp == kQkWarp) {
    tmem_alloc(smem_addr(tmem_slot), C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();  // everything above overlaps the plan; global memory only below
  pdl_trigger();
  bool bad;
  const ChunkStart begin = chunk_begin<TMA ? 384 : kGatherThreads, R, kTile>(
      p, blockIdx.x, reinterpret_cast<int*>(smem + C::kOffKV),
      reinterpret_cast<int*>(smem + C::kOffP), &bad);
  const int nt = begin.nt;  // this CTA's tiles
  int* const error = reinterpret_cast<int*>(reinterpret_cast<char*>(p.hdr) + kErrorWords) + blockIdx.x;
  if (threadIdx.x == 0) {
    *error = 0;
    if (bad && p.mode == kCut) p.recs[blockIdx.x] = ChunkUnit{-1};
    if (blockIdx.x == 0) {
      p.hdr->words = gridDim.x;
      if (p.mode != kPlanned) p.hdr->error = bad ? 2 : 0;
    }
  }
  __syncthreads();
  const PipeWait wc{abort_flag, error, p.wait_timeout_ns};
  using Walk = Cursor<R, kTile>;

  if (TMA && warp == kTmaWarp) {
    // ===================================================== KV tiles by TMA
    // Lane i < kBoxes loads box i of 16 rows of every tile, each half of D as soon
    // as the PV MMAs that last read it are done.  (Boxes of 8 rows, and bulk
    // prefetches of the tile two ahead into L2, kept this warp busier than the
    // tensor pipe: one TMA instruction costs about 90 cycles of issue.)
    const int behind = (int)((p.g.total_pages - p.g.base) / 8);
    bool over = false;
    auto box_of = [&](const Walk& c) {
      return lane < C::kBoxes
                 ? box_group(p, error, c, c.start() + lane * 16, &over)
                 : behind;
    };
    Walk c;  // runs a tile ahead of the copies
    c.init(p.g, begin);
    int y = behind;
    if (c.left > 0) {
      y = box_of(c);
      c.next(p.g);
    }
    bool ok = true;
    int loads = 0;
    for (int g = 0; g < nt && ok; ++g) {
      const int s = g % KS;
#pragma unroll
      for (int h = 0; h < HV; ++h) {
        if (g >= KS) ok = warp_wait(pv_done(s, h), ((g / KS) - 1) & 1, wc);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(kv_full(s, h), C::kHalf);
        __syncwarp();
        const uint32_t dst = sKV + s * C::kStage + h * C::kHalf + lane * C::kBox;
        if (lane < C::kBoxes) tma_load_4d(dst, &tmap_kv, 0, 0, h * C::kPanelsH, y, kv_full(s, h));
        ++loads;
      }
      if (c.left > 0) {  // (after this tile's copies: the table entry is a while coming)
        y = box_of(c);
        c.next(p.g);
      }
    }
    if (over) atomicExch(error, 3);
    // copies in flight land before the CTA's memory goes away (the last KS stages)
    for (int x = max(0, loads - KS * HV); x < loads; ++x)
      pipe_drain(kv_full((x / HV) % KS, x % HV), (x / HV / KS) & 1, wc);
  } else if (!TMA && warp >= kLoadWarp0) {
    // ===================================================== KV rows one by one
    setmaxnreg_dec<64>();
    constexpr int kRows = kTile / kLoadWarps;          // 6 or 8 rows per warp and tile
    constexpr int kCh = D / 8 / HV;                    // 16-byte chunks of a row's half
    constexpr int kRowsPer = 32 / kCh;                 // rows per warp-wide copy
    const int v = warp - kLoadWarp0;
    const uint4* kv4 = reinterpret_cast<const uint4*>(p.kv);
    auto slot_of = [&](const Walk& c) {  // lanes 0 .. kRows - 1: rows kRows v + lane
      return lane < kRows
                 ? seen_row(p, error, c, c.start() + v * kRows + lane)
                 : -1;
    };
    auto prefetch = [&](int slot) {
      if (slot >= 0) bulk_prefetch_l2(reinterpret_cast<const uint8_t*>(p.kv) + (size_t)slot * D * 2, D * 2);
    };
    Walk c;  // runs two tiles ahead of the copies
    c.init(p.g, begin);
    int sl0 = -1, sl1 = -1;
    if (c.left > 0) {
      sl0 = slot_of(c);
      c.next(p.g);
    }
    if (c.left > 0) {
      sl1 = slot_of(c);
      c.next(p.g);
    }
    bool ok = true;
    for (int g = 0; g < nt && ok; ++g) {
      const int s = g % KS;
      const uint32_t stage = sKV + s * C::kStage;
#pragma unroll
      for (int h = 0; h < HV; ++h) {
        if (g >= KS) ok = warp_wait(pv_done(s, h), ((g / KS) - 1) & 1, wc);
        if (!ok) break;
        const int ch = h * kCh + lane % kCh;  // 16-byte chunk of the row
#pragma unroll
        for (int x = 0; x < kRows; x += kRowsPer) {
          const int rl = x + lane / kCh;  // (past the warp's rows where kRowsPer does not divide them)
          const int slot = __shfl_sync(0xffffffffu, sl0, rl & 31);
          const int r = v * kRows + rl;
          const uint32_t dst = stage + h * C::kHalf + (r >> 3) * C::kGroup +
                               ((lane % kCh) >> 3) * 1024 + (r & 7) * 128 +
                               (((ch & 7) ^ (r & 7)) << 4);
          const uint4* src = slot >= 0 ? kv4 + (size_t)slot * (D / 8) + ch : kv4;
          if (rl < kRows) cp_async16(dst, src, slot >= 0 ? 16u : 0u);
        }
        // arrives once this thread's copies have landed, so that the warp goes
        // on to the next stage meanwhile (the reader fences to the async proxy)
        cp_async_arrive(kv_full(s, h));
      }
      prefetch(sl1);
      sl0 = sl1;
      sl1 = -1;
      if (c.left > 0) {
        sl1 = slot_of(c);
        c.next(p.g);
      }
    }
    cp_async_wait_all();
  } else if (warp == kQkWarp) {
    // ===================================================== QK MMAs
    Walk c;
    c.init(p.g, begin);
    int pieces = 0, q_loads = 0;
    bool ok = true;
    auto load_q = [&]() {
      const int row = c.row0;
      if (elect_one()) {
        mbar_arrive_expect_tx(bar(kQFull), C::kPanels * C::kPanelQ);
#pragma unroll
        for (int x = 0; x < C::kPanels; ++x)
          tma_load_2d(sQ + x * C::kPanelQ, &tmap_q, x * 64, row, bar(kQFull));
      }
      __syncwarp();
      ++q_loads;
    };
    if (c.left > 0) load_q();
    const uint64_t a0 = sdesc_sw128(sQ, 16, 1024);
    for (int g = 0; g < nt; ++g) {
      const int s = g & 1, ks = g % KS;
      if (g >= 2) ok = warp_wait(bar(kSEmpty0 + s), ((g >> 1) - 1) & 1, wc);
      if (ok && c.first) ok = warp_wait(bar(kQFull), pieces & 1, wc);
      const uint64_t b0 = sdesc_sw128(sKV + ks * C::kStage, 16, C::kGroup);
      const bool last = c.last();
#pragma unroll
      for (int h = 0; h < HV; ++h) {
        if (ok) ok = warp_wait(kv_full(ks, h), (g / KS) & 1, wc);
        if (!ok) break;
        if (!TMA) fence_proxy_async_smem();  // the copies were made through the generic proxy
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int x = 0; x < C::kPanelsH; ++x) {
            const int pn = h * C::kPanelsH + x;
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_bf16(tmem + s * 64, sdesc_advance(a0, pn * C::kPanelQ + k * 32),
                       sdesc_advance(b0, h * C::kHalf + x * 1024 + k * 32), C::kIdescQK, (pn || k) ? 1u : 0u);
          }
          if (h == HV - 1) {
            mma_commit(bar(kSFull0 + s));
            if (last) mma_commit(bar(kQEmpty));
          }
        }
        __syncwarp();
      }
      if (!ok) break;
      c.next(p.g);
      if (last) {
        if (c.left > 0) {  // q of the next unit, once this unit's MMAs have read q
          ok = warp_wait(bar(kQEmpty), pieces & 1, wc);
          if (!ok) break;
          load_q();
        }
        ++pieces;
      }
    }
    if (elect_one()) {
      mma_commit(bar(kDrainQk));
      pipe_drain(bar(kDrainQk), 0, wc);
      if (q_loads > 0) pipe_drain(bar(kQFull), (q_loads - 1) & 1, wc);
    }
    __syncwarp();
  } else if (warp == kPvWarp) {
    // ===================================================== PV MMAs
    Walk c;
    c.init(p.g, begin);
    for (int g = 0; g < nt; ++g) {
      const int s = g & 1, ks = g % KS;
      if (!warp_wait(bar(kPReady0 + s), (g >> 1) & 1, wc)) break;
      if (!TMA) fence_proxy_async_smem();
      tc_fence_after();
      const uint64_t a0 = sdesc_sw128(sKV + ks * C::kStage, 1024, C::kGroup);
      const uint64_t b0 = sdesc_sw128(sP + s * C::kPBytes, 16, 1024);
      const uint32_t add = c.first ? 0u : 1u;
      if (elect_one()) {
#pragma unroll
        for (int b = 0; b < C::kBlocks; ++b) {
#pragma unroll
          for (int k = 0; k < kTile / 16; ++k)
            mma_bf16(tmem + C::kOCol + b * R,
                     sdesc_advance(a0, b / C::kBlocksH * C::kHalf + 2 * (b % C::kBlocksH) * 1024 +
                                           k * 2 * C::kGroup),
                     sdesc_advance(b0, k * 32), C::kIdescPV, k ? 1u : add);
          if ((b + 1) % C::kBlocksH == 0) mma_commit(pv_done(ks, b / C::kBlocksH));
        }
      }
      __syncwarp();
      c.next(p.g);
    }
    if (elect_one()) {
      mma_commit(bar(kDrainPv));
      pipe_drain(bar(kDrainPv), 0, wc);
    }
    __syncwarp();
  } else if (warp < kSmWarps) {
    // ===================================================== softmax and epilogue
    if constexpr (!TMA) setmaxnreg_inc<128>();
    // Warp w reads TMEM lane quadrant q4 = w % 4 and half hc = w / 4 of each
    // tile's positions: thread t holds rows hA = 16 q4 + t / 4 and hB = hA + 8 at
    // the positions kPos hc + 8 rep + 2 (t % 4) + {0, 1}.
    constexpr int kPos = kTile / 2, kReps = kPos / 8, kE = 4 * kReps;
    const int q4 = warp & 3, hc = warp >> 2, st = threadIdx.x, tq = lane & 3;
    const int hA = q4 * 16 + (lane >> 2), hB = hA + 8;
    const uint32_t lane_base = (uint32_t)(q4 * 32) << 16;
    float* s_alpha = reinterpret_cast<float*>(smem + C::kOffAlpha);
    float* s_fac = reinterpret_cast<float*>(smem + C::kOffFac);
    float* s_lsum = reinterpret_cast<float*>(smem + C::kOffLSum);
    float* s_hmax = reinterpret_cast<float*>(smem + C::kOffHMax);
    const float sc = p.qk_scale_log2;
    const int H = p.g.H, window = p.g.window, nfirst = p.g.first;
    const bool held = hA < R;  // this warp's rows exist in P (uniform over the warp)
    // Control flow is the same in the eight warps (it depends on the plan and
    // on block-wide votes), so every named barrier is reached by all of them
    // even after a wait timed out.
    int g = 0;
    UnitWalk uw;
    uw.init(p.g, R, begin);
    for (int pieces = 0; g < nt; ++pieces) {
      if (pieces > 0) uw.next(p.g, R);
      const ChunkUnit un = chunk_unit(p.g, R, kTile, uw.b, uw.r);
      const int i0 = g == 0 ? begin.off : 0;
      const int i1 = min(un.ntiles, i0 + nt - g);
      const bool whole = i0 == 0 && i1 == un.ntiles;
      const bool vA = hA < un.nrows, vB = hB < un.nrows;
      const int tokA = div_h(p.g, un.h0 + hA), tokB = div_h(p.g, un.h0 + hB);
      const int posA = un.pos0 + tokA, posB = un.pos0 + tokB;
      const int p_lo = un.pos0, p_hi = un.pos0 + div_h(p.g, un.h0 + un.nrows - 1);
      const float sinkA = whole && vA ? __ldg(p.attn_sink + un.h0 + hA - tokA * H) : 0.f;
      const float sinkB = whole && vB ? __ldg(p.attn_sink + un.h0 + hB - tokB * H) : 0.f;
      const float scA = vA ? sc : 0.f, scB = vB ? sc : 0.f;
      float mA = kNoScore, mB = kNoScore, lA = 0.f, lB = 0.f;  // l: this thread's share
      for (int i = i0; i < i1; ++i, ++g) {
        const int s = g & 1;
        const int j0 = chunk_tile_start(i, un.nf, un.lo, kTile);
        // whether every row of the unit sees the whole tile
        const bool full = j0 + kTile - 1 <= p_lo &&
                          (window == 0 || j0 > p_hi - window || j0 + kTile <= nfirst);
        // P buffer s is free once the PV of tile g - 2 is done (long before the scores are)
        if (g >= 2) warp_wait(pv_done((g - 2) % KS, HV - 1), ((g - 2) / KS) & 1, wc);
        warp_wait(bar(kSFull0 + s), (g >> 1) & 1, wc);
        tc_fence_after();
        float x[kE];
        {
          const uint32_t ta = tmem + lane_base + s * 64 + kPos * hc;
          uint32_t v[kE];
          if constexpr (kReps == 4) {
            tmem_ld_16x256b_x4(ta, v);
          } else {
            static_assert(kReps == 3, "24 positions");
            uint32_t v2[8], v1[4];
            tmem_ld_16x256b_x2(ta, v2);
            tmem_ld_16x256b_x1(ta + 16, v1);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < kE; ++e) v[e] = e < 8 ? v2[e] : v1[e - 8];
          }
          if constexpr (kReps == 4) tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < kE; ++e) x[e] = __uint_as_float(v[e]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kSEmpty0 + s));
        uint32_t see = 0xffffu;  // bit e: row and position of element e see each other
        bool poison = false;     // a score that is masked and not finite
        if (!full) {
          see = 0;
#pragma unroll
          for (int e = 0; e < kE; ++e) {
            const int j = j0 + kPos * hc + 8 * (e >> 2) + 2 * tq + (e & 1);
            const int pos = (e & 3) < 2 ? posA : posB;
            const bool ok = j <= pos && (window == 0 || j > pos - window || j < nfirst);
            see |= ok ? 1u << e : 0u;
            poison |= !ok && !(fabsf(x[e]) < INFINITY);
          }
          // A cached row with an infinity or NaN that some row of this tile
          // does not see: its weight there is 0, but 0 x inf = NaN in the MMA.
          // Such rows are cleared in shared memory (the rows that do see it
          // have a NaN weight already, or 0 where the score is -inf), after the QK MMAs
          // have read them.
          if (named_bar_or(1, kSmThreads, poison)) {
            uint8_t* stage = smem + C::kOffKV + (g % KS) * C::kStage;
            const int r = st >> 2, part = st & 3;  // 4 threads per cached row
            auto chunk = [&](int ch) {  // 16 bytes of the row
              const int pn = ch >> 3;
              return reinterpret_cast<uint4*>(stage + pn / C::kPanelsH * C::kHalf + (r >> 3) * C::kGroup +
                                              pn % C::kPanelsH * 1024 + (r & 7) * 128 +
                                              (((ch & 7) ^ (r & 7)) << 4));
            };
            uint32_t bad = 0;
            for (int ch = part; ch < D / 8 && r < kTile; ch += 4) {
              const uint4 w = *chunk(ch);
              const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int e = 0; e < 4; ++e)
                bad |= (ws[e] & 0x7f80u) == 0x7f80u || (ws[e] & 0x7f800000u) == 0x7f800000u;
            }
            bad |= __shfl_xor_sync(0xffffffffu, bad, 1);
            bad |= __shfl_xor_sync(0xffffffffu, bad, 2);
            for (int ch = part; bad && ch < D / 8; ch += 4)
              *chunk(ch) = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();  // read by the PV MMA, issued after a later barrier
          }
        }
        // p = 2^(x scale - m) in bf16 into rows hA, hB of P (K-major, 128-byte
        // swizzle) with two stmatrix.x4.  The MMA multiplies the rounded p, the
        // denominator sums the unrounded ones: each weight is off by at most
        // 2^-8 of itself, as the output's own rounding, and lse has none.
        const uint32_t prow = sP + s * C::kPBytes + (2 * q4) * 1024 + (lane & 7) * 128;
        auto pchunk = [&](int c) {  // this lane's address of a matrix of stmatrix: chunk c of its row
          return prow + (uint32_t)(((kReps * hc + c) ^ (lane & 7)) << 4);
        };
        float sumA, sumB;
        // (rows past the unit's end have factor 0: their weights, never used, stay finite
        // and cast no vote)
        auto weights = [&](auto masked) {
          float top = -INFINITY;
          sumA = sumB = 0.f;
          uint32_t pa[kReps], pb[kReps];
#pragma unroll
          for (int rep = 0; rep < kReps; ++rep) {
            float e[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float arg = fmaf(x[4 * rep + k], k < 2 ? scA : scB, -((k < 2) ? mA : mB));
              const bool ok = !decltype(masked)::value || ((see >> (4 * rep + k)) & 1u);
              top = fmaxf(top, ok ? arg : -INFINITY);
              e[k] = ok ? ex2_approx(arg) : 0.f;
            }
            sumA += e[0] + e[1];
            sumB += e[2] + e[3];
            const __nv_bfloat162 a = __floats2bfloat162_rn(e[0], e[1]);
            const __nv_bfloat162 b = __floats2bfloat162_rn(e[2], e[3]);
            pa[rep] = *reinterpret_cast<const uint32_t*>(&a);
            pb[rep] = *reinterpret_cast<const uint32_t*>(&b);
          }
          if (held) {
            if constexpr (kReps == 4) {
              stmatrix_x4(pchunk(lane >> 3), pa[0], pa[1], pa[2], pa[3]);
              stmatrix_x4(pchunk(lane >> 3) + 1024, pb[0], pb[1], pb[2], pb[3]);
            } else {
              stmatrix_x2(pchunk((lane >> 3) & 1), pa[0], pa[1]);
              stmatrix_x1(pchunk(2), pa[2]);
              stmatrix_x2(pchunk((lane >> 3) & 1) + 1024, pb[0], pb[1]);
              stmatrix_x1(pchunk(2) + 1024, pb[2]);
            }
          }
          return top > kHeadroom;
        };
        // The first tile of a piece sets m to its exact row maxima; a later one
        // is weighted against the current m, and only if a score exceeds it by
        // the headroom do the warps raise m and rescale O^T (p stays below 2^8).
        bool exact = i == i0;
        if (!exact) {
          const bool over = full ? weights(std::false_type{}) : weights(std::true_type{});
          fence_proxy_async_smem();
          exact = named_bar_or(1, kSmThreads, over);
        }
        if (exact) {
          float eA = -INFINITY, eB = -INFINITY;
#pragma unroll
          for (int e = 0; e < kE; ++e) {
            if ((see >> e) & 1u) {
              if ((e & 3) < 2) eA = fmaxf(eA, x[e] * scA);
              else eB = fmaxf(eB, x[e] * scB);
            }
          }
#pragma unroll
          for (int o = 1; o <= 2; o <<= 1) {
            eA = fmaxf(eA, __shfl_xor_sync(0xffffffffu, eA, o));
            eB = fmaxf(eB, __shfl_xor_sync(0xffffffffu, eB, o));
          }
          {  // the other half of the tile: warp w ^ 4
            float* hm = s_hmax + (g & 1) * 128;
            if (tq == 0) {
              hm[hc * 64 + hA] = eA;
              hm[hc * 64 + hB] = eB;
            }
            named_bar_sync(2 + q4, 64);
            eA = fmaxf(eA, hm[(hc ^ 1) * 64 + hA]);
            eB = fmaxf(eB, hm[(hc ^ 1) * 64 + hB]);
          }
          float alphaA = 1.f, alphaB = 1.f;
          if (eA > mA + kHeadroom) {
            alphaA = ex2_approx(mA - eA);  // 0 when there was no score
            lA *= alphaA;
            mA = eA;
          }
          if (eB > mB + kHeadroom) {
            alphaB = ex2_approx(mB - eB);
            lB *= alphaB;
            mB = eB;
          }
          weights(std::true_type{});
          fence_proxy_async_smem();
          if (i > i0) {
            if (tq == 0 && hc == 0) {
              s_alpha[hA] = alphaA;
              s_alpha[hB] = alphaB;
            }
            named_bar_sync(1, kSmThreads);
            // O^T must be quiescent: wait for the PV of tile g - 1
            warp_wait(pv_done((g - 1) % KS, HV - 1), ((g - 1) / KS) & 1, wc);
            __syncwarp();
            tc_fence_after();
#pragma unroll 1
            for (int b = hc; b < C::kBlocks; b += 2) {
#pragma unroll 1
              for (int c = 0; c < R / 16; ++c) {
                uint32_t ov[16];
                const uint32_t ta = tmem + lane_base + C::kOCol + b * R + c * 16;
                tmem_ld16(ta, ov);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e)
                  ov[e] = __float_as_uint(__uint_as_float(ov[e]) * s_alpha[c * 16 + e]);
                tmem_st16(ta, ov);
              }
            }
            tmem_wait_st();
          }
          tc_fence_before();
          named_bar_sync(1, kSmThreads);
        }
        lA += sumA;
        lB += sumB;
        // the last barrier (the vote, or the exact path's) has seen every warp's P
        if (st == 0) mbar_arrive(bar(kPReady0 + s));
      }
      // ---------------------------------------------- end of the piece
      lA += __shfl_xor_sync(0xffffffffu, lA, 1);
      lA += __shfl_xor_sync(0xffffffffu, lA, 2);
      lB += __shfl_xor_sync(0xffffffffu, lB, 1);
      lB += __shfl_xor_sync(0xffffffffu, lB, 2);
      // (the last tile's barrier lies behind every read of s_alpha, which s_lsum aliases)
      if (tq == 0) {
        s_lsum[hc * 64 + hA] = lA;
        s_lsum[hc * 64 + hB] = lB;
      }
      warp_wait(pv_done((g - 1) % KS, HV - 1), ((g - 1) / KS) & 1, wc);
      __syncwarp();
      tc_fence_after();
      named_bar_sync(1, kSmThreads);
      const int slot = 2 * (int)blockIdx.x + (i0 == 0 ? 1 : 0);
      if (tq == 0 && hc == 0) {
#pragma unroll
        for (int w2 = 0; w2 < 2; ++w2) {
          const int r = w2 ? hB : hA;
          if (r >= R) continue;
          const float mw = w2 ? mB : mA, m = mw == kNoScore ? -INFINITY : mw;
          const float l = s_lsum[r] + s_lsum[64 + r];  // read before fac[r] overwrites s_lsum[64 + r]
          float f = 0.f;
          if (whole) {
            if (w2 ? vB : vA) {
              const float ms = (w2 ? sinkB : sinkA) * kLog2e;
              const float M = fmaxf(m, ms);
              float lse = M * kLn2;
              if (M != -INFINITY && ms != INFINITY) {
                const float a = m == -INFINITY ? 0.f : ex2_approx(m - M);
                const float den = fmaf(l, a, ex2_approx(ms - M));
                f = a / den;
                lse = (M + log2f(den)) * kLn2;
              }
              // (the sink alone: as it is; a NaN that was seen: NaN)
              p.lse[un.row0 + r] = l != l ? l : (m == -INFINITY ? (w2 ? sinkB : sinkA) : lse);
            }
          } else {
            p.part_ml[(size_t)slot * R + r] = make_float2(m, l);
          }
          s_fac[r] = f;
        }
      }
      named_bar_sync(1, kSmThreads);
      if (whole) {
        // block by block of O^T through the P buffers: scaled, packed to bf16 and
        // transposed with stmatrix into two boxes of R rows x 64 columns, then row
        // by row to out.  Warp w takes 32 rows of D (q4) and half hc of the rows.
        uint8_t* stg = smem + C::kOffP;
        constexpr int kRc = R == 16 ? 16 : 32;
        const bool mine = R > 16 || hc == 0;
        const int r0 = R > 16 ? hc * kRc : 0;
        float fac[kRc / 4];
#pragma unroll
        for (int rep = 0; rep < kRc / 8; ++rep) {
          fac[2 * rep] = s_fac[r0 + 8 * rep + 2 * tq];
          fac[2 * rep + 1] = s_fac[r0 + 8 * rep + 2 * tq + 1];
        }
#pragma unroll 1
        for (int b = 0; b < C::kBlocks; ++b) {
          if (mine) {
            uint32_t rr[2][kRc / 2];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const uint32_t ta =
                  tmem + ((uint32_t)(q4 * 32 + 16 * half) << 16) + C::kOCol + b * R + r0;
              if constexpr (kRc == 32) tmem_ld_16x256b_x4(ta, rr[half]);
              else tmem_ld_16x256b_x2(ta, rr[half]);
            }
            tmem_wait_ld();
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              uint32_t pk[kRc / 4];
#pragma unroll
              for (int rep = 0; rep < kRc / 8; ++rep) {
#pragma unroll
                for (int dg = 0; dg < 2; ++dg) {
                  // "+ 0.f" turns -0 into +0 when the factor is 0 (sink = +inf)
                  const __nv_bfloat162 v2 = __floats2bfloat162_rn(
                      __uint_as_float(rr[half][4 * rep + 2 * dg]) * fac[2 * rep] + 0.f,
                      __uint_as_float(rr[half][4 * rep + 2 * dg + 1]) * fac[2 * rep + 1] + 0.f);
                  pk[2 * rep + dg] = *reinterpret_cast<const uint32_t*>(&v2);
                }
              }
              const int mt = lane >> 3, jr = lane & 7;
              const int dl = q4 * 32 + 16 * half + 8 * (mt & 1);
              const int box = dl >> 6, chunk = (dl & 63) >> 3;
#pragma unroll
              for (int rep0 = 0; rep0 < kRc / 8; rep0 += 2) {
                const int r = r0 + 8 * (rep0 + (mt >> 1)) + jr;
                stmatrix_x4_trans(smem_addr(stg) + box * (R * 128) + r * 128 + ((chunk ^ (r & 7)) << 4),
                                  pk[2 * rep0], pk[2 * rep0 + 1], pk[2 * rep0 + 2], pk[2 * rep0 + 3]);
              }
            }
          }
          named_bar_sync(1, kSmThreads);
          constexpr int kW = D < 128 ? D / 8 : 16;  // 16-byte chunks of a row of this block
          for (int e = st; e < un.nrows * kW; e += kSmThreads) {
            const int r = e / kW, ch = e % kW;
            const uint4 w = *reinterpret_cast<const uint4*>(stg + (ch >> 3) * (R * 128) + r * 128 +
                                                            (((ch & 7) ^ (r & 7)) << 4));
            *reinterpret_cast<uint4*>(p.out + (size_t)(un.row0 + r) * D + b * 128 + ch * 8) = w;
          }
          named_bar_sync(1, kSmThreads);  // the area may be rewritten
        }
      } else {
#pragma unroll 1
        for (int b = hc; b < C::kBlocks; b += 2) {
          const int d = b * 128 + q4 * 32 + lane;
#pragma unroll 1
          for (int c = 0; c < R / 16; ++c) {
            uint32_t ov[16];
            tmem_ld16(tmem + lane_base + C::kOCol + b * R + c * 16, ov);
            tmem_wait_ld();
            float* o = p.part_o + ((size_t)slot * R + c * 16) * D + d;
            if (d < D) {
#pragma unroll
              for (int e = 0; e < 16; ++e) o[(size_t)e * D] = __uint_as_float(ov[e]);
            }
          }
        }
      }
      tc_fence_before();
      named_bar_sync(1, kSmThreads);
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kQkWarp) tmem_dealloc(tmem, C::kTmemCols);
}

template <typename F>
cudaError_t for_shape(int R, int D, bool tma, F&& f) {
#define SDA_CASE(RV, DV)                                                                   \
  if (R == RV && D == DV)                                                                  \
    return tma ? f(chunk_attn_kernel<RV, DV, true>, (size_t)Cfg<RV, DV>::kSmem, dim3(384)) \
               : f(chunk_attn_kernel<RV, DV, false>, (size_t)Cfg<RV, DV>::kSmem,           \
                   dim3(kGatherThreads));
  SDA_CASE(16, 64) SDA_CASE(16, 128) SDA_CASE(16, 256) SDA_CASE(16, 512)
  SDA_CASE(64, 64) SDA_CASE(64, 128) SDA_CASE(64, 256) SDA_CASE(64, 512)
#undef SDA_CASE
  return cudaErrorInvalidValue;
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

}  // namespace

static EncodeTiledFn encode_fn() {
  static const EncodeTiledFn fn = []() -> EncodeTiledFn {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    return reinterpret_cast<EncodeTiledFn>(f);
  }();
  return fn;
}

bool pipe_map_2d(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows, uint32_t box_cols,
                 uint32_t box_rows) {
  const cuuint64_t dims[2] = {cols, rows}, strides[1] = {cols * 2};
  const cuuint32_t box[2] = {box_cols, box_rows}, estr[2] = {1, 1};
  return encode_fn() &&
         encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides,
                     box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool pipe_map_pool(CUtensorMap* m, const void* base, uint64_t D, uint64_t groups, uint32_t panels,
                   uint32_t box_groups) {
  const cuuint64_t dims[4] = {64, 8, D / 64, groups}, strides[3] = {D * 2, 128, D * 16};
  const cuuint32_t box[4] = {64, 8, panels, box_groups}, estr[4] = {1, 1, 1, 1};
  return encode_fn() &&
         encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides,
                     box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// setmaxnreg.inc waits until the other warps have released registers: a build
// whose launch allocation is smaller than the split assumes is never launched.
cudaError_t chunk_prepare() {
  for (int R : {16, 64}) {
    for (int D : {64, 128, 256, 512}) {
      for (bool tma : {false, true}) {
        const cudaError_t e = for_shape(R, D, tma, [&](auto kernel, size_t smem, dim3) {
          cudaError_t r =
              cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
          cudaFuncAttributes a;
          if (r == cudaSuccess) r = cudaFuncGetAttributes(&a, kernel);
          if (r == cudaSuccess && !tma && a.numRegs < kGatherRegs) r = cudaErrorInvalidConfiguration;
          return r;
        });
        if (e != cudaSuccess) return e;
      }
    }
  }
  return pair_prepare();
}

ChunkParams chunk_params(const void* kv, const ChunkGeom& g, const float* attn_sink, float scale,
                         void* out, float* lse, const ChunkLayout& L, void* ws) {
  char* base = static_cast<char*>(ws);
  ChunkParams p;
  p.kv = static_cast<const __nv_bfloat16*>(kv);
  p.attn_sink = attn_sink;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.hdr = reinterpret_cast<ChunkHeader*>(base);
  p.starts = reinterpret_cast<ChunkStart*>(base + L.start_off);
  p.recs = reinterpret_cast<ChunkUnit*>(base + L.rec_off);
  p.mode = L.mode;
  p.workers = L.grid;
  p.part_ml = reinterpret_cast<float2*>(base + L.ml_off);
  p.part_o = reinterpret_cast<float*>(base + L.o_off);
  p.g = g;
  p.qk_scale_log2 = scale * kLog2e;
  p.wait_timeout_ns = current_wait_fault().timeout_ns;
  return p;
}

cudaError_t launch_chunk_attn(const void* q, const void* kv, const ChunkGeom& g,
                              const float* attn_sink, float scale, void* out, float* lse,
                              const ChunkLayout& L, void* ws, cudaStream_t st) {
  const bool tma = chunk_boxes(g);
  const ChunkParams p = chunk_params(kv, g, attn_sink, scale, out, lse, L, ws);
  CUtensorMap tq, tkv = {};
  if (!pipe_map_2d(&tq, q, g.D, (uint64_t)g.T * g.H, 64, L.pair ? L.R / 2 : L.R) ||
      (tma && !pipe_map_pool(&tkv, p.kv + g.base * g.D, g.D, (uint64_t)(g.total_pages - g.base) / 8,
                             g.D >= 256 ? g.D / 128 : g.D / 64, 2)))
    return cudaErrorInvalidValue;
  if (L.pair) return launch_chunk_pair(tq, tkv, p, tma, L, st);
  return for_shape(L.R, g.D, tma, [&](auto kernel, size_t smem, dim3 threads) {
    return launch_pdl(kernel, dim3(L.grid), threads, smem, st, tq, tkv, p);
  });
}

}  // namespace sda
