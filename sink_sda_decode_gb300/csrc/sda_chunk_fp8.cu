// sda_chunk_fp8.cu -- chunk attention over a cache of E4M3 codes with a scale for each
// block (tcgen05 / TMEM): one CTA a tile of queries.
//
// The operator and its tiles are those of sda_chunk_attn.cu (S = Q K^T with M = 64 rows,
// O^T += V^T P^T with M = 128 of D, a cached row key and value from the same shared tile);
// the numbers are sda_chunk_fp8.cuh's.  What differs is how a tile comes to shared memory:
// eight warps load its codes row by row into registers a tile (or a few) ahead, and write
// them as f16 into the tile's swizzled place once the MMAs that last read it are done.
// So blocks of any size take the same way, and a cached row costs shared memory no more
// bandwidth than its f16 form does.
// One token of 64 heads over 8 caches of 16384 to 65536 positions, D = 512 (183 MB of codes):
// 92 us, 2.0 TB/s.  A tile of 64 positions takes 3250 cycles, 2700 of them MMAs; the loaders'
// loop is the period (600 to convert and store, up to 1900 until the next tile's loads are
// issued: with 208 KB of shared memory in use L1 holds few of them in flight).  Tiles of 48 in three
// stages took 98 us; loads issued between the stores, so in front of the fence, 97.
// Roles:
//   warps 0..7    softmax and epilogue
//   warp 8        QK MMAs and the q loads (TMA)
//   warp 9        PV MMAs
//   warps 10, 11  q from bf16 to f16, in place
//   warps 12..19  KV tiles
#include <cuda_bf16.h>

#include <type_traits>

#include "sda_chunk_fp8.cuh"

namespace sda {

namespace {

using namespace ptx;

constexpr int kSmWarps = 8;
constexpr int kSmThreads = kSmWarps * 32;
constexpr int kQkWarp = 8, kPvWarp = 9, kQWarp0 = 10, kQWarps = 2, kLoadWarp0 = 12, kLoadWarps = 8;
constexpr int kMaxStages = 6;
// 640 threads launch with 96 registers each, which the loaders keep; the softmax warps grow
// to 104 and the others shrink to 80.  (Nothing is spilled: L1, beside 227 KB of shared
// memory, would not hold it.)
constexpr int kThreads = 640, kRegs = 96;
static_assert(kSmThreads * 104 + kLoadWarps * 32 * 96 + 128 * 80 <= kThreads * kRegs,
              "register split exceeds the launch allocation");

enum Bar : int {
  kQFull = 0,
  kQReady,
  kQEmpty,
  kSFull0,
  kSEmpty0 = kSFull0 + 2,
  kPReady0 = kSEmpty0 + 2,
  kDrainQk = kPReady0 + 2,
  kDrainPv,
  kKvFull0,
  kPvDone0 = kKvFull0 + kMaxStages,
  kBars = kPvDone0 + kMaxStages
};

template <int R, int D>
struct Cfg {
  static constexpr int kTile = 64;
  static constexpr int kPanels = D / 64;
  static constexpr int kBlocks = (D + 127) / 128;  // 128-row blocks of O^T
  static constexpr int kGroup = kPanels * 1024;    // 8 rows of a stage: [panels][1 KB atom]
  static constexpr int kStage = kTile / 8 * kGroup;
  static constexpr int kStages = D == 512 ? (R == 64 ? 2 : 3) : (D == 256 ? 5 : 6);
  // the loaders' share of a tile, in 16-byte loads, and how many tiles ahead they are
  static constexpr int kRows = kTile / kLoadWarps, kLanes = D / 16, kRowsPer = 32 / kLanes;
  static constexpr int kLoads = (kRows + kRowsPer - 1) / kRowsPer;
  static constexpr int kAhead = kLoads >= 8 ? 1 : (kLoads >= 4 ? 2 : 4);
  static constexpr int kPanelQ = R * 128;
  static constexpr int kPBytes = R * 128;
  static constexpr int kOffQ = 0;
  static constexpr int kOffKV = kPanels * kPanelQ;
  static constexpr int kOffP = kOffKV + kStages * kStage;  // two P buffers; the epilogue's staging
  static constexpr int kOffBar = kOffP + 2 * kPBytes;
  static constexpr int kOffMisc = kOffBar + (8 * kBars + 15) / 16 * 16;
  static constexpr int kOffAlpha = kOffMisc + 16;       // float [64]
  // float [2][64]: maxima within a tile; at the end of a piece the sums, then (the second
  // half) the factors
  static constexpr int kOffHMax = kOffAlpha + 4 * 64;
  static constexpr int kOffScale = kOffHMax + 4 * 128;  // float [stages][kTile]: kWeightUnit s_j
  static constexpr int kOffQs = kOffScale + 4 * kTile * kStages;  // [4 pieces][64]: exponents of q's 2^-k
  // As in sda_chunk_attn.cu, the QK MMA reads 64 rows of a q panel and the PV MMA 128
  // columns of D whatever R and D are; what lies behind lands in lanes that nothing reads.
  static constexpr int kUsed = kOffQs + 256;
  static constexpr int kSmem = kUsed + 1024;
  static constexpr int kOCol = 128;
  static constexpr int kTmemCols = kOCol + kBlocks * R <= 256 ? 256 : 512;
  static constexpr uint32_t kIdescQK = idesc_f16_f32(64, kTile, false);
  static constexpr uint32_t kIdescPV = idesc_f16_f32(128, R, true);
  static_assert(kOCol + kBlocks * R <= 512, "TMEM columns");
  static_assert(kOffKV % 1024 == 0 && kOffP % 1024 == 0 && kPBytes % 1024 == 0, "swizzle atoms");
  static_assert((kPanels - 1) * kPanelQ + 64 * 128 <= kOffBar, "padded QK operand inside smem");
  static_assert(D >= 128 || 2 * kPBytes >= 1024, "padded PV operand inside smem");
  static_assert(kTile % 16 == 0 && kTile <= 64, "MMA shapes");
  static_assert(kStages * kStage >= 4 * (kFusedSeqs + 1), "chunk_begin's words");
  static_assert(kRows % kRowsPer == 0 || kRowsPer > kRows || kRowsPer == 1, "rows of a load");
  static_assert(kSmem <= 232448, "shared memory budget");
};

template <int R, int D>
__global__ void __launch_bounds__(kThreads, 1)
chunk_fp8_kernel(const __grid_constant__ CUtensorMap tmap_q, const ChunkFp8Params fp) {
  using C = Cfg<R, D>;
  const ChunkParams& p = fp.c;
  constexpr int KS = C::kStages;
  constexpr int kTile = C::kTile;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_addr(smem);
  const uint32_t sQ = sbase + C::kOffQ, sKV = sbase + C::kOffKV, sP = sbase + C::kOffP;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  float* s_scale = reinterpret_cast<float*>(smem + C::kOffScale);
  uint8_t* s_qs = smem + C::kOffQs;
  auto bar = [&](int i) { return sbase + C::kOffBar + 8u * (uint32_t)i; };
  auto kv_full = [&](int s) { return bar(kKvFull0 + s); };
  auto pv_done = [&](int s) { return bar(kPvDone0 + s); };

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(bar(kQFull), 1);
    mbar_init(bar(kQReady), kQWarps);
    mbar_init(bar(kQEmpty), 1);
    for (int s = 0; s < KS; ++s) {
      mbar_init(kv_full(s), kLoadWarps);
      mbar_init(pv_done(s), 1);
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
  const ChunkStart begin =
      chunk_begin<kThreads, R, kTile>(p, blockIdx.x, reinterpret_cast<int*>(smem + C::kOffKV),
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

  // A share of q of piece n from bf16 to f16, in place: warp w of `among`.  With the first
  // piece, which everything waits for, the softmax warps help the two whose work it is.
  auto q_to_f16 = [&](int n, int w, int among) {
    constexpr int kQLanes = D / 8 < 32 ? D / 8 : 32, kQRows = 32 / kQLanes;  // rows of a pass
#pragma unroll 1
    for (int r0 = w * kQRows; r0 < R; r0 += among * kQRows) {
      const int r = r0 + lane / kQLanes;
      const uint32_t down = q_row_to_f16<D>(
          [&](int ch) {
            return reinterpret_cast<uint4*>(smem + C::kOffQ + (ch >> 3) * C::kPanelQ + r * 128 +
                                            (((ch & 7) ^ (r & 7)) << 4));
          },
          lane);
      if (lane % kQLanes == 0) s_qs[(n & 3) * 64 + r] = (uint8_t)down;
    }
    fence_proxy_async_smem();
    __syncwarp();
  };

  if (warp >= kQkWarp && warp < kLoadWarp0) setmaxnreg_dec<80>();
  if (warp >= kLoadWarp0) {
    // ===================================================== KV tiles
    // A load takes four lanes' 64 codes, half a panel's row, of a row and of the next in
    // turn: eight lanes' stores then meet all banks.
    constexpr int NL = C::kLoads, NA = C::kAhead;
    constexpr int kGroups = D / 64;  // 64 codes of a row
    const int v = warp - kLoadWarp0, q = lane >> 2;
    auto row_of = [&](int i) {  // of this lane's codes in load i
      return kGroups == 1 ? i * 8 + q
                          : i * 8 / (2 * kGroups) * 2 + (kGroups < 4 ? q / (2 * kGroups) * 2 : 0) + (q & 1);
    };
    auto group_of = [&](int i) { return kGroups == 1 ? 0 : (i * 8 % (2 * kGroups) + q % (2 * kGroups)) >> 1; };
    uint4 x[NA][NL];
    float sc[NA];  // lane < kRows: kWeightUnit times the scale of row kRows v + lane
    Walk c;        // runs kAhead + 2 tiles ahead of the stores
    c.init(p.g, begin);
    int slot = -1;  // lane < kRows: the next tile's rows
    float sc_next = 0.f;
    // The tile after that: its table entries are under way while this one's rows are read.
    int at_b = -1, at_blk = 0;  // row in the block, or -1; the block
    auto look_up = [&]() {
      slot = -1;
      sc_next = 0.f;
      if (at_b >= 0) {
        const long long row = p.g.base + (long long)at_blk * p.g.k_per_block + at_b;
        if (at_blk < 0 || row >= p.g.total_pages) {
          atomicExch(error, 3);
        } else {
          slot = (int)row;
          sc_next = __ldg(fp.scale + at_blk) * kWeightUnit;
          // (the row's load follows a tile later)
#pragma unroll
          for (int b = 0; b < D; b += 128) prefetch_line(fp.codes + (size_t)slot * D + b);
        }
      }
      at_b = -1;
      if (c.left > 0) {
        const int j = c.start() + v * C::kRows + lane;
        if (lane < C::kRows && j < c.hi && (j >= c.lo || j < p.g.first)) {
          const int jb = (int)(((unsigned long long)(unsigned)j * fp.k_mul) >> fp.k_shift);
          at_blk = __ldg(p.g.block_table + (size_t)c.b * p.g.max_blocks + jb);
          at_b = j - jb * p.g.k_per_block;
        }
        c.next(p.g);
      }
    };
    auto load = [&](uint4& to, int i) {
      const int rl = row_of(i);
      const int from = __shfl_sync(0xffffffffu, slot, rl & 31);
      to = make_uint4(0, 0, 0, 0);
      if (from >= 0 && rl < C::kRows)
        to = load_codes(fp.codes + (size_t)from * D + group_of(i) * 64 + (lane & 3) * 16);
    };
    look_up();
    look_up();
#pragma unroll
    for (int a = 0; a < NA; ++a) {
#pragma unroll
      for (int i = 0; i < NL; ++i) load(x[a][i], i);
      sc[a] = sc_next;
      look_up();
    }
    bool ok = true;
    for (int g0 = 0; g0 < nt && ok; g0 += NA) {
#pragma unroll
      for (int a = 0; a < NA; ++a) {
        const int g = g0 + a;
        if (g >= nt || !ok) break;
        const int s = g % KS;
        if (g >= KS) ok = tile_wait(pv_done(s), ((g / KS) - 1) & 1, wc);
        if (!ok) break;
        const uint32_t stage = sKV + s * C::kStage;
#pragma unroll
        for (int i = 0; i < NL; ++i) {
          const uint4 w = x[a][i];
          uint32_t h[8];
          codes_to_f16(w.x, h[0], h[1]);
          codes_to_f16(w.y, h[2], h[3]);
          codes_to_f16(w.z, h[4], h[5]);
          codes_to_f16(w.w, h[6], h[7]);
          const int rl = row_of(i), r = v * C::kRows + rl, ch = 2 * (lane & 3);
          const uint32_t row = stage + (r >> 3) * C::kGroup + group_of(i) * 1024 + (r & 7) * 128;
          if (rl < C::kRows) {
            st_shared16(row + ((ch ^ (r & 7)) << 4), h[0], h[1], h[2], h[3]);
            st_shared16(row + (((ch ^ 1) ^ (r & 7)) << 4), h[4], h[5], h[6], h[7]);
          }
        }
        if (lane < C::kRows) s_scale[s * kTile + v * C::kRows + lane] = sc[a];
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(kv_full(s));
        // Tile g + kAhead, behind the fence: that waits for a thread's loads, too.
#pragma unroll
        for (int i = 0; i < NL; ++i) load(x[a][i], i);
        sc[a] = sc_next;
        look_up();
      }
    }
  } else if (warp >= kQWarp0 && warp < kQWarp0 + kQWarps) {
    // ===================================================== q from bf16 to f16
    int pieces = 0;
    UnitWalk uw;
    uw.init(p.g, R, begin);
    for (int g = 0; g < nt; ++pieces) {
      if (pieces > 0) uw.next(p.g, R);
      const ChunkUnit un = chunk_unit(p.g, R, kTile, uw.b, uw.r);
      const int i0 = g == 0 ? begin.off : 0;
      g += min(un.ntiles, i0 + nt - g) - i0;
      const bool ok = tile_wait(bar(kQFull), pieces & 1, wc);
      if (ok) q_to_f16(pieces, warp - kQWarp0, pieces == 0 ? kQWarps + kSmWarps : kQWarps);
      if (pieces == 0) named_bar_sync(6, kSmThreads + kQWarps * 32);
      if (!ok) break;
      if (lane == 0) mbar_arrive(bar(kQReady));
    }
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
      if (g >= 2) ok = tile_wait(bar(kSEmpty0 + s), ((g >> 1) - 1) & 1, wc);
      if (ok && c.first) ok = tile_wait(bar(kQReady), pieces & 1, wc);
      if (ok) ok = tile_wait(kv_full(ks), (g / KS) & 1, wc);
      if (!ok) break;
      tc_fence_after();
      const uint64_t b0 = sdesc_sw128(sKV + ks * C::kStage, 16, C::kGroup);
      const bool last = c.last();
      if (elect_one()) {
#pragma unroll
        for (int x = 0; x < C::kPanels; ++x) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_bf16(tmem + s * 64, sdesc_advance(a0, x * C::kPanelQ + k * 32),
                     sdesc_advance(b0, x * 1024 + k * 32), C::kIdescQK, (x || k) ? 1u : 0u);
        }
        mma_commit(bar(kSFull0 + s));
        if (last) mma_commit(bar(kQEmpty));
      }
      __syncwarp();
      c.next(p.g);
      if (last) {
        if (c.left > 0) {  // q of the next unit, once this unit's MMAs have read q
          ok = tile_wait(bar(kQEmpty), pieces & 1, wc);
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
      if (!tile_wait(bar(kPReady0 + s), (g >> 1) & 1, wc)) break;
      tc_fence_after();
      const uint64_t a0 = sdesc_sw128(sKV + ks * C::kStage, 1024, C::kGroup);
      const uint64_t b0 = sdesc_sw128(sP + s * C::kPBytes, 16, 1024);
      const uint32_t add = c.first ? 0u : 1u;
      if (elect_one()) {
#pragma unroll
        for (int b = 0; b < C::kBlocks; ++b) {
#pragma unroll
          for (int k = 0; k < kTile / 16; ++k)
            mma_bf16(tmem + C::kOCol + b * R, sdesc_advance(a0, 2 * b * 1024 + k * 2 * C::kGroup),
                     sdesc_advance(b0, k * 32), C::kIdescPV, k ? 1u : add);
        }
        mma_commit(pv_done(ks));
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
    setmaxnreg_inc<104>();
    // Warp w reads TMEM lane quadrant q4 = w % 4 and half hc = w / 4 of each
    // tile's positions: thread t holds rows hA = 16 q4 + t / 4 and hB = hA + 8 at
    // the positions kPos hc + 8 rep + 2 (t % 4) + {0, 1}.
    constexpr int kPos = kTile / 2, kReps = kPos / 8, kE = 4 * kReps;
    static_assert(kReps == 4, "loads and stores of 32 positions");
    const int q4 = warp & 3, hc = warp >> 2, st = threadIdx.x, tq = lane & 3;
    const int hA = q4 * 16 + (lane >> 2), hB = hA + 8;
    const uint32_t lane_base = (uint32_t)(q4 * 32) << 16;
    float* s_alpha = reinterpret_cast<float*>(smem + C::kOffAlpha);
    float* hm = reinterpret_cast<float*>(smem + C::kOffHMax);
    float* s_lsum = hm;
    float* s_fac = hm + 64;
    const float sc = p.qk_scale_log2 / kWeightUnit;
    const int H = p.g.H, window = p.g.window, nfirst = p.g.first;
    const bool held = hA < R;  // this warp's rows exist in P (uniform over the warp)
    // Control flow is the same in the eight warps (it depends on the plan and
    // on block-wide votes), so every named barrier is reached by all of them
    // even after a wait timed out.
    int g = 0;
    if (nt > 0) {  // (nothing else to do until the first scores come)
      if (tile_wait(bar(kQFull), 0, wc)) q_to_f16(0, kQWarps + warp, kQWarps + kSmWarps);
      named_bar_sync(6, kSmThreads + kQWarps * 32);
    }
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
      float scA = 0.f, scB = 0.f;
      float mA = kNoScore, mB = kNoScore, lA = 0.f, lB = 0.f;  // l: this thread's share
      for (int i = i0; i < i1; ++i, ++g) {
        const int s = g & 1;
        const int j0 = chunk_tile_start(i, un.nf, un.lo, kTile);
        // whether every row of the unit sees the whole tile
        const bool full = j0 + kTile - 1 <= p_lo &&
                          (window == 0 || j0 > p_hi - window || j0 + kTile <= nfirst);
        // P buffer s is free once the PV of tile g - 2 is done (long before the scores are)
        if (g >= 2) tile_wait(pv_done((g - 2) % KS), ((g - 2) / KS) & 1, wc);
        tile_wait(bar(kSFull0 + s), (g >> 1) & 1, wc);
        tc_fence_after();
        // (the scores' MMAs waited for q's and the tile's factors, too)
        if (i == i0) {
          scA = vA ? sc * q_factor(s_qs[(pieces & 3) * 64 + hA]) : 0.f;
          scB = vB ? sc * q_factor(s_qs[(pieces & 3) * 64 + hB]) : 0.f;
        }
        float sj[2 * kReps];  // kWeightUnit s_j of this thread's positions
#pragma unroll
        for (int rep = 0; rep < kReps; ++rep) {
          const float2 f =
              *reinterpret_cast<const float2*>(s_scale + (g % KS) * kTile + kPos * hc + 8 * rep + 2 * tq);
          sj[2 * rep] = f.x;
          sj[2 * rep + 1] = f.y;
        }
        float x[kE];
        {
          const uint32_t ta = tmem + lane_base + s * 64 + kPos * hc;
          uint32_t v[kE];
          tmem_ld_16x256b_x4(ta, v);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < kE; ++e) x[e] = __uint_as_float(v[e]) * sj[2 * (e >> 2) + (e & 1)];
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
          // A cached row with a NaN that some row of this tile does not see: its weight
          // there is 0, but 0 x NaN = NaN in the MMA.  Such rows are cleared in shared
          // memory (the rows that do see it have a NaN weight already), after the QK
          // MMAs have read them.
          if (named_bar_or(1, kSmThreads, poison)) {
            uint8_t* stage = smem + C::kOffKV + (g % KS) * C::kStage;
            const int r = st >> 2, part = st & 3;  // 4 threads per cached row
            auto chunk = [&](int ch) {             // 16 bytes of the row
              return reinterpret_cast<uint4*>(stage + (r >> 3) * C::kGroup + (ch >> 3) * 1024 +
                                              (r & 7) * 128 + (((ch & 7) ^ (r & 7)) << 4));
            };
            uint32_t bad = 0;
            for (int ch = part; ch < D / 8; ch += 4) {
              const uint4 w = *chunk(ch);
              bad |= f16_bad(w.x) || f16_bad(w.y) || f16_bad(w.z) || f16_bad(w.w);
            }
            bad |= __shfl_xor_sync(0xffffffffu, bad, 1);
            bad |= __shfl_xor_sync(0xffffffffu, bad, 2);
            for (int ch = part; bad && ch < D / 8; ch += 4)
              *chunk(ch) = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();  // read by the PV MMA, issued after a later barrier
          }
        }
        // w = kWeightUnit s_j 2^(x scale - m) in f16 into rows hA, hB of P (K-major,
        // 128-byte swizzle) with stmatrix.  The denominator sums the unrounded 2^(..).
        const uint32_t prow = sP + s * C::kPBytes + (2 * q4) * 1024 + (lane & 7) * 128;
        auto pchunk = [&](int c) {  // this lane's address of a matrix of stmatrix: chunk c of its row
          return prow + (uint32_t)(((kReps * hc + c) ^ (lane & 7)) << 4);
        };
        float sumA, sumB;
        // (rows past the unit's end have factor 0: their weights, never used, stay finite
        // and cast no vote)
        auto weights = [&](auto masked) {
          float top = 0.f;
          sumA = sumB = 0.f;
          uint32_t pa[kReps], pb[kReps];
#pragma unroll
          for (int rep = 0; rep < kReps; ++rep) {
            float e[4], w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float arg = fmaf(x[4 * rep + k], k < 2 ? scA : scB, -((k < 2) ? mA : mB));
              const bool ok = !decltype(masked)::value || ((see >> (4 * rep + k)) & 1u);
              e[k] = ok ? ex2_approx(arg) : 0.f;
              w[k] = ok ? e[k] * sj[2 * rep + (k & 1)] : 0.f;
              top = fmaxf(top, fabsf(w[k]));
            }
            sumA += e[0] + e[1];
            sumB += e[2] + e[3];
            pa[rep] = pack_f16(w[0], w[1]);
            pb[rep] = pack_f16(w[2], w[3]);
          }
          if (held) {
            stmatrix_x4(pchunk(lane >> 3), pa[0], pa[1], pa[2], pa[3]);
            stmatrix_x4(pchunk(lane >> 3) + 1024, pb[0], pb[1], pb[2], pb[3]);
          }
          return top > kWeightTop || fmaxf(sumA, sumB) > kSumTop;
        };
        // The first tile of a piece sets m to its exact row maxima; a later one
        // is weighted against the current m, and only if a weight exceeds the headroom do
        // the warps raise m and rescale O^T.
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
              const float ls = scale_log(sj[2 * (e >> 2) + (e & 1)]);
              if ((e & 3) < 2) eA = fmaxf(eA, fmaf(x[e], scA, ls));
              else eB = fmaxf(eB, fmaf(x[e], scB, ls));
            }
          }
#pragma unroll
          for (int o = 1; o <= 2; o <<= 1) {
            eA = fmaxf(eA, __shfl_xor_sync(0xffffffffu, eA, o));
            eB = fmaxf(eB, __shfl_xor_sync(0xffffffffu, eB, o));
          }
          {  // the other half of the tile: warp w ^ 4
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
            lA = times_exp2(lA, mA - eA);
            mA = eA;
          }
          if (eB > mB + kHeadroom) {
            alphaB = ex2_approx(mB - eB);
            lB = times_exp2(lB, mB - eB);
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
            tile_wait(pv_done((g - 1) % KS), ((g - 1) / KS) & 1, wc);
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
      // (the last tile's barrier lies behind every read of the maxima)
      if (tq == 0) {
        s_lsum[hc * 64 + hA] = lA;
        s_lsum[hc * 64 + hB] = lB;
      }
      tile_wait(pv_done((g - 1) % KS), ((g - 1) / KS) & 1, wc);
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
                const float den = denominator(l, m - M, ex2_approx(ms - M));
                f = a / den / kWeightUnit;
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
              for (int e = 0; e < 16; ++e) o[(size_t)e * D] = __uint_as_float(ov[e]) / kWeightUnit;
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
cudaError_t for_shape(int R, int D, F&& f) {
#define SDA_CASE(RV, DV) \
  if (R == RV && D == DV) return f(chunk_fp8_kernel<RV, DV>, (size_t)Cfg<RV, DV>::kSmem);
  SDA_CASE(16, 64) SDA_CASE(16, 128) SDA_CASE(16, 256) SDA_CASE(16, 512)
  SDA_CASE(64, 64) SDA_CASE(64, 128) SDA_CASE(64, 256) SDA_CASE(64, 512)
#undef SDA_CASE
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t chunk_fp8_prepare() {
  for (int R : {16, 64}) {
    for (int D : {64, 128, 256, 512}) {
      const cudaError_t e = for_shape(R, D, [&](auto kernel, size_t smem) {
        cudaError_t r = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        cudaFuncAttributes a;
        if (r == cudaSuccess) r = cudaFuncGetAttributes(&a, kernel);
        // (setmaxnreg.inc waits for registers that the launch has to have)
        if (r == cudaSuccess && a.numRegs < kRegs) r = cudaErrorInvalidConfiguration;
        return r;
      });
      if (e != cudaSuccess) return e;
    }
  }
  const cudaError_t e = pair_fp8_prepare();
  return e != cudaSuccess ? e : pair_scaled_prepare();
}

ChunkLayout chunk_fp8_layout(const ChunkGeom& g, int num_sms) { return chunk_layout(g, num_sms, true); }

cudaError_t launch_chunk_fp8(const void* q, const void* codes, const float* scale, const ChunkGeom& g,
                             const float* attn_sink, float softmax_scale, void* out, float* lse,
                             const ChunkLayout& L, void* ws, cudaStream_t st) {
  ChunkFp8Params p{chunk_params(nullptr, g, attn_sink, softmax_scale, out, lse, L, ws),
                   static_cast<const uint8_t*>(codes), scale, 0, 0};
  division(g.k_per_block, &p.k_mul, &p.k_shift);
  CUtensorMap tq, tkv = {};
  if (!pipe_map_2d(&tq, q, g.D, (uint64_t)g.T * g.H, 64, L.pair ? L.R / 2 : L.R)) return cudaErrorInvalidValue;
  if (L.pair) {
    const bool tma = chunk_boxes(g);
    if (tma && !pipe_map_codes(&tkv, p.codes + g.base * g.D, g.D, (uint64_t)(g.total_pages - g.base) / 8))
      return cudaErrorInvalidValue;
    return launch_chunk_pair_fp8(tq, tkv, p, tma, L, st);
  }
  return for_shape(L.R, g.D, [&](auto kernel, size_t smem) {
    return launch_pdl(kernel, dim3(L.grid), dim3(kThreads), smem, st, tq, (const ChunkFp8Params&)p);
  });
}

}  // namespace sda
