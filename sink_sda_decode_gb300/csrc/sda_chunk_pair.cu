// sda_chunk_pair.cu -- the chunk attention for sequences with many rows: two
// CTAs of a cluster work as one on 128 rows of q (tcgen05 cta_group::2).
//
// What bounds the one-CTA kernel at D = 512 is shared-memory bandwidth: with 64
// rows of q, every 48 positions its MMAs read 190 KB of shared memory (128 bytes
// a cycle) while TMA writes 48 KB.  A pair halves the operand that its CTAs share:
//   S [128 x 64] = Q K^T     CTA r holds q rows 64 r .. and positions 32 r .. of the tile
//   O^T [D x 128] += V^T P^T CTA r holds the D / 2 columns from r D / 2 on of all 64
//                            positions (so O^T of those columns, for all 128 rows) and
//                            the weights P of its own 64 rows
// Measured: 26 cycles for QK's M128 N64 K16 and 65 for PV's M256 N128 K16, 1365 a
// tile against 1839 with one CTA a tile.  A cached row then lies in shared memory as
// key (32 rows, all of D) and as value (64 rows, half of D); the two rings are freed
// by different MMAs, so that the keys of the next tile land while the weights of
// this one are computed.  2048 tokens of 64 heads over 8192 positions, D = 512 (1.92
// TFLOP): 1.32 to 1.40 ms between runs, about 1400 TFLOP/s, against 2.09 ms with
// one CTA a tile and tiles multicast to two CTAs.  A tile takes about 1600 cycles, 1365
// of them MMAs.
//
// S [M = 128, cta_group::2]: TMEM lanes 0..63 of CTA r hold its rows at the tile's
// first 32 positions, lanes 64..127 the same rows at the other 32.
//
// Roles in each CTA (the MMA warps issue in CTA 0, for both):
//   warps 0..7   softmax of the CTA's own 64 rows
//   warp 8       QK MMAs; q loads        warp 9   PV MMAs, and the decision below
//   warp 10, 11  keys and values: by TMA, or (gather kernel) passing on to CTA 0
//                that the CTA's loader warps have landed a stage
//   warps 12..15 epilogue of the CTA's own half of D, while the softmax warps are
//                already at the next unit (with the window of 128 a unit has 4 tiles)
//   warps 16..23 (gather kernel) 4 warps copy keys, 4 values, 16-byte cp.async
//
// O^T of a row lies in both CTAs, so raising the row's running reference (rare) takes
// both: with its weights of tile g ready, each CTA tells CTA 0 whether it raised one;
// the PV warp passes the answers on to all softmax warps ("decided"), which look at it
// before they give tile g + 1 to the MMAs; if a reference was raised they scale O^T,
// and the PV MMAs of tile g wait for that.
#include <type_traits>

#include "sda_chunk_dev.cuh"

namespace sda {

namespace {

using namespace ptx;

constexpr int kR = 64;      // rows of q of a CTA
constexpr int kTile = 64;   // positions of a tile
constexpr int kKeys = 32;   // of them, keys of a CTA
constexpr int kSmThreads = 256, kSmWarps = 8;
constexpr int kQkWarp = 8, kPvWarp = 9, kKeyWarp = 10, kValWarp = 11;
constexpr int kEpiWarp0 = 12, kEpiWarps = 4;
constexpr int kLoadWarp0 = 16, kLoadWarps = 4;  // gather kernel: 4 for keys, then 4 for values
constexpr int kTmaThreads = 512;
// Gather kernel: 768 threads launch with 80 registers each; the softmax warps
// grow to 120, the loaders shrink to 48 and the others to 72.
constexpr int kGatherThreads = 768, kGatherRegs = 80;
static_assert(kSmThreads * 120 + 2 * kLoadWarps * 32 * 48 + 256 * 72 <= kGatherThreads * kGatherRegs,
              "register split exceeds the launch allocation");
constexpr int kMaxStages = 3;

enum Bar : int {
  kQFull = 0,   // CTA 0: q of both CTAs
  kQEmpty,      // both
  kSFull0,      // both
  kSEmpty0 = kSFull0 + 2,   // CTA 0: the softmax warps of both
  kPReady0 = kSEmpty0 + 2,  // CTA 0: weights of both
  kDecided0 = kPReady0 + 2, // both
  kScaled = kDecided0 + 2,  // CTA 0: the softmax warps of both
  kFac,                     // both: the final factors of the CTA's own and the other's rows
  kODone,                   // both: the epilogue warps of both have read O^T and the factors
  kKFull0,                             // CTA 0
  kVFull0 = kKFull0 + kMaxStages,      // CTA 0
  kKFree0 = kVFull0 + kMaxStages,      // both
  kVFree0 = kKFree0 + kMaxStages,      // both
  kKLanded0 = kVFree0 + kMaxStages,    // gather kernel: this CTA's keys / values
  kVLanded0 = kKLanded0 + kMaxStages,
  kBars = kVLanded0 + kMaxStages
};
enum Cmd : int { kRaise0 = 1, kRaise1 = 2, kPoison = 4 };

template <int D>
struct Cfg {
  static constexpr int kPanels = D / 64, kPanelsH = kPanels / 2;
  static constexpr int kBlocks = D / 256;             // PV MMAs of 256 rows of O^T
  static constexpr int kStages = D == 512 ? 2 : 3;
  static constexpr int kGroup = kPanelsH * 1024;      // 8 rows of half of D
  static constexpr int kKHalf = kKeys / 8 * kGroup;
  static constexpr int kKBytes = 2 * kKHalf;          // keys: [half of D][4 groups]
  static constexpr int kVBytes = kTile / 8 * kGroup;  // values: [8 groups] of the CTA's half
  static constexpr int kBox = 2 * kGroup;             // a TMA box: 16 rows of a half
  static constexpr int kPBytes = kR * 128;
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kPanels * kR * 128;
  static constexpr int kOffV = kOffK + kStages * kKBytes;
  static constexpr int kOffP = kOffV + kStages * kVBytes;  // two P buffers
  static constexpr int kOffBar = kOffP + 2 * kPBytes;
  static constexpr int kOffMisc = kOffBar + (8 * kBars + 15) / 16 * 16;  // tmem base, abort flag
  static constexpr int kOffFlag = kOffMisc + 16;           // int [2 tiles][2 CTAs] (CTA 0)
  static constexpr int kOffCmd = kOffFlag + 16;            // int [2 tiles]
  static constexpr int kOffAlpha = kOffCmd + 16;           // float [2 tiles][128 rows]
  static constexpr int kOffFac = kOffAlpha + 1024;         // float [128 rows]
  static constexpr int kOffStage = kOffFac + 512;          // epilogue staging: 2 KB a warp
  static constexpr int kOffPart = kOffStage + kEpiWarps * 2048;           // float [2 tiles][4 parts][64]: maxima; at the end l, m
  static constexpr int kSmem = kOffPart + 2048 + 1024;
  static constexpr int kOCol = 64;                         // O^T block b at columns 64 + 128 b
  static constexpr uint32_t kIdescQK = idesc_bf16_f32(128, kTile, false, false);
  static constexpr uint32_t kIdescPV = idesc_bf16_f32(256, 128, true, false);
  static_assert(kOCol + 128 * kBlocks <= 512, "TMEM columns");
  static_assert(kOffStage % 16 == 0, "16-byte staging accesses");
  static_assert(kStages * kKBytes >= 4 * (kFusedSeqs + 1), "chunk_begin's words");
  static_assert(kSmem <= 232448, "shared memory budget");
};

template <int D, bool TMA>
__global__ void __launch_bounds__(TMA ? kTmaThreads : kGatherThreads, 1)
chunk_pair_kernel(const __grid_constant__ CUtensorMap tmap_q,
                  const __grid_constant__ CUtensorMap tmap_kv, const ChunkParams p) {
  using C = Cfg<D>;
  constexpr int KS = C::kStages;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_addr(smem);
  const uint32_t sQ = sbase + C::kOffQ, sK = sbase + C::kOffK, sV = sbase + C::kOffV,
                 sP = sbase + C::kOffP;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  auto bar = [&](int i) { return sbase + C::kOffBar + 8u * (uint32_t)i; };
  const int rank = (int)(blockIdx.x & 1), worker = (int)(blockIdx.x >> 1);
  auto bar0 = [&](int i) { return map_cta(bar(i), 0); };  // of CTA 0
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(bar(kQFull), 1);
    mbar_init(bar(kQEmpty), 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(kSFull0 + s), 1);
      mbar_init(bar(kSEmpty0 + s), 2 * kSmWarps);
      mbar_init(bar(kPReady0 + s), 2);
      mbar_init(bar(kDecided0 + s), 1);
    }
    mbar_init(bar(kScaled), 2 * kSmWarps);
    mbar_init(bar(kFac), 1);  // once the CTA's own are written; the other's are counted in bytes
    mbar_init(bar(kODone), 2 * kEpiWarps);
    for (int s = 0; s < KS; ++s) {
      mbar_init(bar(kKFull0 + s), TMA ? 1 : 2);  // an expected count of bytes, or one CTA each
      mbar_init(bar(kVFull0 + s), TMA ? 1 : 2);
      mbar_init(bar(kKFree0 + s), 1);
      mbar_init(bar(kVFree0 + s), 1);
      mbar_init(bar(kKLanded0 + s), kLoadWarps * 32);
      mbar_init(bar(kVLanded0 + s), kLoadWarps * 32);
    }
    *abort_flag = 0;
    for (int i = 0; i < 4; ++i) reinterpret_cast<int*>(smem + C::kOffFlag)[i] = 0;
    for (int i = 0; i < 2; ++i) reinterpret_cast<int*>(smem + C::kOffCmd)[i] = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmap_q);
    if (TMA) tma_prefetch_desc(&tmap_kv);
  }
  if (warp == kQkWarp) {  // both CTAs' warps together
    tmem_alloc_pair(smem_addr(tmem_slot), 512);
  }
  tc_fence_before();
  __syncwarp();
  cluster_sync();  // both CTAs' barriers and TMEM are ready
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();  // everything above overlaps the plan; global memory only below
  pdl_trigger();
  bool bad;
  const ChunkStart begin = chunk_begin<TMA ? kTmaThreads : kGatherThreads, 2 * kR, kTile>(
      p, worker, reinterpret_cast<int*>(smem + C::kOffK), reinterpret_cast<int*>(smem + C::kOffP),
      &bad);
  const int nt = begin.nt;  // the pair's tiles
  int* const error = reinterpret_cast<int*>(reinterpret_cast<char*>(p.hdr) + kErrorWords) + blockIdx.x;
  if (threadIdx.x == 0) {
    *error = 0;
    if (bad && p.mode == kCut) p.recs[worker] = ChunkUnit{-1};
    if (blockIdx.x == 0) {
      p.hdr->words = gridDim.x;
      if (p.mode != kPlanned) p.hdr->error = bad ? 2 : 0;
    }
  }
  __syncthreads();
  const PipeWait wc{abort_flag, error, p.wait_timeout_ns};
  using Walk = Cursor<2 * kR, kTile>;

  if constexpr (!TMA) {
    if (warp >= kQkWarp && warp < kLoadWarp0) setmaxnreg_dec<72>();
  }
  if (warp == kKeyWarp || warp == kValWarp) {
    const bool keys = warp == kKeyWarp;
    const int full0 = keys ? kKFull0 : kVFull0, free0 = keys ? kKFree0 : kVFree0;
    bool ok = true;
    int g = 0;
    if constexpr (TMA) {
      // ===================================================== keys / values by TMA
      // Lane i < 4 loads a box of 16 rows of half of D: of the keys, half i / 2 of
      // rows 16 (i % 2) .. of the CTA's 32; of the values, the CTA's half of rows 16 i ..
      const int off = keys ? rank * kKeys + (lane & 1) * 16 : lane * 16;
      const int half = keys ? (lane >> 1) & 1 : rank;
      const uint32_t dst0 = keys ? sK + half * C::kKHalf + (lane & 1) * C::kBox : sV + lane * C::kBox;
      const uint32_t bytes = keys ? C::kKBytes : C::kVBytes;
      const int behind = (int)((p.g.total_pages - p.g.base) / 8);
      bool over = false;
      auto box_of = [&](const Walk& c) {
        return lane < 4 ? box_group(p, error, c, c.start() + off, &over) : behind;
      };
      Walk c;  // runs a tile ahead of the copies
      c.init(p.g, begin);
      int y = behind;
      if (c.left > 0) {
        y = box_of(c);
        c.next(p.g);
      }
      for (; g < nt; ++g) {
        const int s = g % KS;
        if (g >= KS) ok = warp_wait(bar(free0 + s), ((g / KS) - 1) & 1, wc);
        if (!ok) break;
        // (CTA 1's bytes may land before CTA 0 has said how many to expect: the
        // barrier's phase cannot end before that arrival)
        if (rank == 0 && lane == 0) mbar_arrive_expect_tx(bar(full0 + s), 2 * bytes);
        __syncwarp();
        if (lane < 4)
          tma_pair_4d(dst0 + s * bytes, &tmap_kv, 0, 0, half * C::kPanelsH, y, bar0(full0 + s));
        if (c.left > 0) {  // (after this tile's copies: the table entry is a while coming)
          y = box_of(c);
          c.next(p.g);
        }
      }
      if (over) atomicExch(error, 3);
    } else {
      // ===================================================== passing on landed stages
      for (; g < nt; ++g) {
        const int s = g % KS;
        ok = warp_wait(bar((keys ? kKLanded0 : kVLanded0) + s), (g / KS) & 1, wc);
        if (!ok) break;
        fence_proxy_async_smem();  // the copies were made through the generic proxy
        if (lane == 0) arrive_cluster(bar0(full0 + s));
        __syncwarp();
      }
    }
    // Every stage that was filled has been read (so its copies have landed) and
    // every arrival of the MMA warps has come in before this CTA's memory goes away.
    for (int x = max(0, g - KS); x < g; ++x) pipe_drain(bar(free0 + x % KS), (x / KS) & 1, wc);
  } else if (!TMA && warp >= kLoadWarp0) {
    // ===================================================== rows one by one
    setmaxnreg_dec<48>();
    const bool keys = warp < kLoadWarp0 + kLoadWarps;
    const int v = (warp - kLoadWarp0) % kLoadWarps;
    const int free0 = keys ? kKFree0 : kVFree0, landed0 = keys ? kKLanded0 : kVLanded0;
    // a warp copies 8 key rows of D, or 16 value rows of half of D
    constexpr int kChK = D / 8, kChV = D / 16;
    const int rows = keys ? kKeys / kLoadWarps : kTile / kLoadWarps;
    const int off = keys ? rank * kKeys + v * rows : v * rows;
    const uint4* kv4 = reinterpret_cast<const uint4*>(p.kv);
    auto slot_of = [&](const Walk& c) {
      return lane < rows ? seen_row(p, error, c, c.start() + off + lane) : -1;
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
    for (int g = 0; g < nt; ++g) {
      const int s = g % KS;
      if (g >= KS) ok = warp_wait(bar(free0 + s), ((g / KS) - 1) & 1, wc);
      if (!ok) break;
      auto copy = [&](uint32_t dst, int slot, int ch) {
        const uint4* src = slot >= 0 ? kv4 + (size_t)slot * (D / 8) + ch : kv4;
        cp_async16(dst, src, slot >= 0 ? 16u : 0u);
      };
      if (keys) {
        for (int x = 0; x < kKeys / kLoadWarps; ++x) {
          const int slot = __shfl_sync(0xffffffffu, sl0, x);
          const int r = v * (kKeys / kLoadWarps) + x;
          const uint32_t row = sK + s * C::kKBytes + (r >> 3) * C::kGroup + (r & 7) * 128;
#pragma unroll
          for (int c0 = 0; c0 < kChK; c0 += 32) {
            const int ch = c0 + lane, pn = ch >> 3;
            copy(row + pn / C::kPanelsH * C::kKHalf + pn % C::kPanelsH * 1024 + (((ch & 7) ^ (r & 7)) << 4),
                 slot, ch);
          }
        }
      } else {
        constexpr int kRowsPer = 32 / kChV;
        for (int x = 0; x < kTile / kLoadWarps; x += kRowsPer) {
          const int rl = x + lane / kChV;
          const int slot = __shfl_sync(0xffffffffu, sl0, rl);
          const int r = v * (kTile / kLoadWarps) + rl, ch = lane % kChV;
          copy(sV + s * C::kVBytes + (r >> 3) * C::kGroup + (ch >> 3) * 1024 + (r & 7) * 128 +
                   (((ch & 7) ^ (r & 7)) << 4),
               slot, rank * kChV + ch);
        }
      }
      cp_async_arrive(bar(landed0 + s));  // once this thread's copies have landed
      sl0 = sl1;
      sl1 = -1;
      if (c.left > 0) {
        sl1 = slot_of(c);
        c.next(p.g);
      }
    }
    cp_async_wait_all();
  } else if (warp == kQkWarp) {
    // ===================================================== q loads (both), QK MMAs (CTA 0)
    Walk c;
    c.init(p.g, begin);
    constexpr uint32_t kQBytes = C::kPanels * kR * 128;
    int pieces = 0;
    bool ok = true;
    auto load_q = [&]() {
      const int row = c.row0 + rank * kR;
      if (elect_one()) {
        if (rank == 0) mbar_arrive_expect_tx(bar(kQFull), 2 * kQBytes);
#pragma unroll
        for (int x = 0; x < C::kPanels; ++x)
          tma_pair_2d(sQ + x * kR * 128, &tmap_q, x * 64, row, bar0(kQFull));
      }
      __syncwarp();
    };
    bool loaded = false;
    if (c.left > 0) {
      load_q();
      loaded = true;
    }
    const uint64_t a0 = sdesc_sw128(sQ, 16, 1024);
    for (int g = 0; g < nt; ++g) {
      const int s = g & 1, ks = g % KS;
      const bool last = c.last();
      if (rank == 0) {
        if (g >= 2) ok = warp_wait(bar(kSEmpty0 + s), ((g >> 1) - 1) & 1, wc);
        if (ok && c.first) ok = warp_wait(bar(kQFull), pieces & 1, wc);
        if (ok) ok = warp_wait(bar(kKFull0 + ks), (g / KS) & 1, wc);
        if (!ok) break;
        if (!TMA) fence_proxy_async_smem();
        tc_fence_after();
        const uint64_t b0 = sdesc_sw128(sK + ks * C::kKBytes, 16, C::kGroup);
        if (elect_one()) {
#pragma unroll
          for (int pn = 0; pn < C::kPanels; ++pn) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_pair(tmem + s * 32, sdesc_advance(a0, pn * kR * 128 + k * 32),
                       sdesc_advance(b0, pn / C::kPanelsH * C::kKHalf + pn % C::kPanelsH * 1024 + k * 32),
                       C::kIdescQK, (pn || k) ? 1u : 0u);
          }
          commit_pair(bar(kSFull0 + s));
          commit_pair(bar(kKFree0 + ks));
          if (last) commit_pair(bar(kQEmpty));
        }
        __syncwarp();
      }
      c.next(p.g);
      if (last) {  // q of the next unit, once this unit's MMAs have read q
        ok = warp_wait(bar(kQEmpty), pieces & 1, wc);
        loaded = false;
        if (!ok) break;
        if (c.left > 0) {
          load_q();
          loaded = true;
        }
        ++pieces;
      }
    }
    // a q load that nothing has read (after a timeout) lands before the memory goes away
    if (loaded && rank == 0) pipe_drain(bar(kQFull), pieces & 1, wc);
  } else if (warp == kPvWarp) {
    // ===================================================== decision, PV MMAs (CTA 0)
    if (rank == 0) {
      Walk c;
      c.init(p.g, begin);
      volatile int* flag = reinterpret_cast<volatile int*>(smem + C::kOffFlag);
      int scaled = 0, pieces = 0, said[2] = {0, 0};
      for (int g = 0; g < nt; ++g) {
        const int s = g & 1, ks = g % KS;
        bool ok = warp_wait(bar(kPReady0 + s), (g >> 1) & 1, wc);
        const int f0 = flag[2 * s], f1 = flag[2 * s + 1];
        const int cmd = (f0 & 1 ? kRaise0 : 0) | (f1 & 1 ? kRaise1 : 0) | ((f0 | f1) & 2 ? kPoison : 0);
        if (cmd && ok) ok = warp_wait(bar(kVFull0 + ks), (g / KS) & 1, wc);  // values to be looked at
        if (!ok) break;
        if (lane < 2) {  // one lane tells each CTA
          if (cmd != said[s]) {
            store_cluster(map_cta(sbase + C::kOffCmd + 4 * s, lane), (uint32_t)cmd);
            fence_cluster();
          }
          arrive_cluster(map_cta(bar(kDecided0 + s), lane));
        }
        said[s] = cmd;
        __syncwarp();
        if (cmd) {
          fence_cluster();
          if (lane < 2) flag[2 * s + lane] = 0;  // for tile g + 2, which says nothing unless it has to
          ok = warp_wait(bar(kScaled), scaled & 1, wc);
          ++scaled;
        }
        if (ok) ok = warp_wait(bar(kVFull0 + ks), (g / KS) & 1, wc);
        // O^T of the piece before has been read
        if (ok && c.first && pieces > 0) ok = warp_wait(bar(kODone), (pieces - 1) & 1, wc);
        pieces += c.first;
        if (!ok) break;
        if (!TMA) fence_proxy_async_smem();
        tc_fence_after();
        const uint64_t a0 = sdesc_sw128(sV + ks * C::kVBytes, 1024, C::kGroup);
        const uint64_t b0 = sdesc_sw128(sP + s * C::kPBytes, 16, 1024);
        const uint32_t add = c.first ? 0u : 1u;
        if (elect_one()) {
#pragma unroll
          for (int b = 0; b < C::kBlocks; ++b) {
#pragma unroll
            for (int k = 0; k < kTile / 16; ++k)
              mma_pair(tmem + C::kOCol + b * 128, sdesc_advance(a0, 2 * b * 1024 + k * 2 * C::kGroup),
                       sdesc_advance(b0, k * 32), C::kIdescPV, k ? 1u : add);
          }
          commit_pair(bar(kVFree0 + ks));
        }
        __syncwarp();
        c.next(p.g);
      }
    }
  } else if (warp < kSmWarps) {
    // ===================================================== softmax and epilogue
    // Warp w reads TMEM lane quadrant q4 = w % 4 -- rows 32 (q4 % 2) .. + 31 at the
    // tile's positions 32 kh .., kh = q4 / 2 -- and of these the 16 positions from
    // 16 hc on, hc = w / 4.  Thread t holds rows base + t / 4 + 8 i, i = 0..3, at the
    // positions 8 rep + 2 (t % 4) + {0, 1}, rep = 0, 1: element 4 i + 2 rep + {0, 1}.
    if constexpr (!TMA) setmaxnreg_inc<120>();
    const int q4 = warp & 3, hc = warp >> 2, st = threadIdx.x, tq = lane & 3;
    const int kh = q4 >> 1, rb = (q4 & 1) * 32, part = 2 * kh + hc, row0 = rb + (lane >> 2);
    const uint32_t lane_base = (uint32_t)(q4 * 32) << 16;
    float* s_alpha = reinterpret_cast<float*>(smem + C::kOffAlpha);
    float* s_fac = reinterpret_cast<float*>(smem + C::kOffFac);
    float* s_part = reinterpret_cast<float*>(smem + C::kOffPart);
    volatile int* s_cmd = reinterpret_cast<volatile int*>(smem + C::kOffCmd);
    const float sc = p.qk_scale_log2;
    const int H = p.g.H, window = p.g.window, nfirst = p.g.first;
    const uint32_t s_empty[2] = {bar0(kSEmpty0), bar0(kSEmpty0 + 1)};
    const uint32_t p_ready[2] = {bar0(kPReady0), bar0(kPReady0 + 1)};
    const uint32_t my_flag = map_cta(sbase + C::kOffFlag, 0) + 4 * rank;
    int g = 0, pieces = 0;
    // What was decided on tile x: scales O^T or clears bad values if it has to be
    // (the PV MMAs of tile x wait for that).  Uniform over both CTAs' softmax warps.
    auto decided = [&](int x) {
      const int s = x & 1;
      warp_wait(bar(kDecided0 + s), (x >> 1) & 1, wc);
      const int cmd = *abort_flag ? 0 : s_cmd[s];
      if (cmd == 0) return;
      fence_cluster();
      if (cmd & (kRaise0 | kRaise1)) {
        // O^T is quiescent once the PV MMAs of tile x - 1 are done
        if (x > 0) warp_wait(bar(kVFree0 + (x - 1) % KS), ((x - 1) / KS) & 1, wc);
        tc_fence_after();
        const int c0 = cmd & kRaise0 ? 0 : 64, c1 = cmd & kRaise1 ? 128 : 64;
#pragma unroll 1
        for (int b = 0; b < C::kBlocks; ++b) {
#pragma unroll 1
          for (int col = c0 + 16 * hc; col < c1; col += 32) {
            uint32_t ov[16];
            const uint32_t ta = tmem + lane_base + C::kOCol + b * 128 + col;
            tmem_ld16(ta, ov);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e)
              ov[e] = __float_as_uint(__uint_as_float(ov[e]) * s_alpha[s * 128 + col + e]);
            tmem_st16(ta, ov);
          }
        }
        tmem_wait_st();
        tc_fence_before();
      }
      if (cmd & kPoison) {
        // Values with an infinity or NaN, which some row does not see: its weight
        // there is 0, but 0 x inf = NaN in the MMA.  They are cleared; the rows that
        // do see them have a NaN weight already, or 0 where the score is -inf.
        const int r = st >> 2, part4 = st & 3;  // 4 threads per row
        auto chunk = [&](int ch) {
          return reinterpret_cast<uint4*>(smem + C::kOffV + (x % KS) * C::kVBytes + (r >> 3) * C::kGroup +
                                          (ch >> 3) * 1024 + (r & 7) * 128 + (((ch & 7) ^ (r & 7)) << 4));
        };
        uint32_t bad = 0;
        for (int ch = part4; ch < D / 16; ch += 4) {
          const uint4 w = *chunk(ch);
          const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            bad |= (ws[e] & 0x7f80u) == 0x7f80u || (ws[e] & 0x7f800000u) == 0x7f800000u;
        }
        bad |= __shfl_xor_sync(0xffffffffu, bad, 1);
        bad |= __shfl_xor_sync(0xffffffffu, bad, 2);
        for (int ch = part4; bad && ch < D / 16; ch += 4) *chunk(ch) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) arrive_cluster(bar0(kScaled));
    };

    UnitWalk uw;
    uw.init(p.g, 2 * kR, begin);
    while (g < nt) {
      if (pieces > 0) uw.next(p.g, 2 * kR);
      const ChunkUnit un = chunk_unit(p.g, 2 * kR, kTile, uw.b, uw.r);
      const int i0 = g == 0 ? begin.off : 0;
      const int i1 = min(un.ntiles, i0 + nt - g);
      const bool whole = i0 == 0 && i1 == un.ntiles;
      const int h0 = un.h0 + rank * kR, nrows = max(0, min(kR, un.nrows - rank * kR));
      const int p_lo = un.pos0 + div_h(p.g, h0), p_hi = un.pos0 + div_h(p.g, h0 + max(nrows, 1) - 1);
      const float sink =
          whole && st < nrows ? __ldg(p.attn_sink + h0 + st - div_h(p.g, h0 + st) * H) : 0.f;  // of row st
      float m[4], l[4], scr[4];  // l: this thread's share
      int pos[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        m[i] = kNoScore;
        l[i] = 0.f;
        // (rows past the unit's end have factor 0: their weights, never used, stay
        // finite and raise nothing)
        scr[i] = row0 + 8 * i < nrows ? sc : 0.f;
        pos[i] = un.pos0 + div_h(p.g, h0 + row0 + 8 * i);
      }
      for (int i = i0; i < i1; ++i, ++g) {
        const int s = g & 1;
        const int j0 = chunk_tile_start(i, un.nf, un.lo, kTile);
        // whether every row of this CTA sees the whole tile
        const bool full = j0 + kTile - 1 <= p_lo &&
                          (window == 0 || j0 > p_hi - window || j0 + kTile <= nfirst);
        warp_wait(bar(kSFull0 + s), (g >> 1) & 1, wc);
        tc_fence_after();
        float x[16];
        {
          uint32_t va[8], vb[8];
          const uint32_t ta = tmem + lane_base + s * 32 + 16 * hc;
          tmem_ld_16x256b_x2(ta, va);
          tmem_ld_16x256b_x2(ta + (16u << 16), vb);
          tmem_wait_ld();
          // register 4 rep + k: row + 8 (k / 2), position 8 rep + 2 (t % 4) + k % 2
#pragma unroll
          for (int rep = 0; rep < 2; ++rep) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              x[4 * (k >> 1) + 2 * rep + (k & 1)] = __uint_as_float(va[4 * rep + k]);
              x[8 + 4 * (k >> 1) + 2 * rep + (k & 1)] = __uint_as_float(vb[4 * rep + k]);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_cluster(s_empty[s]);
        uint32_t see = 0xffffu;
        int flags = 0;
        if (!full) {
          // bits 0, 1, 8, 9 of a row's ten positions are its elements 0..3
          see = 0;
#pragma unroll
          for (int i4 = 0; i4 < 4; ++i4) {
            const uint32_t m10 = seen_bits(pos[i4], j0 + 32 * kh + 16 * hc + 2 * tq, window, nfirst);
            see |= ((m10 & 3u) | ((m10 >> 6) & 12u)) << (4 * i4);
          }
          bool poison = false;  // a score that is masked and not finite
          float zero = 0.f;  // NaN if a score is not finite
#pragma unroll
          for (int e = 0; e < 16; ++e) zero = fmaf(x[e], 0.f, zero);
          if (zero != 0.f) {
            uint32_t bad = 0;
#pragma unroll
            for (int e = 0; e < 16; ++e) bad |= fabsf(x[e]) < INFINITY ? 0u : 1u << e;
            poison = (bad & ~see) != 0;
          }
          if (named_bar_or(1, kSmThreads, poison)) flags = 2;
        }
        // P buffer s is free once the PV MMAs of tile g - 2 are done
        if (g >= 2) warp_wait(bar(kVFree0 + (g - 2) % KS), ((g - 2) / KS) & 1, wc);
        // p = 2^(x scale - m) in bf16 into P (K-major, 128-byte swizzle).  The MMA
        // multiplies the rounded p, the denominator sums the unrounded ones: each
        // weight is off by at most 2^-8 of itself, as the output's own rounding.
        const uint32_t pbuf = sP + s * C::kPBytes;
        float sum[4];
        auto weights = [&](auto masked) {
          float top = -INFINITY;
          uint32_t pk[4][2];
#pragma unroll
          for (int i4 = 0; i4 < 4; ++i4) {
            float e[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float arg = fmaf(x[4 * i4 + k], scr[i4], -m[i4]);
              const bool ok = !decltype(masked)::value || ((see >> (4 * i4 + k)) & 1u);
              top = fmaxf(top, ok ? arg : -INFINITY);
              e[k] = ok ? ex2_approx(arg) : 0.f;
            }
            sum[i4] = (e[0] + e[1]) + (e[2] + e[3]);
            const __nv_bfloat162 a = __floats2bfloat162_rn(e[0], e[1]);
            const __nv_bfloat162 b = __floats2bfloat162_rn(e[2], e[3]);
            pk[i4][0] = *reinterpret_cast<const uint32_t*>(&a);
            pk[i4][1] = *reinterpret_cast<const uint32_t*>(&b);
          }
          // matrices of a stmatrix.x4: rows + 8 (mi % 2), chunk + mi / 2
          const int mi = lane >> 3, r8 = lane & 7;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int r = rb + 16 * half + 8 * (mi & 1) + r8, ch = 4 * kh + 2 * hc + (mi >> 1);
            stmatrix_x4(pbuf + (r >> 3) * 1024 + r8 * 128 + ((ch ^ r8) << 4), pk[2 * half][0],
                        pk[2 * half + 1][0], pk[2 * half][1], pk[2 * half + 1][1]);
          }
          return top > kHeadroom;
        };
        // The first tile of a piece sets m to its exact row maxima; a later one is
        // weighted against the current m, and only if a score exceeds it by the
        // headroom is m raised (p stays below 2^8).
        bool exact = i == i0;
        if (!exact) {
          const bool over = full ? weights(std::false_type{}) : weights(std::true_type{});
          fence_proxy_async_smem();
          exact = named_bar_or(1, kSmThreads, over);
        }
        if (exact) {
          float* hm = s_part + (g & 1) * 256;
          float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int e = 0; e < 16; ++e)
            top[e >> 2] = fmaxf(top[e >> 2], (see >> e) & 1u ? x[e] * scr[e >> 2] : -INFINITY);
#pragma unroll
          for (int i4 = 0; i4 < 4; ++i4) {
            top[i4] = fmaxf(top[i4], __shfl_xor_sync(0xffffffffu, top[i4], 1));
            top[i4] = fmaxf(top[i4], __shfl_xor_sync(0xffffffffu, top[i4], 2));
            if (tq == 0) hm[part * 64 + row0 + 8 * i4] = top[i4];
          }
          named_bar_sync(1, kSmThreads);
#pragma unroll
          for (int i4 = 0; i4 < 4; ++i4) {
            const int r = row0 + 8 * i4;
            const float t = fmaxf(fmaxf(hm[r], hm[64 + r]), fmaxf(hm[128 + r], hm[192 + r]));
            float alpha = 1.f;
            // (the second condition adds nothing to the first but its code: replayed drafted
            // tokens take 122.4 us with it, 124.1 without)
            if (t > m[i4] + kHeadroom || (m[i4] == kNoScore && t > m[i4])) {
              alpha = ex2_approx(m[i4] - t);  // 0 when there was no score
              l[i4] *= alpha;
              m[i4] = t;
            }
            if (i > i0 && tq == 0 && part == 0) {  // both CTAs hold O^T of this row
#pragma unroll
              for (int cta = 0; cta < 2; ++cta)
                store_cluster(map_cta(sbase + C::kOffAlpha + 4 * (s * 128 + rank * 64 + r), cta),
                              __float_as_uint(alpha));
            }
          }
          if (i > i0) {
            flags |= 1;
            fence_cluster();
          }
          if (full) weights(std::false_type{});
          else weights(std::true_type{});
          fence_proxy_async_smem();
          named_bar_sync(1, kSmThreads);
        }
#pragma unroll
        for (int i4 = 0; i4 < 4; ++i4) l[i4] += sum[i4];
        // What was decided on tile g - 1 has long come in by now; its PV MMAs, if they
        // wait for O^T to be scaled, come before tile g's.
        if (g > 0) decided(g - 1);
        if (st == 0) {
          if (flags) {
            store_cluster(my_flag + 8 * s, (uint32_t)flags);
            fence_cluster();
          }
          arrive_cluster(p_ready[s]);
        }
      }
      // ---------------------------------------------- end of the piece
      // (the last tile's barriers lie behind every read of the maxima)
      float* s_l = s_part;            // [4 parts][64]
      float* s_m = s_part + 256;      // [64]
      named_bar_sync(1, kSmThreads);
#pragma unroll
      for (int i4 = 0; i4 < 4; ++i4) {
        float t = l[i4];
        t += __shfl_xor_sync(0xffffffffu, t, 1);
        t += __shfl_xor_sync(0xffffffffu, t, 2);
        if (tq == 0) {
          s_l[part * 64 + row0 + 8 * i4] = t;
          if (part == 0) s_m[row0 + 8 * i4] = m[i4];
        }
      }
      named_bar_sync(1, kSmThreads);
      // the factors of the piece before have been read in both CTAs
      if (pieces > 0) warp_wait(bar(kODone), (pieces - 1) & 1, wc);
      if (st < kR) {
        const float mp = s_m[st], mr = mp == kNoScore ? -INFINITY : mp;
        const float lr = (s_l[st] + s_l[64 + st]) + (s_l[128 + st] + s_l[192 + st]);
        float f = 0.f;
        if (whole) {
          if (st < nrows) {
            const float ms = sink * kLog2e;
            const float M = fmaxf(mr, ms);
            float lse = M * kLn2;
            if (M != -INFINITY && ms != INFINITY) {
              const float a = mr == -INFINITY ? 0.f : ex2_approx(mr - M);
              const float den = fmaf(lr, a, ex2_approx(ms - M));
              f = a / den;
              lse = (M + log2f(den)) * kLn2;
            }
            // (the sink alone: as it is; a NaN that was seen: NaN)
            p.lse[un.row0 + rank * kR + st] = lr != lr ? lr : (mr == -INFINITY ? sink : lse);
          }
        } else {
          const int slot = 2 * worker + (i0 == 0 ? 1 : 0);
          p.part_ml[(size_t)slot * 2 * kR + rank * kR + st] = make_float2(mr, lr);
        }
        s_fac[rank * kR + st] = f;
        store_async(map_cta(sbase + C::kOffFac + 4 * (rank * kR + st), rank ^ 1), __float_as_uint(f),
                    map_cta(bar(kFac), rank ^ 1));
      }
      named_bar_sync(1, kSmThreads);  // (s_part may be rewritten, too)
      if (st == 0) mbar_arrive_expect_tx(bar(kFac), kR * 4);
      ++pieces;
    }
    if (g > 0) decided(g - 1);
  } else if (warp >= kEpiWarp0 && warp < kEpiWarp0 + kEpiWarps) {
    // ===================================================== epilogue
    // Warp q4 takes the TMEM lanes 32 q4 .., so columns 32 q4 .. of each block of the
    // CTA's half of D, for all 128 rows, 32 rows at a time.
    const int q4 = warp & 3, tq = lane & 3, mt = lane >> 3, jr = lane & 7;
    const float* s_fac = reinterpret_cast<const float*>(smem + C::kOffFac);
    uint8_t* stg = smem + C::kOffStage + q4 * 2048;
    int g = 0, pieces = 0;
    UnitWalk uw;
    uw.init(p.g, 2 * kR, begin);
    while (g < nt) {
      if (pieces > 0) uw.next(p.g, 2 * kR);
      const ChunkUnit un = chunk_unit(p.g, 2 * kR, kTile, uw.b, uw.r);
      const int i0 = g == 0 ? begin.off : 0;
      const int i1 = min(un.ntiles, i0 + nt - g);
      const bool whole = i0 == 0 && i1 == un.ntiles;
      g += i1 - i0;
      warp_wait(bar(kFac), pieces & 1, wc);
      warp_wait(bar(kVFree0 + (g - 1) % KS), ((g - 1) / KS) & 1, wc);  // O^T is complete
      tc_fence_after();
      if (whole) {
        // scaled, packed to bf16, transposed with stmatrix (row r: 64 bytes, 16-byte
        // chunk c at c ^ (r / 2 % 4)) and stored to out as 64-byte pieces of rows
#pragma unroll 1
        for (int x = 0; x < 4 * C::kBlocks; ++x) {
          const int b = x >> 2, r0 = (x & 3) * 32;  // block of D, first row
          if (r0 >= un.nrows) continue;
          uint32_t rr[2][16];
#pragma unroll
          for (int half = 0; half < 2; ++half)
            tmem_ld_16x256b_x4(tmem + ((uint32_t)(q4 * 32 + 16 * half) << 16) + C::kOCol + b * 128 + r0,
                               rr[half]);
          tmem_wait_ld();
          float fac[8];
#pragma unroll
          for (int rep = 0; rep < 4; ++rep) {
            fac[2 * rep] = s_fac[r0 + 8 * rep + 2 * tq];
            fac[2 * rep + 1] = s_fac[r0 + 8 * rep + 2 * tq + 1];
          }
          __syncwarp();  // the step before has read the staging area
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t pk[8];
#pragma unroll
            for (int rep = 0; rep < 4; ++rep) {
#pragma unroll
              for (int dg = 0; dg < 2; ++dg) {
                // "+ 0.f" turns -0 into +0 when the factor is 0 (sink = +inf)
                const __nv_bfloat162 v2 = __floats2bfloat162_rn(
                    __uint_as_float(rr[half][4 * rep + 2 * dg]) * fac[2 * rep] + 0.f,
                    __uint_as_float(rr[half][4 * rep + 2 * dg + 1]) * fac[2 * rep + 1] + 0.f);
                pk[2 * rep + dg] = *reinterpret_cast<const uint32_t*>(&v2);
              }
            }
            // matrix mt of a stmatrix.x4: rows 8 (rep0 + mt / 2) .., columns 16 half + 8 (mt % 2) ..
#pragma unroll
            for (int rep0 = 0; rep0 < 4; rep0 += 2) {
              const int r = 8 * (rep0 + (mt >> 1)) + jr, ch = 2 * half + (mt & 1);
              stmatrix_x4_trans(smem_addr(stg) + r * 64 + ((ch ^ ((r >> 1) & 3)) << 4), pk[2 * rep0],
                                pk[2 * rep0 + 1], pk[2 * rep0 + 2], pk[2 * rep0 + 3]);
            }
          }
          __syncwarp();
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = 8 * e + (lane >> 2), ch = lane & 3;
            const uint4 w = *reinterpret_cast<const uint4*>(stg + r * 64 + ((ch ^ ((r >> 1) & 3)) << 4));
            if (r0 + r < un.nrows)
              *reinterpret_cast<uint4*>(p.out + (size_t)(un.row0 + r0 + r) * D + rank * (D / 2) + b * 128 +
                                        q4 * 32 + ch * 8) = w;
          }
        }
      } else {
        const int slot = 2 * worker + (i0 == 0 ? 1 : 0);
#pragma unroll 1
        for (int b = 0; b < C::kBlocks; ++b) {
          const int d = rank * (D / 2) + b * 128 + q4 * 32 + lane;
#pragma unroll 1
          for (int col = 0; col < un.nrows; col += 16) {
            uint32_t ov[16];
            tmem_ld16(tmem + ((uint32_t)(q4 * 32) << 16) + C::kOCol + b * 128 + col, ov);
            tmem_wait_ld();
            float* o = p.part_o + ((size_t)slot * 2 * kR + col) * D + d;
#pragma unroll
            for (int e = 0; e < 16; ++e) o[(size_t)e * D] = __uint_as_float(ov[e]);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane < 2) arrive_cluster(map_cta(bar(kODone), lane));
      ++pieces;
    }
    // (the other CTA's last arrivals come in before this CTA's memory goes away)
    if (pieces > 0) pipe_drain(bar(kODone), (pieces - 1) & 1, wc);
  }

  __syncwarp();
  tc_fence_before();
  cluster_sync();  // neither CTA leaves while the other may still reach its memory
  tc_fence_after();
  if (warp == kQkWarp)
    tmem_dealloc_pair(tmem, 512);
}

template <typename F>
cudaError_t for_shape(int D, bool tma, F&& f) {
#define SDA_CASE(DV)                                                                        \
  if (D == DV)                                                                              \
    return tma ? f(chunk_pair_kernel<DV, true>, (size_t)Cfg<DV>::kSmem, dim3(kTmaThreads))  \
               : f(chunk_pair_kernel<DV, false>, (size_t)Cfg<DV>::kSmem, dim3(kGatherThreads));
  SDA_CASE(256) SDA_CASE(512)
#undef SDA_CASE
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t pair_prepare() {
  for (int D : {256, 512}) {
    for (bool tma : {false, true}) {
      const cudaError_t e = for_shape(D, tma, [&](auto kernel, size_t smem, dim3) {
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
  return cudaSuccess;
}

cudaError_t launch_chunk_pair(const CUtensorMap& tq, const CUtensorMap& tkv, const ChunkParams& p,
                              bool tma, const ChunkLayout& L, cudaStream_t st) {
  return for_shape(p.g.D, tma, [&](auto kernel, size_t smem, dim3 threads) {
    return launch_pdl_cluster(kernel, dim3(2 * L.grid), threads, 2, smem, st, tq, tkv, p);
  });
}

}  // namespace sda
