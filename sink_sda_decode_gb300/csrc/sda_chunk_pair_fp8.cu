// sda_chunk_pair_fp8.cu -- chunk attention over a cache of E4M3 codes for sequences with
// many rows: two CTAs of a cluster work as one on 128 rows of q (tcgen05 cta_group::2).
//
// The division of work is sda_chunk_pair.cu's, with tiles of 128 positions:
//   S [128 x 128] = Q K^T     CTA r holds q rows 64 r .. and positions 64 r .. of the tile
//   O^T [D x 128] += V^T P^T  CTA r holds the D / 2 columns from r D / 2 on of all 128
//                             positions and the weights P of its own 64 rows
// The keys are the codes themselves (kind::f8f6f4), so nothing converts them and they take
// half the room of 16-bit keys, which is what makes tiles of 128 fit: an MMA of N = 128
// reads 4 KB of shared memory for as many products as two of N = 64 with 6.  q, bf16,
// becomes the sum of two 8-bit terms: times the power of two that brings its row's largest
// element to [2^7, 2^8), q1 = e4m3(q) and q2 = e5m2(q - q1).  q - q1 is at most 8 units of
// bf16's last place, which three bits hold, so elements down to 2^-13 of the largest are
// exact; smaller ones are off by at most 2^-21 of it.  Two MMAs a step add up in the same
// accumulator.  The values are f16, converted on the way to shared memory, and the weights
// and scales are sda_chunk_fp8.cuh's.
//
// S [M = 128, cta_group::2]: TMEM lanes 0..63 of CTA r hold its rows at the tile's
// first 64 positions, lanes 64..127 the same rows at the other 64.
//
// Roles in each CTA (the MMA warps issue in CTA 0, for both):
//   warps 0..7   softmax of the CTA's own 64 rows
//   warp 8       QK MMAs; q loads        warp 9   PV MMAs, and the decision below
//   warp 10      keys by TMA, or (gather kernel) passing on to CTA 0 that they landed
//   warp 11      looks the positions up: pool rows and scales, a few tiles ahead
//   warps 12..15 epilogue of the CTA's own half of D; q of the next unit into its two terms
//   warps 16..23 values: codes into registers a tile ahead, then as f16 to shared memory
//                (gather kernel: keys, too, by 16-byte cp.async)
//
// O^T of a row lies in both CTAs, so raising the row's running reference (rare) takes
// both; the decision about it is sda_chunk_pair.cu's.
//
// For 65 rows of q a sequence on average to some hundred (above that, and with the workspace
// for it, sda_spread.cu's way is faster).  One token of 128 heads over 32 caches of 1000 to 8192
// positions, D = 512: 73 us, of 23 of MMAs at their rate.  A tile takes 3800 cycles, 2200 of them
// MMAs: the softmax warps bound it.
#include <type_traits>

#include "sda_chunk_fp8.cuh"

namespace sda {

namespace {

using namespace ptx;

constexpr int kR = 64;       // rows of q of a CTA
constexpr int kTile = 128;   // positions of a tile
constexpr int kHalf = 64;    // of them, keys of a CTA
constexpr int kQuarter = 32; // and of a stage of values
constexpr int kSmThreads = 256, kSmWarps = 8;
constexpr int kQkWarp = 8, kPvWarp = 9, kKeyWarp = 10, kLookWarp = 11;
constexpr int kEpiWarp0 = 12, kEpiWarps = 4;
constexpr int kLoadWarp0 = 16, kLoadWarps = 8;
// 768 threads launch with 80 registers each; the softmax warps grow to 104, the loaders
// shrink to 72 and the others to 64.  (What is spilled misses L1, of which 227 KB of shared
// memory leave little: with 56 for the loaders, 45 registers were, and a prompt chunk took
// 2.89 ms.)
constexpr int kThreads = 768, kRegs = 80;
static_assert(kSmThreads * 104 + 256 * 64 + kLoadWarps * 32 * 72 <= kThreads * kRegs,
              "register split exceeds the launch allocation");
constexpr int kKStages = 1, kVStages = 5;
constexpr int kLook = 4;  // tiles that are looked up ahead

enum Bar : int {
  kQFull = 0,   // this CTA's q
  kQReady,      // CTA 0: the epilogue warps of both have converted it
  kQEmpty,      // both
  kSFull0,      // both
  kSEmpty0 = kSFull0 + 2,   // CTA 0: the softmax warps of both
  kPReady0 = kSEmpty0 + 2,  // CTA 0: weights of both (+ 2 * buffer + half of the tile)
  kPFree0 = kPReady0 + 4,   // both: the PV MMAs have read a buffer
  kDecided0 = kPFree0 + 2,  // both
  kScaled = kDecided0 + 2,  // CTA 0: the softmax warps of both
  kFac,                     // both: the final factors of the CTA's own and the other's rows
  kODone,                   // both: the epilogue warps of both have read O^T and the factors
  kLkFull0,                        // a tile's rows and scales are looked up
  kLkFree0 = kLkFull0 + kLook,     // the softmax warps and the loaders have read them
  kKFull0 = kLkFree0 + kLook,      // CTA 0
  kVFull0 = kKFull0 + kKStages,    // CTA 0
  kKFree0 = kVFull0 + kVStages,    // both
  kVFree0 = kKFree0 + kKStages,    // both
  kKLanded0 = kVFree0 + kVStages,  // gather kernel: this CTA's keys
  kBars = kKLanded0 + kKStages
};
enum Cmd : int { kRaise0 = 1, kRaise1 = 2 };

// Instruction descriptor of kind::f8f6f4 with E4M3 B, E4M3 or E5M2 A, and fp32 D.
constexpr uint32_t idesc_f8_f32(int M, int N, bool a_e5m2) {
  return (1u << 4) | ((a_e5m2 ? 1u : 0u) << 7) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// A shared-memory descriptor (sdesc_sw128) in halves: the upper one, of a stride between
// groups of 8 rows, is a constant; the lower one holds the address, in units of 16 bytes.
constexpr uint32_t desc_hi(uint32_t sbo) { return (sbo >> 4) | 1u << 14 | 2u << 29; }
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) {
  return ((saddr & 0x3FFFFu) >> 4) | (lbo >> 4) << 16;
}
template <bool F8, uint32_t HA, uint32_t HB>
__device__ __forceinline__ void mma_of(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
  if constexpr (F8)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %6};\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a, b, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(acc), "n"(HA), "n"(HB)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %6};\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(acc), "n"(HA), "n"(HB)
        : "memory");
}

template <int D>
struct Cfg {
  static constexpr int kPanelsQ = D / 64;             // of 64 bf16, then D / 128 of q1 and of q2 codes
  static constexpr int kPanelsK = D / 128;            // of 128 codes
  static constexpr int kPanelsV = D / 128;            // of 64 f16: half of D
  static constexpr int kBlocks = D / 256;             // PV MMAs of 256 rows of O^T
  static constexpr int kGroupK = kPanelsK * 1024;     // 8 rows of keys
  static constexpr int kGroupV = kPanelsV * 1024;     // 8 rows of values
  static constexpr int kKBytes = kHalf / 8 * kGroupK;
  static constexpr int kVBytes = kQuarter / 8 * kGroupV;
  static constexpr int kBox = 2 * kGroupK;            // a TMA box: 16 rows
  static constexpr int kPHalf = kR * 128;
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kPanelsQ * kR * 128;
  static constexpr int kOffV = kOffK + kKStages * kKBytes;
  static constexpr int kOffP = kOffV + kVStages * kVBytes;  // weights: two buffers, by halves of the tile
  static constexpr int kOffBar = kOffP + 4 * kPHalf;
  static constexpr int kOffMisc = kOffBar + (8 * kBars + 15) / 16 * 16;  // tmem base, abort flag
  static constexpr int kOffFlag = kOffMisc + 16;           // int [2 tiles][2 CTAs] (CTA 0)
  static constexpr int kOffCmd = kOffFlag + 16;            // int [2 tiles]
  static constexpr int kOffAlpha = kOffCmd + 16;           // float [2 tiles][128 rows]
  static constexpr int kOffFac = kOffAlpha + 1024;         // float [128 rows]
  static constexpr int kOffStage = kOffFac + 512;          // epilogue staging: 2 KB a warp
  static constexpr int kOffPart = kOffStage + kEpiWarps * 2048;  // float [2 tiles][4 parts][64]: maxima; at the end l, m
  static constexpr int kOffScale = kOffPart + 2048;        // float [kLook tiles][128]: kWeightUnit s_j
  static constexpr int kOffRow = kOffScale + 512 * kLook;  // int [kLook tiles][128]: pool rows, or -1
  static constexpr int kOffMask = kOffRow + 512 * kLook;   // int [kLook tiles]: some row does not see all of the tile
  static constexpr int kOffQs = kOffMask + 4 * kLook;      // [4 pieces][64]: exponents of q's 2^-k
  static constexpr int kSmem = kOffQs + 256 + 1024;
  static constexpr int kOCol = 128;                        // O^T block b at columns 128 + 128 b
  static constexpr uint32_t kIdescQ1 = idesc_f8_f32(128, kTile, false), kIdescQ2 = idesc_f8_f32(128, kTile, true);
  static constexpr uint32_t kIdescPV = idesc_f16_f32(256, 128, true);
  // a loader's share of a stage of values: 8 rows of half of D, in 16-byte loads
  static constexpr int kRowsPer = 1024 / D, kLoads = 8 / kRowsPer;
  static_assert(kOCol + 128 * kBlocks <= 512, "TMEM columns");
  static_assert(kOffStage % 16 == 0 && kOffScale % 16 == 0, "16-byte accesses");
  static_assert(kKStages * kKBytes >= 4 * (kFusedSeqs + 1), "chunk_begin's words");
  static_assert(kSmem <= 232448, "shared memory budget");
};

// One row of q in shared memory (`at(ch)`: the place of 16-byte chunk ch of its bf16 form)
// into its two terms: q1's codes over the row's first half, q2's over the second.  Lane l of
// LANES holds elements 16 l ..  Returns the exponent (as fp32 holds it) of 2^-k, or 255 for
// a row that holds an infinity or NaN.
template <int LANES, typename At>
__device__ __forceinline__ uint32_t q_row_to_f8(At at, int lane) {
  const int l = lane % LANES;
  const uint4 v0 = *at(2 * l), v1 = *at(2 * l + 1);
  const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) top = __vmaxu2(top, w[e] & 0x7fff7fffu);
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
  const uint32_t most = max(top & 0xffffu, top >> 16);
  const int k2 = most == 0 ? 0 : min(7 + 127 - (int)(most >> 7), 126);
  const float up = __uint_as_float((uint32_t)(127 + k2) << 23);
  uint32_t a[4] = {0, 0, 0, 0}, b[4] = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float lo = __uint_as_float(w[e] << 16) * up, hi = __uint_as_float(w[e] & 0xffff0000u) * up;
    uint16_t c1, c2;
    uint32_t back;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c1) : "f"(hi), "f"(lo));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back) : "h"(c1));
    const __half2 h = *reinterpret_cast<const __half2*>(&back);
    const float rl = lo - __low2float(h), rh = hi - __high2float(h);
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(c2) : "f"(rh), "f"(rl));
    a[e >> 1] |= (uint32_t)c1 << (16 * (e & 1));
    b[e >> 1] |= (uint32_t)c2 << (16 * (e & 1));
  }
  __syncwarp();  // (the row has been read)
  *at(l) = make_uint4(a[0], a[1], a[2], a[3]);
  *at(LANES + l) = make_uint4(b[0], b[1], b[2], b[3]);
  return most >= 0x7f80u ? 255u : (uint32_t)(127 - k2);
}

template <int D, bool TMA>
__global__ void __launch_bounds__(kThreads, 1)
chunk_pair_fp8_kernel(const __grid_constant__ CUtensorMap tmap_q,
                      const __grid_constant__ CUtensorMap tmap_kv, const ChunkFp8Params fp) {
  using C = Cfg<D>;
  const ChunkParams& p = fp.c;
  constexpr int KS = kKStages, VS = kVStages;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_addr(smem);
  const uint32_t sQ = sbase + C::kOffQ, sK = sbase + C::kOffK, sV = sbase + C::kOffV,
                 sP = sbase + C::kOffP;
  float* s_scale = reinterpret_cast<float*>(smem + C::kOffScale);
  int* s_row = reinterpret_cast<int*>(smem + C::kOffRow);
  int* s_mask = reinterpret_cast<int*>(smem + C::kOffMask);
  uint8_t* s_qs = smem + C::kOffQs;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  auto bar = [&](int i) { return sbase + C::kOffBar + 8u * (uint32_t)i; };
  const int rank = (int)(blockIdx.x & 1), worker = (int)(blockIdx.x >> 1);
  auto bar0 = [&](int i) { return map_cta(bar(i), 0); };  // of CTA 0
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(bar(kQFull), 1);
    mbar_init(bar(kQReady), 2 * kEpiWarps);
    mbar_init(bar(kQEmpty), 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(kSFull0 + s), 1);
      mbar_init(bar(kSEmpty0 + s), 2 * kSmWarps);
      mbar_init(bar(kPReady0 + 2 * s), kSmWarps);
      mbar_init(bar(kPReady0 + 2 * s + 1), kSmWarps);
      mbar_init(bar(kPFree0 + s), 1);
      mbar_init(bar(kDecided0 + s), 1);
    }
    for (int s = 0; s < kLook; ++s) {
      mbar_init(bar(kLkFull0 + s), 1);
      mbar_init(bar(kLkFree0 + s), kSmWarps + kLoadWarps);
    }
    mbar_init(bar(kScaled), 2 * kSmWarps);
    mbar_init(bar(kFac), 1);  // once the CTA's own are written; the other's are counted in bytes
    mbar_init(bar(kODone), 2 * kEpiWarps);
    for (int s = 0; s < KS; ++s) {
      mbar_init(bar(kKFull0 + s), TMA ? 1 : 2);  // an expected count of bytes, or one CTA each
      mbar_init(bar(kKFree0 + s), 1);
      mbar_init(bar(kKLanded0 + s), kLoadWarps * 32);
    }
    for (int s = 0; s < VS; ++s) {
      mbar_init(bar(kVFull0 + s), kLoadWarps);  // four of each CTA
      mbar_init(bar(kVFree0 + s), 1);
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
  const ChunkStart begin = chunk_begin<kThreads, 2 * kR, kTile>(
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

  // A share of q of piece n from bf16 into its two terms: warp w of `among`.  The epilogue
  // warps do that; with the first piece, which everything waits for, the softmax warps help
  // them (a step of 128 heads: q is ready after 4 us in place of 8).
  auto q_to_f8 = [&](int n, int w, int among) {
    constexpr int kQLanes = D / 16, kQRows = 32 / kQLanes;
#pragma unroll 1
    for (int r0 = w * kQRows; r0 < kR; r0 += among * kQRows) {
      const int r = r0 + lane / kQLanes;
      const uint32_t down = q_row_to_f8<kQLanes>(
          [&](int ch) {
            return reinterpret_cast<uint4*>(smem + C::kOffQ + (ch >> 3) * (kR * 128) + r * 128 +
                                            (((ch & 7) ^ (r & 7)) << 4));
          },
          lane);
      if (lane % kQLanes == 0) s_qs[(n & 3) * 64 + r] = (uint8_t)down;
    }
    fence_proxy_async_smem();
    __syncwarp();
  };

  if (warp >= kQkWarp && warp < kEpiWarp0) setmaxnreg_dec<64>();
  if (warp == kKeyWarp) {
    bool ok = true;
    int g = 0;
    if constexpr (TMA) {
      // ===================================================== keys by TMA
      // Lane i < 4 loads rows 16 i .. of the CTA's 64.
      const int behind = (int)((p.g.total_pages - p.g.base) / 8);
      bool over = false;
      Walk c;  // runs a tile ahead of the copies
      c.init(p.g, begin);
      auto box_of = [&]() {
        return lane < 4 ? box_group(p, error, c, c.start() + rank * kHalf + lane * 16, &over) : behind;
      };
      int y = behind;
      if (c.left > 0) {
        y = box_of();
        c.next(p.g);
      }
      for (; g < nt; ++g) {
        const int s = g % KS;
        if (g >= KS) ok = tile_wait(bar(kKFree0 + s), ((g / KS) - 1) & 1, wc);
        if (!ok) break;
        // (CTA 1's bytes may land before CTA 0 has said how many to expect: the
        // barrier's phase cannot end before that arrival)
        if (rank == 0 && lane == 0) mbar_arrive_expect_tx(bar(kKFull0 + s), 2 * C::kKBytes);
        __syncwarp();
        if (lane < 4)
          tma_pair_4d(sK + s * C::kKBytes + lane * C::kBox, &tmap_kv, 0, 0, 0, y, bar0(kKFull0 + s));
        if (c.left > 0) {  // (after this tile's copies: the table entry is a while coming)
          y = box_of();
          c.next(p.g);
        }
      }
      if (over) atomicExch(error, 3);
    } else {
      // ===================================================== passing on landed keys
      for (; g < nt; ++g) {
        const int s = g % KS;
        ok = tile_wait(bar(kKLanded0 + s), (g / KS) & 1, wc);
        if (!ok) break;
        fence_proxy_async_smem();  // the copies were made through the generic proxy
        if (lane == 0) arrive_cluster(bar0(kKFull0 + s));
        __syncwarp();
      }
    }
    // Every stage that was filled has been read (so its copies have landed) and
    // every arrival of the MMA warps has come in before this CTA's memory goes away.
    for (int x = max(0, g - KS); x < g; ++x) pipe_drain(bar(kKFree0 + x % KS), (x / KS) & 1, wc);
  } else if (warp == kLookWarp) {
    // ===================================================== rows and scales of the positions
    UnitWalk uw;
    uw.init(p.g, 2 * kR, begin);
    bool ok = true;
    for (int g = 0, pieces = 0; g < nt && ok; ++pieces) {
      if (pieces > 0) uw.next(p.g, 2 * kR);
      const ChunkUnit un = chunk_unit(p.g, 2 * kR, kTile, uw.b, uw.r);
      const int i0 = g == 0 ? begin.off : 0, i1 = min(un.ntiles, i0 + nt - g);
      const int p_hi = un.pos0 + div_h(p.g, un.h0 + un.nrows - 1), window = p.g.window;
      for (int i = i0; i < i1; ++i, ++g) {
        const int s = g % kLook, j0 = chunk_tile_start(i, un.nf, un.lo, kTile);
        float sc[4];
        int row[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) row[x] = code_row(fp, error, un, j0 + 32 * x + lane, &sc[x]);
#pragma unroll
        for (int x = 0; x < 4; ++x) {  // (the values' loads follow some tiles later)
          if (row[x] >= 0) {
#pragma unroll
            for (int d = 0; d < D / 2; d += 128)
              prefetch_line(fp.codes + (size_t)row[x] * D + rank * (D / 2) + d);
          }
        }
        if (g >= kLook) ok = tile_wait(bar(kLkFree0 + s), ((g / kLook) - 1) & 1, wc);
        if (!ok) break;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          s_scale[s * kTile + 32 * x + lane] = sc[x];
          s_row[s * kTile + 32 * x + lane] = row[x];
        }
        if (lane == 0)  // whether some row of the unit does not see all of the tile
          s_mask[s] = !(j0 + kTile - 1 <= un.pos0 &&
                        (window == 0 || j0 > p_hi - window || j0 + kTile <= p.g.first));
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kLkFull0 + s));
      }
    }
    // (as the key warp's)
    for (int x = max(0, 4 * nt - VS); x < 4 * nt; ++x) pipe_drain(bar(kVFree0 + x % VS), (x / VS) & 1, wc);
    for (int x = max(0, nt - 2); x < nt; ++x) pipe_drain(bar(kPFree0 + (x & 1)), (x >> 1) & 1, wc);
  } else if (warp >= kLoadWarp0) {
    // ===================================================== values (and keys one by one)
    setmaxnreg_dec<72>();
    constexpr int NL = C::kLoads, kRowsPer = C::kRowsPer;
    // Warps 0..3 fill the even stages, 4..7 the odd ones.  A load takes kRowsPer rows: eight
    // lanes in a row, whose stores follow one another, are four 16-byte pieces of each of
    // two rows, and so meet all banks.
    const int w8 = warp - kLoadWarp0, v = w8 & 3;
    const int sub = D == 512 ? (lane >> 2) & 1 : ((lane >> 2) & 1) | ((lane >> 4) << 1);
    const int c16 = (lane & 3) | ((D == 512 ? lane >> 3 : (lane >> 3) & 1) << 2);
    const uint8_t* half_of = fp.codes + rank * (D / 2) + c16 * 16;
    uint4 x[NL];
    auto load = [&](int st) {  // stage st: quarter st % 4 of tile st / 4
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        const int from = s_row[(st & (4 * kLook - 1)) * kQuarter + v * 8 + i * kRowsPer + sub];
        x[i] = make_uint4(0, 0, 0, 0);
        if (from >= 0) x[i] = load_codes(half_of + (size_t)from * D);
      }
    };
    auto keys = [&](int g) {  // tile g's, of the CTA's half of the positions
      const int s = g % KS;
      if (g >= KS && !tile_wait(bar(kKFree0 + s), ((g / KS) - 1) & 1, wc)) return false;
      constexpr int kL = D / 16, kPer = 32 / kL;
#pragma unroll
      for (int i = 0; i < 8; i += kPer) {
        const int ch = lane % kL, r = w8 * 8 + i + lane / kL;
        const int from = s_row[(g % kLook) * kTile + rank * kHalf + r];
        cp_async16(sK + s * C::kKBytes + (r >> 3) * C::kGroupK + (ch >> 3) * 1024 + (r & 7) * 128 +
                       (((ch & 7) ^ (r & 7)) << 4),
                   from >= 0 ? fp.codes + (size_t)from * D + ch * 16 : fp.codes, from >= 0 ? 16u : 0u);
      }
      cp_async_arrive(bar(kKLanded0 + s));  // once this thread's copies have landed
      return true;
    };
    auto looked_up = [&](int g) { return tile_wait(bar(kLkFull0 + g % kLook), (g / kLook) & 1, wc); };
    auto rows_read = [&](int g) {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kLkFree0 + g % kLook));
    };
    bool ok = nt > 0 && looked_up(0);
    if (ok) {
      load(w8 >> 2);
      if constexpr (!TMA) ok = keys(0);
    }
#pragma unroll 1
    for (int st = w8 >> 2; st < 4 * nt && ok; st += 2) {
      const int g = st >> 2, s = st % VS;
      const bool masked = s_mask[g % kLook] != 0;
      if (st & 2) {  // this warp's next stage is another tile's
        rows_read(g);
        if (g + 1 < nt) {
          ok = looked_up(g + 1);
          if constexpr (!TMA) ok = ok && keys(g + 1);  // a tile ahead of the values
        }
      }
      if (ok && st >= VS) ok = tile_wait(bar(kVFree0 + s), ((st / VS) - 1) & 1, wc);
      if (!ok) break;
      const uint32_t stage = sV + s * C::kVBytes + v * C::kGroupV + (c16 >> 2) * 1024;
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        uint32_t f[8];
        codes_to_f16(x[i].x, f[0], f[1]);
        codes_to_f16(x[i].y, f[2], f[3]);
        codes_to_f16(x[i].z, f[4], f[5]);
        codes_to_f16(x[i].w, f[6], f[7]);
        // A value of NaN has a weight of NaN where it is seen; where it is not, 0 x NaN
        // would be NaN, too: any number does in its place.
        if (masked) {
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = f16_number(f[e]);
        }
        const int r = i * kRowsPer + sub, ch = 2 * (c16 & 3);
        st_shared16(stage + r * 128 + ((ch ^ r) << 4), f[0], f[1], f[2], f[3]);
        st_shared16(stage + r * 128 + (((ch + 1) ^ r) << 4), f[4], f[5], f[6], f[7]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) arrive_cluster(bar0(kVFull0 + s));
      __syncwarp();
      // (behind the fence, which waits for all of the thread's memory operations)
      if (st + 2 < 4 * nt) load(st + 2);
    }
    if constexpr (!TMA) cp_async_wait_all();
  } else if (warp == kQkWarp) {
    // ===================================================== q loads (both), QK MMAs (CTA 0)
    Walk c;
    c.init(p.g, begin);
    constexpr uint32_t kQBytes = C::kPanelsQ * kR * 128;
    int pieces = 0;
    bool ok = true;
    auto load_q = [&]() {
      const int row = c.row0 + rank * kR;
      if (elect_one()) {
        mbar_arrive_expect_tx(bar(kQFull), kQBytes);
#pragma unroll
        for (int x = 0; x < C::kPanelsQ; ++x)
          tma_load_2d(sQ + x * kR * 128, &tmap_q, x * 64, row, bar(kQFull));
      }
      __syncwarp();
    };
    bool loaded = false;
    if (c.left > 0) {
      load_q();
      loaded = true;
    }
    for (int g = 0; g < nt; ++g) {
      const int s = g & 1, ks = g % KS;
      const bool last = c.last();
      if (rank == 0) {
        // keys, room for the scores and q, with one wait (a barrier that is not waited for: the
        // keys' once more)
        const uint32_t on = lane == 0 && g >= 2 ? kSEmpty0 + s : lane == 1 && c.first ? kQReady : kKFull0 + ks;
        const int parity = lane == 0 && g >= 2 ? (g >> 1) - 1 : lane == 1 && c.first ? pieces : g / KS;
        ok = tile_wait(bar(on), parity & 1, wc);
        if (!ok) break;
        if (!TMA) fence_proxy_async_smem();
        tc_fence_after();
        if (elect_one()) {
          constexpr uint32_t HQ = desc_hi(1024), HK = desc_hi(C::kGroupK);
          uint32_t a = desc_lo(sQ, 16), b = desc_lo(sK + ks * C::kKBytes, 16);
          const uint32_t d = tmem + s * 64;
          // (a loop: the instructions of all roles have to stay in the instruction cache)
#pragma unroll 1
          for (uint32_t pn = 0; pn < C::kPanelsK; ++pn, a += kR * 128 / 16, b += 1024 / 16) {
#pragma unroll
            for (uint32_t k = 0; k < 4; ++k) {
              mma_of<true, HQ, HK>(d, a + 2 * k, b + 2 * k, C::kIdescQ1, k ? 1u : pn);
              mma_of<true, HQ, HK>(d, a + C::kPanelsK * kR * 8 + 2 * k, b + 2 * k, C::kIdescQ2, 1u);
            }
          }
          commit_pair(bar(kSFull0 + s));
          commit_pair(bar(kKFree0 + ks));
          if (last) commit_pair(bar(kQEmpty));
        }
        __syncwarp();
      }
      c.next(p.g);
      if (last) {  // q of the next unit, once this unit's MMAs have read q
        ok = tile_wait(bar(kQEmpty), pieces & 1, wc);
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
    if (loaded) pipe_drain(bar(kQFull), pieces & 1, wc);
  } else if (warp == kPvWarp) {
    // ===================================================== decision, PV MMAs (CTA 0)
    if (rank == 0) {
      Walk c;
      c.init(p.g, begin);
      volatile int* flag = reinterpret_cast<volatile int*>(smem + C::kOffFlag);
      int scaled = 0, pieces = 0, said = 0;  // said: bits 2 s ..: what buffer s of the commands holds
      uint32_t vs = 0, vphase = 0;           // stage of values
      for (int g = 0; g < nt; ++g) {
        const int s = g & 1;
        int cmd = 0;
        auto tell = [&]() {  // one lane tells each CTA
          if (lane < 2) {
            if (cmd != ((said >> (2 * s)) & 3)) {
              store_cluster(map_cta(sbase + C::kOffCmd + 4 * s, lane), (uint32_t)cmd);
              fence_cluster();
            }
            arrive_cluster(map_cta(bar(kDecided0 + s), lane));
          }
          said = (said & ~(3 << (2 * s))) | cmd << (2 * s);
          __syncwarp();
        };
        uint32_t add = c.first ? 0u : 1u;
        bool ok = true;
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          // this half's weights and its two stages of values, with one wait
          const uint32_t vs1 = vs + 1 == VS ? 0 : vs + 1, vphase1 = vs + 1 == VS ? vphase ^ 1 : vphase;
          const uint32_t on = lane == 0 ? kPReady0 + 2 * s + h : kVFull0 + (lane == 1 ? vs : vs1);
          ok = tile_wait(bar(on), lane == 0 ? (g >> 1) & 1 : lane == 1 ? vphase : vphase1, wc);
          if (!ok) break;
          if (h == 0) {
            const int f0 = flag[2 * s], f1 = flag[2 * s + 1];
            cmd = (f0 ? kRaise0 : 0) | (f1 ? kRaise1 : 0);
            if (cmd) {
              tell();
              fence_cluster();
              if (lane < 2) flag[2 * s + lane] = 0;  // for tile g + 2, which says nothing unless it has to
              ok = tile_wait(bar(kScaled), scaled & 1, wc);
              ++scaled;
            }
            // O^T of the piece before has been read
            if (ok && c.first && pieces > 0) ok = tile_wait(bar(kODone), (pieces - 1) & 1, wc);
            pieces += c.first;
            if (!ok) break;
          }
          tc_fence_after();
          if (elect_one()) {
            constexpr uint32_t HV = desc_hi(C::kGroupV), HP = desc_hi(1024);
            const uint32_t b = desc_lo(sP + (2 * s + h) * C::kPHalf, 16);
#pragma unroll
            for (int qt = 0; qt < 2; ++qt) {
              const uint32_t a = desc_lo(sV + (qt ? vs1 : vs) * C::kVBytes, 1024);
#pragma unroll
              for (int blk = 0; blk < C::kBlocks; ++blk) {
#pragma unroll
                for (int k = 0; k < kQuarter / 16; ++k)
                  mma_of<false, HV, HP>(tmem + C::kOCol + blk * 128, a + (2 * blk * 1024 + k * 2 * C::kGroupV) / 16,
                                        b + 4 * qt + 2 * k, C::kIdescPV, qt || k ? 1u : add);
              }
              commit_pair(bar(kVFree0 + (qt ? vs1 : vs)));
            }
            if (h) commit_pair(bar(kPFree0 + s));
          }
          __syncwarp();
          add = 1u;
          vphase = vs1 + 1 == VS ? vphase1 ^ 1 : vphase1;
          vs = vs1 + 1 == VS ? 0 : vs1 + 1;
          if (h == 0 && !cmd) tell();  // (looked at once the next tile's weights are there)
        }
        if (!ok) break;
        c.next(p.g);
      }
    }
  } else if (warp < kSmWarps) {
    // ===================================================== softmax and epilogue
    // Warp w reads TMEM lane quadrant q4 = w % 4 -- rows 32 (q4 % 2) .. + 31 at the
    // tile's positions 64 kh .., kh = q4 / 2 -- and of these the 32 positions from
    // 32 hc on, hc = w / 4.  Thread t holds rows base + t / 4 + 8 i, i = 0..3, at the
    // positions 8 rep + 2 (t % 4) + {0, 1}, rep = 0..3: element 8 i + 2 rep + {0, 1}.
    setmaxnreg_inc<104>();
    const int q4 = warp & 3, hc = warp >> 2, st = threadIdx.x, tq = lane & 3;
    const int kh = q4 >> 1, rb = (q4 & 1) * 32, part = 2 * kh + hc, row0 = rb + (lane >> 2);
    const uint32_t lane_base = (uint32_t)(q4 * 32) << 16;
    float* s_alpha = reinterpret_cast<float*>(smem + C::kOffAlpha);
    float* s_fac = reinterpret_cast<float*>(smem + C::kOffFac);
    float* s_part = reinterpret_cast<float*>(smem + C::kOffPart);
    volatile int* s_cmd = reinterpret_cast<volatile int*>(smem + C::kOffCmd);
    const float sc = p.qk_scale_log2 / kWeightUnit;
    const int H = p.g.H, window = p.g.window, nfirst = p.g.first;
    const uint32_t s_empty = bar0(kSEmpty0), p_ready = bar0(kPReady0);  // (8 bytes a barrier)
    const uint32_t my_flag = map_cta(sbase + C::kOffFlag, 0) + 4 * rank;
    int g = 0, pieces = 0;
    if (nt > 0) {  // (nothing else to do until the first scores come)
      if (tile_wait(bar(kQFull), 0, wc)) q_to_f8(0, kEpiWarps + warp, kEpiWarps + kSmWarps);
      named_bar_sync(2, kSmThreads + kEpiWarps * 32);
    }
    // What was decided on tile x: scales O^T if it has to be (the PV MMAs of tile x wait
    // for that).  Uniform over both CTAs' softmax warps.
    auto decided = [&](int x) {
      const int s = x & 1;
      tile_wait(bar(kDecided0 + s), (x >> 1) & 1, wc);
      const int cmd = *abort_flag ? 0 : s_cmd[s];
      if (cmd == 0) return;
      fence_cluster();
      {
        // O^T is quiescent once the PV MMAs of tile x - 1 are done
        if (x > 0) tile_wait(bar(kPFree0 + ((x - 1) & 1)), ((x - 1) >> 1) & 1, wc);
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
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        m[i] = kNoScore;
        l[i] = 0.f;
        scr[i] = 0.f;
      }
      for (int i = i0; i < i1; ++i, ++g) {
        const int s = g & 1;
        const int j0 = chunk_tile_start(i, un.nf, un.lo, kTile);
        // whether every row of this CTA sees the whole tile
        const bool full = j0 + kTile - 1 <= p_lo &&
                          (window == 0 || j0 > p_hi - window || j0 + kTile <= nfirst);
        // the scores, and the positions' scales, with one wait
        tile_wait(bar(lane == 0 ? kSFull0 + s : kLkFull0 + g % kLook), (lane == 0 ? g >> 1 : g / kLook) & 1, wc);
        tc_fence_after();
        if (i == i0) {
          // (rows past the unit's end have factor 0: their weights, never used, stay
          // finite and raise nothing; a row of q with an infinity or NaN has NaN)
#pragma unroll
          for (int i4 = 0; i4 < 4; ++i4) {
            const uint32_t e = s_qs[(pieces & 3) * 64 + row0 + 8 * i4];
            scr[i4] = row0 + 8 * i4 < nrows ? sc * q_factor(e) : 0.f;
          }
        }
        // kWeightUnit s_j of positions 8 rep + 2 (t % 4) + {0, 1}
        uint64_t sj[4];
#pragma unroll
        for (int rep = 0; rep < 4; ++rep)
          sj[rep] = *reinterpret_cast<const uint64_t*>(s_scale + (g % kLook) * kTile + 64 * kh + 32 * hc +
                                                       8 * rep + 2 * tq);
        uint32_t see = 0xffffffffu;  // bit 8 i + 2 rep + k: row i and that position see each other
        if (!full) {
          // bits 0, 1, 8, 9 of a row's ten positions are four of its elements
          see = 0;
#pragma unroll
          for (int i4 = 0; i4 < 4; ++i4) {
            const int pos = un.pos0 + div_h(p.g, h0 + row0 + 8 * i4);
#pragma unroll
            for (int r2 = 0; r2 < 2; ++r2) {
              const uint32_t m10 =
                  seen_bits(pos, j0 + 64 * kh + 32 * hc + 16 * r2 + 2 * tq, window, nfirst);
              see |= ((m10 & 3u) | ((m10 >> 6) & 12u)) << (8 * i4 + 4 * r2);
            }
          }
        }
        // The scores are read from TMEM whenever they are needed (twice and a third time
        // where the reference is set), so that no register holds them over a barrier.
        auto scores = [&](int half, auto use) {  // use(row i, rep, pair of scaled scores)
          uint32_t v[16];
          tmem_ld_16x256b_x4(tmem + lane_base + ((uint32_t)(16 * half) << 16) + s * 64 + 32 * hc, v);
          tmem_wait_ld();
          // register 4 rep + k: row + 8 (k / 2), position 8 rep + 2 (t % 4) + k % 2
#pragma unroll
          for (int i2 = 0; i2 < 2; ++i2) {
#pragma unroll
            for (int rep = 0; rep < 4; ++rep)
              use(2 * half + i2, rep,
                  f2_mul(f2_pack(__uint_as_float(v[4 * rep + 2 * i2]), __uint_as_float(v[4 * rep + 2 * i2 + 1])),
                         sj[rep]));
          }
        };
        // w = kWeightUnit s_j 2^(x scale - m) in f16; the denominator sums the unrounded 2^(..).
        float sum[4];
        uint32_t pk[4][4];
        auto weights = [&](auto masked) {
          uint32_t top = 0;  // largest size of the weights, two f16
          uint64_t both[4] = {0, 0, 0, 0};
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            scores(half, [&](int i4, int rep, uint64_t x) {
              float a0, a1;
              f2_unpack(x, a0, a1);
              a0 = fmaf(a0, scr[i4], -m[i4]);
              a1 = fmaf(a1, scr[i4], -m[i4]);
              if constexpr (decltype(masked)::value) {
                a0 = (see >> (8 * i4 + 2 * rep)) & 1u ? a0 : -INFINITY;
                a1 = (see >> (8 * i4 + 2 * rep + 1)) & 1u ? a1 : -INFINITY;
              }
              a0 = ex2_approx(a0);
              a1 = ex2_approx(a1);
              const uint64_t pr = f2_pack(a0, a1);
              both[i4] = f2_add(both[i4], pr);
              f2_unpack(f2_mul(pr, sj[rep]), a0, a1);
              if constexpr (decltype(masked)::value) {  // (0 x a scale that is no number)
                a0 = (see >> (8 * i4 + 2 * rep)) & 1u ? a0 : 0.f;
                a1 = (see >> (8 * i4 + 2 * rep + 1)) & 1u ? a1 : 0.f;
              }
              pk[i4][rep] = pack_f16(a0, a1);
              top = f16_top(top, pk[i4][rep]);
            });
          }
#pragma unroll
          for (int i4 = 0; i4 < 4; ++i4) {
            float t0, t1;
            f2_unpack(both[i4], t0, t1);
            sum[i4] = t0 + t1;
          }
          return max(top & 0xffffu, top >> 16) > kWeightTopBits ||
                 fmaxf(fmaxf(sum[0], sum[1]), fmaxf(sum[2], sum[3])) > kSumTop;
        };
        // The first tile of a piece sets m to its exact row maxima; a later one is
        // weighted against the current m, and only if a weight exceeds the headroom is m
        // raised.
        int flags = 0;
        bool exact = i == i0, again = true;
        if (!exact && full) {
          exact = named_bar_or(1, kSmThreads, weights(std::false_type{}));
          again = exact;
        }
        // (one piece of code for masked tiles and for the rare ones)
#pragma unroll 1
        while (again) {
          if (exact) {
            float* hm = s_part + (g & 1) * 256;
            float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              scores(half, [&](int i4, int rep, uint64_t x) {
                float x0, x1, s0, s1;
                f2_unpack(x, x0, x1);
                f2_unpack(sj[rep], s0, s1);
                if ((see >> (8 * i4 + 2 * rep)) & 1u) top[i4] = fmaxf(top[i4], fmaf(x0, scr[i4], scale_log(s0)));
                if ((see >> (8 * i4 + 2 * rep + 1)) & 1u) top[i4] = fmaxf(top[i4], fmaf(x1, scr[i4], scale_log(s1)));
              });
            }
#pragma unroll
            for (int i4 = 0; i4 < 4; ++i4) {
              top[i4] = fmaxf(top[i4], __shfl_xor_sync(0xffffffffu, top[i4], 1));
              top[i4] = fmaxf(top[i4], __shfl_xor_sync(0xffffffffu, top[i4], 2));
              if (tq == 0) hm[part * 64 + row0 + 8 * i4] = top[i4];
            }
            named_bar_sync(1, kSmThreads);
            // (both CTAs are done with the factors of tile g - 2, in whose place these go)
            if (g >= 2) tile_wait(bar(kPFree0 + s), ((g >> 1) - 1) & 1, wc);
#pragma unroll
            for (int i4 = 0; i4 < 4; ++i4) {
              const int r = row0 + 8 * i4;
              const float t = fmaxf(fmaxf(hm[r], hm[64 + r]), fmaxf(hm[128 + r], hm[192 + r]));
              float alpha = 1.f;
              if (t > m[i4] + kHeadroom) {
                alpha = ex2_approx(m[i4] - t);  // 0 when there was no score
                l[i4] = times_exp2(l[i4], m[i4] - t);
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
          }
          const bool over = weights(std::true_type{});
          again = false;
          if (!exact) again = exact = named_bar_or(1, kSmThreads, over);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          arrive_cluster(s_empty + 8 * s);
          mbar_arrive(bar(kLkFree0 + g % kLook));
        }
        // Into P (K-major, 128-byte swizzle), once the PV MMAs of tile g - 2 have read it.
        if (g >= 2) tile_wait(bar(kPFree0 + s), ((g >> 1) - 1) & 1, wc);
        {
          // matrices of a stmatrix.x4: rows + 8 (mi % 2), chunk + mi / 2
          const int mi = lane >> 3, r8 = lane & 7;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int r = rb + 16 * half + 8 * (mi & 1) + r8;
            const uint32_t row = sP + (2 * s + kh) * C::kPHalf + (r >> 3) * 1024 + r8 * 128;
#pragma unroll
            for (int c2 = 0; c2 < 2; ++c2) {
              const int ch = 4 * hc + 2 * c2 + (mi >> 1);
              stmatrix_x4(row + ((ch ^ r8) << 4), pk[2 * half][2 * c2], pk[2 * half + 1][2 * c2],
                          pk[2 * half][2 * c2 + 1], pk[2 * half + 1][2 * c2 + 1]);
            }
          }
        }
        fence_proxy_async_smem();
#pragma unroll
        for (int i4 = 0; i4 < 4; ++i4) l[i4] += sum[i4];
        // What was decided on tile g - 1 has long come in by now; its PV MMAs, if they
        // wait for O^T to be scaled, come before tile g's.
        if (g > 0) decided(g - 1);
        __syncwarp();
        if (lane == 0) {
          if (st == 0 && flags) {  // (before this warp's arrival on the first half)
            store_cluster(my_flag + 8 * s, (uint32_t)flags);
            fence_cluster();
          }
          arrive_cluster(p_ready + 16 * s + 8 * kh);
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
      if (pieces > 0) tile_wait(bar(kODone), (pieces - 1) & 1, wc);
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
              const float den = denominator(lr, mr - M, ex2_approx(ms - M));
              f = a / den / kWeightUnit;
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
    setmaxnreg_dec<64>();
    int g = 0, pieces = 0;
    UnitWalk uw;
    uw.init(p.g, 2 * kR, begin);
    auto convert_q = [&](int n, int among) {
      const bool ok = tile_wait(bar(kQFull), n & 1, wc);
      if (ok) q_to_f8(n, q4, among);
      if (n == 0) named_bar_sync(2, kSmThreads + kEpiWarps * 32);
      if (ok && lane == 0) arrive_cluster(bar0(kQReady));
      __syncwarp();
    };
    if (nt > 0) convert_q(0, kEpiWarps + kSmWarps);
    while (g < nt) {
      if (pieces > 0) uw.next(p.g, 2 * kR);
      const ChunkUnit un = chunk_unit(p.g, 2 * kR, kTile, uw.b, uw.r);
      const int i0 = g == 0 ? begin.off : 0;
      const int i1 = min(un.ntiles, i0 + nt - g);
      const bool whole = i0 == 0 && i1 == un.ntiles;
      g += i1 - i0;
      if (g < nt) convert_q(pieces + 1, kEpiWarps);  // (its QK MMAs wait; this unit's last weights come later)
      tile_wait(bar(kFac), pieces & 1, wc);
      tile_wait(bar(kPFree0 + ((g - 1) & 1)), ((g - 1) >> 1) & 1, wc);  // O^T is complete
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
            for (int e = 0; e < 16; ++e) o[(size_t)e * D] = __uint_as_float(ov[e]) / kWeightUnit;
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
#define SDA_CASE(DV)                                                         \
  if (D == DV)                                                               \
    return tma ? f(chunk_pair_fp8_kernel<DV, true>, (size_t)Cfg<DV>::kSmem)  \
               : f(chunk_pair_fp8_kernel<DV, false>, (size_t)Cfg<DV>::kSmem);
  SDA_CASE(256) SDA_CASE(512)
#undef SDA_CASE
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t pair_fp8_prepare() {
  for (int D : {256, 512}) {
    for (bool tma : {false, true}) {
      const cudaError_t e = for_shape(D, tma, [&](auto kernel, size_t smem) {
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
  return cudaSuccess;
}

cudaError_t launch_chunk_pair_fp8(const CUtensorMap& tq, const CUtensorMap& tkv, const ChunkFp8Params& p,
                                  bool tma, const ChunkLayout& L, cudaStream_t st) {
  return for_shape(p.c.g.D, tma, [&](auto kernel, size_t smem) {
    return launch_pdl_cluster(kernel, dim3(2 * L.grid), dim3(kThreads), 2, smem, st, tq, tkv, p);
  });
}

}  // namespace sda
