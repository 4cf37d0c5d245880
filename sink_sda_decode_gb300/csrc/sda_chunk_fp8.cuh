// sda_chunk_fp8.cuh -- what the chunk attention over an 8-bit cache shares between its two
// kernels.
//
// The cache holds E4M3 codes and one scale for each block: position j's row is
// s_j c_j, s_j the scale of its block.  Codes become f16 in shared memory (E4M3 fits f16
// exactly, and one instruction converts two codes, where bf16 takes nine for four); q,
// bf16 in memory, becomes f16 too, each row times the power of two that brings its largest
// element to [2^14, 2^15): elements down to 2^-28 of that stay exact, smaller ones are off
// by at most 2^-39 of it.  The scales stay outside the MMAs:
//   x_j = scale 2^-k s_j <2^k q, c_j>,   out = sum_j (p_j s_j) c_j / den,   den = sum_j p_j + ..
// with p_j = 2^(x_j log2 e - m).  The weights w_j = 2^3 p_j s_j are rounded to f16, 2^-11 of
// themselves.  So that they fit, the reference m of a row follows x_j log2 e + log2 |s_j|
// (log2 |s_j| not below -90), not x_j alone: w_j is at most 2^3 when m is set and 2^15
// before it is raised, and one below 2^-14 is off by at most 2^-25, so 2^-28 of a
// weight at the reference (over 2^16 positions that is 2^-12 of it at worst).  With 2^7 in
// the place of 2^3, m is raised often where scales differ: drafted tokens 95 us, now 86.  The denominator's p_j are fp32 and at most 2^102.
#pragma once

#include <cuda_fp16.h>

#include "sda_chunk_dev.cuh"
#include "sda_rows.cuh"

namespace sda {

struct ChunkFp8Params {
  ChunkParams c;
  const uint8_t* codes;  // [total_pages, D] E4M3
  const float* scale;    // a scale for each block
  uint32_t k_mul;        // j / k_per_block = j k_mul >> k_shift, as div_h has it
  int k_shift;
};

cudaError_t chunk_fp8_prepare();
cudaError_t pair_fp8_prepare();
cudaError_t launch_chunk_pair_fp8(const CUtensorMap& tq, const CUtensorMap& tkv, const ChunkFp8Params& p,
                                  bool tma, const ChunkLayout& L, cudaStream_t st);
ChunkLayout chunk_fp8_layout(const ChunkGeom& g, int num_sms);
cudaError_t launch_chunk_fp8(const void* q, const void* codes, const float* scale, const ChunkGeom& g,
                             const float* attn_sink, float softmax_scale, void* out, float* lse,
                             const ChunkLayout& L, void* ws, cudaStream_t st);

// The way by rows of bf16 in the workspace (sda_spread.cu), from byte `from` of it on.
struct SpreadLayout {
  bool worth;
  int S, n_bad;
  size_t rows_off, scale_off, bad_off, table_off, total;
};
SpreadLayout spread_layout(const ChunkGeom& g, int num_sms, size_t from);
ChunkGeom spread_geometry(const ChunkGeom& g, const SpreadLayout& L, void* ws);
cudaError_t launch_spread(const ChunkGeom& g, const void* codes, const float* scale, const SpreadLayout& L,
                          void* ws, cudaStream_t st);
cudaError_t launch_chunk_spread(const void* q, const ChunkGeom& s, const float* attn_sink, float softmax_scale,
                                void* out, float* lse, const ChunkLayout& C, const SpreadLayout& L, void* ws,
                                cudaStream_t st);

#ifdef __CUDACC__
__device__ __forceinline__ float q_factor(uint32_t e) { return __uint_as_float(e << 23 | (e == 255u ? 1u : 0u)); }
constexpr float kWeightUnit = 8.f;         // w_j = kWeightUnit p_j s_j
constexpr float kWeightTop = 32768.f;      // a weight above this raises the reference
constexpr uint32_t kWeightTopBits = 0x7800u;  // it, as f16
constexpr float kSumTop = 5.0706024e30f;   // 2^102: so does a share of the denominator above this (of at
                                           // most 8 p_j, so that one is above 2^98)
constexpr float kLeastLog = -90.f;         // of a scale, for the reference

// log2 |s| as the reference uses it, of kWeightUnit s.
__device__ __forceinline__ float scale_log(float su) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(fabsf(su)));
  return fmaxf(y - 3.f, kLeastLog);
}

// l 2^d + sink, d <= 0 (-inf: the row has no score, and l is 0).
__device__ __forceinline__ float denominator(float l, float d, float sink) {
  return d >= -126.f ? fmaf(l, ex2_approx(d), sink) : times_exp2(l, d) + sink;
}

// warp_wait in less code: these kernels wait at some forty places, and the instructions of
// all roles have to stay in the instruction cache (a pair kernel of 205 KB had 30 % of its
// warps waiting for instructions).  The first try has no time to sleep: 26 cycles where the
// phase is over, 59 with one.
__device__ __forceinline__ bool tile_wait(uint32_t bar, uint32_t parity, const PipeWait& w) {
  bool ok = true;
  if (!ptx::mbar_try_wait(bar, parity)) {
    uint64_t t0 = 0;
#pragma unroll 1
    while (!mbar_try_wait_for(bar, parity, kWaitHintNs)) {
      const uint64_t t = ptx::globaltimer_ns();
      if (t0 == 0) t0 = t;
      if (t - t0 > w.timeout_ns) {
        *w.abort_flag = 1;
        atomicExch(w.error, 1);
      }
      if (*w.abort_flag) {
        ok = false;
        break;
      }
    }
  }
  return __all_sync(0xffffffffu, ok);
}

// Asks for a 128-byte line of L2.  (A bulk prefetch costs the copy engine about 80 cycles a
// row: a prompt chunk took 4.36 ms with them.)
__device__ __forceinline__ void prefetch_line(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p) : "memory");
}

// 16 bytes that are used once: past L1, which the registers spilled elsewhere need.
__device__ __forceinline__ uint4 load_codes(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// Four codes to f16, in order.
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

__device__ __forceinline__ void st_shared16(uint32_t dst, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

// Pool row and scale (times kWeightUnit) of position j of the cursor's unit; -1 and 0
// where no row of the unit sees it, or outside the pool (which raises the error word).
template <typename C>
__device__ __forceinline__ int code_row(const ChunkFp8Params& p, int* error, const C& c, int j, float* su) {
  *su = 0.f;
  if (j >= c.hi || (j < c.lo && j >= p.c.g.first)) return -1;
  const ChunkGeom& g = p.c.g;
  const int jb = (int)(((unsigned long long)(unsigned)j * p.k_mul) >> p.k_shift);
  const int blk = __ldg(g.block_table + (size_t)c.b * g.max_blocks + jb);
  const long long row = g.base + (long long)blk * g.k_per_block + (j - jb * g.k_per_block);
  if (blk < 0 || row >= g.total_pages) {
    atomicExch(error, 3);
    return -1;
  }
  *su = __ldg(p.scale + blk) * kWeightUnit;
  return (int)row;
}

// One row of q in shared memory (D / 8 chunks of 16 bytes over LANES lanes, `at(ch)` the
// place of chunk ch) from bf16 to f16 times a power of two; returns the exponent (as fp32
// holds it) of its inverse, or 255 for a row that holds an infinity or NaN.
template <int D, typename At>
__device__ __forceinline__ uint32_t q_row_to_f16(At at, int lane) {
  constexpr int kLanes = D / 8 < 32 ? D / 8 : 32, kCh = D / 8 / kLanes;
  uint4 v[kCh];
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < kCh; ++k) {
    v[k] = *at(lane % kLanes + k * kLanes);
    const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) top = __vmaxu2(top, w[e] & 0x7fff7fffu);
  }
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
  const uint32_t most = max(top & 0xffffu, top >> 16);
  const int k2 = most == 0 ? 0 : min(14 + 127 - (int)(most >> 7), 126);
  const float up = __uint_as_float((uint32_t)(127 + k2) << 23);
#pragma unroll
  for (int k = 0; k < kCh; ++k) {
    const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
    uint32_t h[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __half2 x = __floats2half2_rn(__uint_as_float(w[e] << 16) * up,
                                          __uint_as_float(w[e] & 0xffff0000u) * up);
      h[e] = *reinterpret_cast<const uint32_t*>(&x);
    }
    *at(lane % kLanes + k * kLanes) = make_uint4(h[0], h[1], h[2], h[3]);
  }
  return most >= 0x7f80u ? 255u : (uint32_t)(127 - k2);
}

// Instruction descriptor of kind::f16 with f16 A / B and fp32 D (idesc_bf16_f32's fields).
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool a_mn) {
  return (1u << 4) | ((a_mn ? 1u : 0u) << 15) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// Of two pairs of f16, the larger sizes (a NaN is smaller than any).
__device__ __forceinline__ uint32_t f16_top(uint32_t top, uint32_t w) {
  const __half2 r = __hmax2(*reinterpret_cast<const __half2*>(&top), __habs2(*reinterpret_cast<const __half2*>(&w)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// Two f16 with a number in the place of a NaN.
__device__ __forceinline__ uint32_t f16_number(uint32_t w) {
  const __half2 r = __hmax2(*reinterpret_cast<const __half2*>(&w), __half2half2(__ushort_as_half(0xfbffu)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// Whether one of two f16 is an infinity or NaN.
__device__ __forceinline__ bool f16_bad(uint32_t w) {
  return (w & 0x7c00u) == 0x7c00u || (w & 0x7c000000u) == 0x7c000000u;
}
#endif

}  // namespace sda
