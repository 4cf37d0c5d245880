// sda_append.cuh -- arguments and launcher of the paged append.
#pragma once

#include <algorithm>

#include "sda_chunk.cuh"

namespace sda {

struct AppendParams {
  const uint16_t* q;          // [T, H, D] bf16 (g.H = 0: none)
  const uint16_t* kv;         // [T, D] bf16
  const uint16_t* q_w;        // [D] bf16 norm weights, or null
  const uint16_t* kv_w;
  const float* cos_cache;     // [max_pos, R / 2]
  const float* sin_cache;
  ChunkGeom g;                // (window, first and the division by H are not used)
  int R, max_pos;
  float eps, inv_d;           // inv_d = 1 / D, 0 where that is not exact
  uint16_t* q_out;            // [T, H, D] bf16 (may be q itself)
  uint16_t* pool;             // [total_pages, D] bf16, or null
  uint8_t* codes;             // [total_pages, D] E4M3, or null
  float* scale;               // a scale for each block, with codes
  int32_t* status;
  bool one_status;            // append_one_status()
  int code_ctas, code_tokens; // CTAs that write codes, and their tokens
  uint32_t k_mul;             // n / k_per_block = n k_mul >> k_shift
  int k_shift;
};
bool append_one_status(const AppendParams& p);
cudaError_t launch_append(AppendParams p, int num_sms, cudaStream_t st);

}  // namespace sda
