// sda_evict.cuh -- arguments of the slot eviction (sda_evict.cu).
#pragma once

#include "sda_internal.cuh"

namespace sda {

// Most columns of a table: the kernels step over them by up to 1024, counted in 32 bits
// (a step past the last of 2^31 - 1 would have wrapped round to negative positions).
constexpr int64_t kMaxEvictLen = 0x7fffffff - 2047;

struct EvictArgs {
  const float* scores;   // [B, S]
  const int32_t* slots;  // [B, S]
  int64_t S;
  const int32_t* kv_len;  // [B]
  int B, budget, first, recent;
  float* out_scores;   // [B, out_S]; may be scores itself (out_S == S)
  int32_t* out_slots;  // [B, out_S]; may be slots itself
  int64_t out_S;
  int32_t* out_len;  // [B]; may be kv_len itself
  int32_t* freed;    // [freed_capacity], at least B * max(S - budget, 0)
  int64_t freed_capacity;
  int32_t* freed_indptr;  // [B + 1]
  int32_t* status;
};

cudaError_t evict_prepare();  // one-time kernel attributes on the current device
cudaError_t launch_evict(const EvictArgs& a, cudaStream_t st);

}  // namespace sda
