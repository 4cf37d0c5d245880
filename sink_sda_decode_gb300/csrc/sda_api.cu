// sda_api.cu -- the extern "C" entry points of libsda (declared in
// include/sda.h): host-side argument checks, kernel-variant choice, the
// workspace layout, and the launches.  Nothing here allocates, synchronises
// or reads device memory from the host.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <mutex>

#include "sda_chunk.cuh"
#include "sda_copy.cuh"
#include "sda_append.cuh"
#include "sda_chunk_fp8.cuh"
#include "sda_evict.cuh"
#include "sda_internal.cuh"
#include "sda_scatter.cuh"

namespace sda {

namespace {

thread_local char g_last_error[256] = "";
// sda_debug_wait_fault: pipeline-wait bound (0 = the default 2 s) and the
// withheld-arrive switch, read by every tensor-core kernel launch.
std::atomic<unsigned long long> g_wait_timeout_ns{0};
std::atomic<int> g_withhold_arrive{0};
constexpr unsigned long long kDefaultWaitTimeoutNs = 2000000000ull;
thread_local cudaEvent_t g_ev_before = nullptr;
thread_local cudaEvent_t g_ev_after = nullptr;

constexpr int kMaxDevices = 64;

struct DeviceInfo {
  std::once_flag once;
  DeviceCaps caps;
  cudaError_t err = cudaSuccess;
};
DeviceInfo g_dev[kMaxDevices];

}  // namespace

void note_cuda_error(cudaError_t e, const char* where) {
  std::snprintf(g_last_error, sizeof g_last_error, "%s: %s (%s)", where, cudaGetErrorName(e),
                cudaGetErrorString(e));
}

// SM count of the current device, queried once per device; also sets the
// tensor-core kernels' shared-memory attributes on that device.
cudaError_t device_caps(DeviceCaps* caps) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  DeviceInfo& d = g_dev[dev];
  std::call_once(d.once, [&]() {
    d.err = cudaDeviceGetAttribute(&d.caps.num_sms, cudaDevAttrMultiProcessorCount, dev);
    for (int nh : {16, 32, 64})
      if (d.err == cudaSuccess) d.err = umma_prepare(nh);
  });
  *caps = d.caps;
  return d.err;
}

namespace {

// device_caps(), and the kernel attributes of one of the paged-cache operators, set at
// that operator's first call on a device: setting them loads the kernels, which is not
// decode's to wait for (its first call took 3.1 ms in place of 0.7 with all of them).
enum PagedOp : int { kOpAttention, kOpMass, kOpEvict, kOpAttentionFp8, kPagedOps };
struct Prepared {
  std::once_flag once;
  cudaError_t err = cudaSuccess;
};
Prepared g_paged[kMaxDevices][kPagedOps];

cudaError_t paged_caps(PagedOp op, DeviceCaps* caps) {
  cudaError_t e = device_caps(caps);
  int dev = 0;
  if (e == cudaSuccess) e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  Prepared& p = g_paged[dev][op];
  std::call_once(p.once, [&]() {
    p.err = op == kOpAttention      ? chunk_prepare()
            : op == kOpMass         ? mass_prepare()
            : op == kOpAttentionFp8 ? chunk_fp8_prepare()
                                    : evict_prepare();
  });
  return p.err;
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Optional A/B switch for tests: SDA_FORCE_VARIANT=simt|umma forces a
// decode kernel (umma only where the shape allows it).
int forced_variant() {
  const char* v = std::getenv("SDA_FORCE_VARIANT");
  if (!v) return -1;
  if (std::strcmp(v, "simt") == 0) return kSimt;
  if (std::strcmp(v, "umma") == 0) return kUmma;
  return -1;
}

}  // namespace

WaitFault current_wait_fault() {
  const unsigned long long t = g_wait_timeout_ns.load();
  return WaitFault{g_withhold_arrive.load(), t ? t : kDefaultWaitTimeoutNs};
}

bool shape_supported(int H, int D) {
  return (D == 64 || D == 128 || D == 256 || D == 512) && H >= 1 && H <= 256;
}

bool tc_shape_supported(int H, int D) {
  return D == 512 && (H == 16 || H == 32 || (H % 64 == 0 && H <= 256));
}

bool choose_plan(int H, int D, const DeviceCaps& caps, LaunchPlan* lp) {
  if (!shape_supported(H, D)) return false;
  lp->num_sms = caps.num_sms;
  const bool tc_shape = tc_shape_supported(H, D);
  const int nh = H < 64 ? H : 64;
  const int forced = forced_variant();
  Variant v = tc_shape ? kUmma : kSimt;
  if (forced == kSimt || (forced == kUmma && tc_shape)) v = static_cast<Variant>(forced);
  lp->variant = v;
  if (v == kUmma) {
    lp->nh = nh;
    lp->hg = H / lp->nh;
    lp->grid = caps.num_sms;  // one CTA per SM (about 200 KB of shared memory each)
    lp->threads = 896;
    lp->smem = umma_smem_bytes(lp->nh);
    lp->tile = kTileSlots;
  } else {
    lp->nh = H;
    lp->hg = 1;
    lp->grid = caps.num_sms * 4;
    lp->threads = 256;
    lp->smem = 0;
    lp->tile = kTileSlots;
  }
  if (lp->grid > kMaxPlanGrid) lp->grid = kMaxPlanGrid;
  return true;
}

WsLayout workspace_layout(int N, int H, int D, int64_t total_indices, const LaunchPlan& lp) {
  WsLayout L;
  // Partial rows: fewer than 2 * grid / hg (each interior range boundary
  // cuts one token) and no more than one per tile (T <= total_indices).
  int64_t p1 = 2 * ((int64_t)(lp.grid + lp.hg - 1) / lp.hg) + 2;
  int64_t p2 = 2 * ((total_indices + lp.tile - 1) / lp.tile) + 2;
  int64_t p_max = p1 < p2 ? p1 : p2;
  int64_t s_max = p_max / 2 + 1;
  if (s_max > N) s_max = N;
  L.p_max = (int)p_max;
  L.s_max = (int)s_max;
  L.u_max = (int)((int64_t)lp.hg * ((int64_t)N + p_max));
  size_t off = sizeof(WsHeader);
  L.units_off = off;
  off = align_up(off + (size_t)L.u_max * 16, 256);
  L.cta_off = off;
  off = align_up(off + (size_t)(lp.grid + 1) * 4, 256);
  L.ctok_off = off;
  off = align_up(off + (size_t)(N > 0 ? N : 1) * 4, 256);
  L.ctp_off = off;
  off = align_up(off + (size_t)(N + 1) * 4, 256);
  L.split_off = off;
  off = align_up(off + (size_t)(s_max > 0 ? s_max : 1) * 16, 256);
  L.ml_off = off;
  off = align_up(off + (size_t)p_max * H * 8, 256);
  L.o_off = off;
  off = align_up(off + (size_t)p_max * H * D * 4, 256);
  L.total = off;
  return L;
}

}  // namespace sda

using namespace sda;

extern "C" {

const char* sda_strerror(sda_status status) {
  switch (status) {
    case SDA_OK: return "SDA_OK";
    case SDA_ERR_INVALID_ARG: return "SDA_ERR_INVALID_ARG: invalid argument";
    case SDA_ERR_UNSUPPORTED: return "SDA_ERR_UNSUPPORTED: unsupported (H, D)";
    case SDA_ERR_CUDA: return "SDA_ERR_CUDA: a CUDA call failed";
    case SDA_ERR_WORKSPACE: return "SDA_ERR_WORKSPACE: workspace too small or misaligned";
    default: return "SDA: unknown status";
  }
}

const char* sda_last_cuda_error(void) { return g_last_error; }

int sda_abi_version(void) { return 1; }

sda_status sda_decode_workspace_size(int N, int H, int D, int64_t total_indices, size_t* bytes) {
  if (!bytes || N < 0 || total_indices < 0) return SDA_ERR_INVALID_ARG;
  if (!shape_supported(H, D)) return SDA_ERR_UNSUPPORTED;
  DeviceCaps caps;
  cudaError_t e = device_caps(&caps);
  if (e != cudaSuccess) {
    note_cuda_error(e, "sda_decode_workspace_size");
    return SDA_ERR_CUDA;
  }
  LaunchPlan lp;
  if (!choose_plan(H, D, caps, &lp)) return SDA_ERR_UNSUPPORTED;
  *bytes = workspace_layout(N, H, D, total_indices, lp).total;
  return SDA_OK;
}

sda_status sda_decode(const void* q, const void* unified_kv, int64_t total_pages,
                      const int32_t* kv_indices, int64_t total_indices,
                      const int32_t* kv_indptr, const float* attn_sink, float softmax_scale,
                      int N, int H, int D, void* out, void* workspace, size_t workspace_bytes,
                      void* stream) {
  if (N < 0 || total_indices < 0 || total_indices > 0x7fffffffll) return SDA_ERR_INVALID_ARG;
  if (total_pages <= 0 || total_pages > 0x7fffffffll) return SDA_ERR_INVALID_ARG;
  if (!shape_supported(H, D)) return SDA_ERR_UNSUPPORTED;
  if (N == 0) return SDA_OK;
  if (!q || !unified_kv || !kv_indptr || !attn_sink || !out || !workspace) return SDA_ERR_INVALID_ARG;
  if (total_indices > 0 && !kv_indices) return SDA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(unified_kv, 16) || !aligned(out, 16) || !aligned(kv_indptr, 4) ||
      !aligned(attn_sink, 4) || (kv_indices && !aligned(kv_indices, 4)))
    return SDA_ERR_INVALID_ARG;
  if (!aligned(workspace, 256)) return SDA_ERR_WORKSPACE;
  DeviceCaps caps;
  cudaError_t e = device_caps(&caps);
  if (e != cudaSuccess) {
    note_cuda_error(e, "sda_decode");
    return SDA_ERR_CUDA;
  }
  LaunchPlan lp;
  choose_plan(H, D, caps, &lp);
  const WsLayout L = workspace_layout(N, H, D, total_indices, lp);
  if (workspace_bytes < L.total) return SDA_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);

  e = launch_plan(kv_indptr, N, total_indices, lp, workspace, L, st);
  if (e == cudaSuccess && g_ev_before && g_ev_after) e = cudaEventRecord(g_ev_before, st);
  if (e == cudaSuccess) {
    if (lp.variant == kUmma)
      e = launch_decode_umma(q, unified_kv, nullptr, total_pages, kv_indices, attn_sink,
                             softmax_scale, N, H, D, out, workspace, L, lp, st);
    else
      e = launch_decode_simt(q, unified_kv, kv_indices, attn_sink, softmax_scale, N, H, D, out,
                             workspace, L, lp, st);
  }
  if (e == cudaSuccess && g_ev_before && g_ev_after) e = cudaEventRecord(g_ev_after, st);
  if (e == cudaSuccess) e = launch_combine(attn_sink, N, H, D, out, workspace, L, caps.num_sms, st);
  if (e != cudaSuccess) {
    note_cuda_error(e, "sda_decode");
    return SDA_ERR_CUDA;
  }
  return SDA_OK;
}

// The FP8-pool entry points run the one-CTA tensor-core kernel only.
static bool fp8_plan(int H, int D, const DeviceCaps& caps, LaunchPlan* lp) {
  if (!tc_shape_supported(H, D) || !choose_plan(H, D, caps, lp)) return false;
  if (lp->variant != kUmma) {  // a forced variant does not apply to the FP8 pool
    lp->variant = kUmma;
    lp->nh = H < 64 ? H : 64;
    lp->hg = H / lp->nh;
    lp->grid = caps.num_sms;
    lp->threads = 896;
    lp->smem = umma_smem_bytes(lp->nh);
    lp->tile = kTileSlots;
  }
  return true;
}

sda_status sda_decode_fp8_workspace_size(int N, int H, int D, int64_t total_indices, size_t* bytes) {
  if (!bytes || N < 0 || total_indices < 0) return SDA_ERR_INVALID_ARG;
  if (!tc_shape_supported(H, D)) return SDA_ERR_UNSUPPORTED;
  DeviceCaps caps;
  cudaError_t e = device_caps(&caps);
  if (e != cudaSuccess) {
    note_cuda_error(e, "sda_decode_fp8_workspace_size");
    return SDA_ERR_CUDA;
  }
  LaunchPlan lp;
  if (!fp8_plan(H, D, caps, &lp)) return SDA_ERR_UNSUPPORTED;
  *bytes = workspace_layout(N, H, D, total_indices, lp).total;
  return SDA_OK;
}

sda_status sda_decode_fp8(const void* q, const void* kv_fp8, const float* kv_scale,
                          int64_t total_pages, const int32_t* kv_indices, int64_t total_indices,
                          const int32_t* kv_indptr, const float* attn_sink, float softmax_scale,
                          int N, int H, int D, void* out, void* workspace, size_t workspace_bytes,
                          void* stream) {
  if (N < 0 || total_indices < 0 || total_indices > 0x7fffffffll) return SDA_ERR_INVALID_ARG;
  if (total_pages <= 0 || total_pages > 0x7fffffffll) return SDA_ERR_INVALID_ARG;
  if (!tc_shape_supported(H, D)) return SDA_ERR_UNSUPPORTED;
  if (N == 0) return SDA_OK;
  if (!q || !kv_fp8 || !kv_scale || !kv_indptr || !attn_sink || !out || !workspace)
    return SDA_ERR_INVALID_ARG;
  if (total_indices > 0 && !kv_indices) return SDA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(kv_fp8, 16) || !aligned(out, 16) || !aligned(kv_scale, 4) ||
      !aligned(kv_indptr, 4) || !aligned(attn_sink, 4) || (kv_indices && !aligned(kv_indices, 4)))
    return SDA_ERR_INVALID_ARG;
  if (!aligned(workspace, 256)) return SDA_ERR_WORKSPACE;
  DeviceCaps caps;
  cudaError_t e = device_caps(&caps);
  if (e != cudaSuccess) {
    note_cuda_error(e, "sda_decode_fp8");
    return SDA_ERR_CUDA;
  }
  LaunchPlan lp;
  fp8_plan(H, D, caps, &lp);
  const WsLayout L = workspace_layout(N, H, D, total_indices, lp);
  if (workspace_bytes < L.total) return SDA_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  e = launch_plan(kv_indptr, N, total_indices, lp, workspace, L, st);
  if (e == cudaSuccess && g_ev_before && g_ev_after) e = cudaEventRecord(g_ev_before, st);
  if (e == cudaSuccess)
    e = launch_decode_umma(q, kv_fp8, kv_scale, total_pages, kv_indices, attn_sink, softmax_scale,
                           N, H, D, out, workspace, L, lp, st);
  if (e == cudaSuccess && g_ev_before && g_ev_after) e = cudaEventRecord(g_ev_after, st);
  if (e == cudaSuccess) e = launch_combine(attn_sink, N, H, D, out, workspace, L, caps.num_sms, st);
  if (e != cudaSuccess) {
    note_cuda_error(e, "sda_decode_fp8");
    return SDA_ERR_CUDA;
  }
  return SDA_OK;
}

// The scalar and pool-argument checks of sda_build_decode(_host) that need
// no workspace-derived pointer; the host-buffer entry point runs them before
// it enqueues its input gather, so that an invalid call enqueues nothing.
static sda_status build_decode_scalars_ok(int N, int win, int k_per_block, int64_t swa_pages,
                                          int64_t total_pages, int64_t capacity,
                                          int64_t comp_total, const void* unified_kv,
                                          const float* kv_scale, const float* attn_sink, int H,
                                          int D) {
  if (N < 0 || win <= 0 || k_per_block <= 0 || swa_pages < 0 || total_pages <= 0 ||
      total_pages > 0x7fffffffll || swa_pages > total_pages || capacity < 0 ||
      capacity > 0x7fffffffll || comp_total < 0 || comp_total > 0x7fffffffll)
    return SDA_ERR_INVALID_ARG;
  const bool fp8 = kv_scale != nullptr;
  if (fp8 ? !tc_shape_supported(H, D) : !shape_supported(H, D)) return SDA_ERR_UNSUPPORTED;
  if (N > 0 && (!unified_kv || !attn_sink || !aligned(unified_kv, 16) || !aligned(attn_sink, 4) ||
                (fp8 && !aligned(kv_scale, 4))))
    return SDA_ERR_INVALID_ARG;
  return SDA_OK;
}

static sda_status build_decode_impl(const int32_t* state_slot, const int32_t* swa_len,
                                    const int32_t* swa_head, const int32_t* comp_indptr,
                                    const int32_t* comp_block, const int32_t* comp_slot,
                                    int64_t comp_total, int win, int k_per_block,
                                    int64_t swa_pages, int32_t* kv_indices, int64_t capacity,
                                    int32_t* kv_indptr, int32_t* status, const void* q,
                                    const void* unified_kv, const float* kv_scale,
                                    int64_t total_pages, const float* attn_sink,
                                    float softmax_scale, int N, int H, int D, void* out,
                                    void* workspace, size_t workspace_bytes, void* stream,
                                    const char* who) {
  // the builder's checks (sda_build_indices)
  if (N < 0 || win <= 0 || k_per_block <= 0 || swa_pages < 0 || total_pages <= 0 ||
      total_pages > 0x7fffffffll || swa_pages > total_pages || capacity < 0 ||
      capacity > 0x7fffffffll || comp_total < 0 || comp_total > 0x7fffffffll)
    return SDA_ERR_INVALID_ARG;
  if (!kv_indptr || !status) return SDA_ERR_INVALID_ARG;
  if (N > 0 && (!state_slot || !swa_len || !swa_head || !comp_indptr)) return SDA_ERR_INVALID_ARG;
  if (comp_total > 0 && (!comp_block || !comp_slot)) return SDA_ERR_INVALID_ARG;
  if (capacity > 0 && !kv_indices) return SDA_ERR_INVALID_ARG;
  // the decode's checks (sda_decode / sda_decode_fp8)
  const bool fp8 = kv_scale != nullptr;
  if (fp8 ? !tc_shape_supported(H, D) : !shape_supported(H, D)) return SDA_ERR_UNSUPPORTED;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (N == 0) {  // the builder still writes kv_indptr[0] and the status word
    const cudaError_t e = launch_build_indices(state_slot, swa_len, swa_head, comp_indptr,
                                               comp_block, comp_slot, comp_total, N, win,
                                               k_per_block, swa_pages, total_pages, kv_indices,
                                               capacity, kv_indptr, status, st);
    if (e != cudaSuccess) {
      note_cuda_error(e, who);
      return SDA_ERR_CUDA;
    }
    return SDA_OK;
  }
  if (!q || !unified_kv || !attn_sink || !out || !workspace) return SDA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(unified_kv, 16) || !aligned(out, 16) || !aligned(kv_indptr, 4) ||
      !aligned(attn_sink, 4) || (kv_indices && !aligned(kv_indices, 4)) ||
      (fp8 && !aligned(kv_scale, 4)))
    return SDA_ERR_INVALID_ARG;
  if (!aligned(workspace, 256)) return SDA_ERR_WORKSPACE;
  DeviceCaps caps;
  cudaError_t e = device_caps(&caps);
  if (e != cudaSuccess) {
    note_cuda_error(e, who);
    return SDA_ERR_CUDA;
  }
  LaunchPlan lp;
  if (fp8) fp8_plan(H, D, caps, &lp);
  else choose_plan(H, D, caps, &lp);
  const WsLayout L = workspace_layout(N, H, D, capacity, lp);
  if (workspace_bytes < L.total) return SDA_ERR_WORKSPACE;
  const EntryCheck ec = entry_check_layout(state_slot, comp_indptr, comp_block, comp_slot,
                                           comp_total, N, k_per_block, swa_pages, total_pages,
                                           capacity, kv_indices, status, caps.num_sms);
  e = launch_build_len(swa_len, swa_head, N, win, kv_indptr, ec, st);
  if (e == cudaSuccess) e = launch_build_scan(N, capacity, kv_indptr, status, ec, st);
  if (e == cudaSuccess) {
    const ScatterArgs sa{state_slot, swa_len, swa_head, comp_indptr, comp_block, comp_slot, N, win,
                         k_per_block, swa_pages, kv_indptr, kv_indices};
    e = launch_scatter_plan(sa, capacity, lp, workspace, L, caps.num_sms, st);
  }
  if (e == cudaSuccess && g_ev_before && g_ev_after) e = cudaEventRecord(g_ev_before, st);
  if (e == cudaSuccess) {
    if (fp8)
      e = launch_decode_umma(q, unified_kv, kv_scale, total_pages, kv_indices, attn_sink,
                             softmax_scale, N, H, D, out, workspace, L, lp, st);
    else if (lp.variant == kUmma)
      e = launch_decode_umma(q, unified_kv, nullptr, total_pages, kv_indices, attn_sink,
                             softmax_scale, N, H, D, out, workspace, L, lp, st);
    else
      e = launch_decode_simt(q, unified_kv, kv_indices, attn_sink, softmax_scale, N, H, D, out,
                             workspace, L, lp, st);
  }
  if (e == cudaSuccess && g_ev_before && g_ev_after) e = cudaEventRecord(g_ev_after, st);
  if (e == cudaSuccess) e = launch_combine(attn_sink, N, H, D, out, workspace, L, caps.num_sms, st);
  if (e != cudaSuccess) {
    note_cuda_error(e, who);
    return SDA_ERR_CUDA;
  }
  return SDA_OK;
}

sda_status sda_build_decode(const int32_t* state_slot, const int32_t* swa_len,
                            const int32_t* swa_head, const int32_t* comp_indptr,
                            const int32_t* comp_block, const int32_t* comp_slot,
                            int64_t comp_total, int win, int k_per_block, int64_t swa_pages,
                            int32_t* kv_indices, int64_t capacity, int32_t* kv_indptr,
                            int32_t* status, const void* q, const void* unified_kv,
                            const float* kv_scale, int64_t total_pages, const float* attn_sink,
                            float softmax_scale, int N, int H, int D, void* out, void* workspace,
                            size_t workspace_bytes, void* stream) {
  return build_decode_impl(state_slot, swa_len, swa_head, comp_indptr, comp_block, comp_slot,
                           comp_total, win, k_per_block, swa_pages, kv_indices, capacity,
                           kv_indptr, status, q, unified_kv, kv_scale, total_pages, attn_sink,
                           softmax_scale, N, H, D, out, workspace, workspace_bytes, stream,
                           "sda_build_decode");
}

// Layout of sda_build_decode_host's device workspace: the staged inputs, the
// builder's outputs, the staged output, then sda_build_decode's workspace.
struct HostWs {
  size_t q, ss, sl, sh, cptr, cb, cs, idx, iptr, st, out, dec, total;
};

static HostWs host_ws_layout(int N, int H, int D, int64_t comp_total, int64_t capacity,
                             size_t dec_bytes) {
  HostWs w;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align_up(off + (bytes > 0 ? bytes : 1), 256);
    return at;
  };
  const size_t qb = (size_t)N * H * D * 2;
  w.q = take(qb);
  w.ss = take((size_t)N * 4);
  w.sl = take((size_t)N * 4);
  w.sh = take((size_t)N * 4);
  w.cptr = take((size_t)(N + 1) * 4);
  w.cb = take((size_t)comp_total * 4);
  w.cs = take((size_t)comp_total * 4);
  w.idx = take((size_t)capacity * 4);
  w.iptr = take((size_t)(N + 1) * 4);
  w.st = take(4);
  w.out = take(qb);
  w.dec = take(dec_bytes);
  w.total = off;
  return w;
}

// Device view of page-locked host memory (NULL if `p` is not page-locked host memory).
static const void* host_view(const void* p) {
  if (!p) return nullptr;
  cudaPointerAttributes a;
  if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
    cudaGetLastError();
    return nullptr;
  }
  return a.type == cudaMemoryTypeHost ? a.devicePointer : nullptr;
}

static sda_status build_decode_ws(int N, int H, int D, int64_t capacity, bool fp8, size_t* bytes) {
  DeviceCaps caps;
  const cudaError_t e = device_caps(&caps);
  if (e != cudaSuccess) {
    note_cuda_error(e, "sda_build_decode_host_workspace_size");
    return SDA_ERR_CUDA;
  }
  LaunchPlan lp;
  if (fp8) fp8_plan(H, D, caps, &lp);
  else choose_plan(H, D, caps, &lp);
  *bytes = workspace_layout(N, H, D, capacity, lp).total;
  return SDA_OK;
}

// ---------------------------------------------------------------- large host batches
// A batch whose q (and out) is at least kPipelineBytes moves through the
// host link in token chunks so that the link's two directions and the SMs
// work at once: two streams of this library carry copy-engine transfers (the
// descriptors and each chunk's q in; each chunk's out back as soon as its
// decode is done) while the caller's stream builds the whole batch's lists
// once and decodes chunk after chunk (the decode takes absolute kv_indptr
// offsets, so a chunk decodes from a slice of the batch's lists).  The
// chunk boundaries depend on N only, never on the contents of the host
// arrays, so a captured graph stays valid when the caller refills them.
constexpr int64_t kPipelineBytes = 8ll << 20;
constexpr int kMaxChunks = 8;

struct PipeRes {
  cudaStream_t cin = nullptr, cout = nullptr;
  cudaEvent_t fork = nullptr, desc = nullptr, built = nullptr, done = nullptr;
  cudaEvent_t q_in[kMaxChunks] = {}, dec_done[kMaxChunks] = {};
  bool ok = false;
};

// Streams and events of the current device, created on its first large
// call (which should therefore come before any stream capture); calls that
// enqueue concurrently from several host threads are serialised.
static std::mutex g_pipe_mu;
static PipeRes g_pipe[64];

static cudaError_t pipe_resources(PipeRes** out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  PipeRes& r = g_pipe[dev];
  if (!r.ok) {
    // all or nothing: a failure destroys whatever this attempt created
    PipeRes n;
    const unsigned fl = cudaEventDisableTiming;
    cudaEvent_t* evs[4 + 2 * kMaxChunks] = {&n.fork, &n.desc, &n.built, &n.done};
    for (int c = 0; c < kMaxChunks; ++c) {
      evs[4 + 2 * c] = &n.q_in[c];
      evs[5 + 2 * c] = &n.dec_done[c];
    }
    e = cudaStreamCreateWithFlags(&n.cin, cudaStreamNonBlocking);
    if (e == cudaSuccess) e = cudaStreamCreateWithFlags(&n.cout, cudaStreamNonBlocking);
    for (cudaEvent_t* p : evs)
      if (e == cudaSuccess) e = cudaEventCreateWithFlags(p, fl);
    if (e != cudaSuccess) {
      for (cudaEvent_t* p : evs)
        if (*p) cudaEventDestroy(*p);
      if (n.cin) cudaStreamDestroy(n.cin);
      if (n.cout) cudaStreamDestroy(n.cout);
      return e;
    }
    n.ok = true;
    r = n;
  }
  *out = &r;
  return cudaSuccess;
}

static sda_status build_decode_host_pipelined(
    const int32_t* state_slot, const int32_t* swa_len, const int32_t* swa_head,
    const int32_t* comp_indptr, const int32_t* comp_block, const int32_t* comp_slot,
    int64_t comp_total, int win, int k_per_block, int64_t swa_pages, int64_t capacity,
    const void* q, const void* unified_kv, const float* kv_scale, int64_t total_pages,
    const float* attn_sink, float softmax_scale, int N, int H, int D, void* out, int32_t* status,
    char* base, const HostWs& w, cudaStream_t st) {
  const char* who = "sda_build_decode_host";
  const bool fp8 = kv_scale != nullptr;
  DeviceCaps caps;
  cudaError_t e = device_caps(&caps);
  if (e != cudaSuccess) {
    note_cuda_error(e, who);
    return SDA_ERR_CUDA;
  }
  LaunchPlan lp;
  if (fp8) fp8_plan(H, D, caps, &lp);
  else choose_plan(H, D, caps, &lp);
  std::lock_guard<std::mutex> lock(g_pipe_mu);
  PipeRes* r = nullptr;
  e = pipe_resources(&r);
  const int64_t row_bytes = (int64_t)H * D * 2;  // q / out bytes per token
  const int64_t q_bytes = (int64_t)N * row_bytes;
  int chunks = (int)(q_bytes / kPipelineBytes);
  chunks = chunks < 2 ? 2 : (chunks > kMaxChunks ? kMaxChunks : chunks);
  if (chunks > N) chunks = N;
  const int per = (N + chunks - 1) / chunks;
  auto H2D = [&](void* dst, const void* src, size_t bytes) {
    return bytes ? cudaMemcpyAsync(dst, src, bytes, cudaMemcpyHostToDevice, r->cin) : cudaSuccess;
  };
  // fork: the copy streams start after everything already on the caller's stream
  if (e == cudaSuccess) e = cudaEventRecord(r->fork, st);
  if (e == cudaSuccess) e = cudaStreamWaitEvent(r->cin, r->fork, 0);
  if (e == cudaSuccess) e = cudaStreamWaitEvent(r->cout, r->fork, 0);
  // descriptors, then the q chunks, on the inbound stream
  if (e == cudaSuccess) e = H2D(base + w.ss, state_slot, (size_t)N * 4);
  if (e == cudaSuccess) e = H2D(base + w.sl, swa_len, (size_t)N * 4);
  if (e == cudaSuccess) e = H2D(base + w.sh, swa_head, (size_t)N * 4);
  if (e == cudaSuccess) e = H2D(base + w.cptr, comp_indptr, (size_t)(N + 1) * 4);
  if (e == cudaSuccess) e = H2D(base + w.cb, comp_block, (size_t)comp_total * 4);
  if (e == cudaSuccess) e = H2D(base + w.cs, comp_slot, (size_t)comp_total * 4);
  if (e == cudaSuccess) e = cudaEventRecord(r->desc, r->cin);
  for (int c = 0; c < chunks && e == cudaSuccess; ++c) {
    const int t0 = c * per, nc = (t0 + per <= N ? per : N - t0);
    if (nc <= 0) break;
    e = H2D(base + w.q + (size_t)t0 * row_bytes, static_cast<const char*>(q) + (size_t)t0 * row_bytes,
            (size_t)nc * row_bytes);
    if (e == cudaSuccess) e = cudaEventRecord(r->q_in[c], r->cin);
  }
  // the whole batch's lists and status on the caller's stream
  int32_t* idx = reinterpret_cast<int32_t*>(base + w.idx);
  int32_t* iptr = reinterpret_cast<int32_t*>(base + w.iptr);
  int32_t* dst_st = reinterpret_cast<int32_t*>(base + w.st);
  if (e == cudaSuccess) e = cudaStreamWaitEvent(st, r->desc, 0);
  if (e == cudaSuccess)
    e = launch_build_indices(reinterpret_cast<const int32_t*>(base + w.ss),
                             reinterpret_cast<const int32_t*>(base + w.sl),
                             reinterpret_cast<const int32_t*>(base + w.sh),
                             reinterpret_cast<const int32_t*>(base + w.cptr),
                             reinterpret_cast<const int32_t*>(base + w.cb),
                             reinterpret_cast<const int32_t*>(base + w.cs), comp_total, N, win,
                             k_per_block, swa_pages, total_pages, idx, capacity, iptr, dst_st, st);
  if (e == cudaSuccess) e = cudaEventRecord(r->built, st);
  // the status word goes back as soon as the build is done
  if (e == cudaSuccess) e = cudaStreamWaitEvent(r->cout, r->built, 0);
  if (e == cudaSuccess) e = cudaMemcpyAsync(status, dst_st, 4, cudaMemcpyDeviceToHost, r->cout);
  // decode chunk after chunk; each chunk's out goes back on the outbound stream
  void* dec = base + w.dec;
  for (int c = 0; c < chunks && e == cudaSuccess; ++c) {
    const int t0 = c * per, nc = (t0 + per <= N ? per : N - t0);
    if (nc <= 0) break;
    const WsLayout L = workspace_layout(nc, H, D, capacity, lp);
    const char* qc = base + w.q + (size_t)t0 * row_bytes;
    char* oc = base + w.out + (size_t)t0 * row_bytes;
    e = cudaStreamWaitEvent(st, r->q_in[c], 0);
    if (e == cudaSuccess) e = launch_plan(iptr + t0, nc, capacity, lp, dec, L, st);
    if (e == cudaSuccess) {
      if (fp8 || lp.variant == kUmma)
        e = launch_decode_umma(qc, unified_kv, kv_scale, total_pages, idx, attn_sink, softmax_scale,
                               nc, H, D, oc, dec, L, lp, st);
      else
        e = launch_decode_simt(qc, unified_kv, idx, attn_sink, softmax_scale, nc, H, D, oc, dec,
                               L, lp, st);
    }
    if (e == cudaSuccess) e = launch_combine(attn_sink, nc, H, D, oc, dec, L, caps.num_sms, st);
    if (e == cudaSuccess) e = cudaEventRecord(r->dec_done[c], st);
    if (e == cudaSuccess) e = cudaStreamWaitEvent(r->cout, r->dec_done[c], 0);
    if (e == cudaSuccess)
      e = cudaMemcpyAsync(static_cast<char*>(out) + (size_t)t0 * row_bytes, oc, (size_t)nc * row_bytes,
                          cudaMemcpyDeviceToHost, r->cout);
  }
  // join: the caller's stream continues after every copy of this call
  if (e == cudaSuccess) e = cudaEventRecord(r->done, r->cout);
  if (e == cudaSuccess) e = cudaStreamWaitEvent(st, r->done, 0);
  if (e == cudaSuccess) e = cudaEventRecord(r->fork, r->cin);  // the inbound stream joins too
  if (e == cudaSuccess) e = cudaStreamWaitEvent(st, r->fork, 0);
  if (e != cudaSuccess) {
    note_cuda_error(e, who);
    return SDA_ERR_CUDA;
  }
  return SDA_OK;
}

sda_status sda_build_decode_host_workspace_size(int N, int H, int D, int64_t comp_total,
                                                int64_t capacity, int fp8, size_t* bytes) {
  if (!bytes || N < 0 || comp_total < 0 || capacity < 0) return SDA_ERR_INVALID_ARG;
  if (fp8 ? !tc_shape_supported(H, D) : !shape_supported(H, D)) return SDA_ERR_UNSUPPORTED;
  size_t dec = 0;
  const sda_status r = build_decode_ws(N, H, D, capacity, fp8 != 0, &dec);
  if (r != SDA_OK) return r;
  *bytes = host_ws_layout(N, H, D, comp_total, capacity, dec).total;
  if ((int64_t)N * H * D * 2 >= kPipelineBytes && N >= 2) {
    // a large batch takes the chunked route: create this device's copy
    // streams now, so that the first call can already be captured
    std::lock_guard<std::mutex> lock(g_pipe_mu);
    PipeRes* res = nullptr;
    const cudaError_t e = pipe_resources(&res);
    if (e != cudaSuccess) {
      note_cuda_error(e, "sda_build_decode_host_workspace_size");
      return SDA_ERR_CUDA;
    }
  }
  return SDA_OK;
}

sda_status sda_build_decode_host(const int32_t* state_slot, const int32_t* swa_len,
                                 const int32_t* swa_head, const int32_t* comp_indptr,
                                 const int32_t* comp_block, const int32_t* comp_slot,
                                 int64_t comp_total, int win, int k_per_block, int64_t swa_pages,
                                 int64_t capacity, const void* q, const void* unified_kv,
                                 const float* kv_scale, int64_t total_pages,
                                 const float* attn_sink, float softmax_scale, int N, int H, int D,
                                 void* out, int32_t* status, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  if (!status || !workspace) return SDA_ERR_INVALID_ARG;
  // everything checkable on the host is checked before the input gather is enqueued
  sda_status r0 = build_decode_scalars_ok(N, win, k_per_block, swa_pages, total_pages, capacity,
                                          comp_total, unified_kv, kv_scale, attn_sink, H, D);
  if (r0 != SDA_OK) return r0;
  const bool fp8 = kv_scale != nullptr;
  if (!aligned(workspace, 256)) return SDA_ERR_WORKSPACE;
  // every host array must be page-locked; q and out 16-byte aligned
  const void* d_st = host_view(status);
  const void* d_ss = N > 0 ? host_view(state_slot) : nullptr;
  const void* d_sl = N > 0 ? host_view(swa_len) : nullptr;
  const void* d_sh = N > 0 ? host_view(swa_head) : nullptr;
  const void* d_cp = host_view(comp_indptr);
  const void* d_cb = comp_total > 0 ? host_view(comp_block) : nullptr;
  const void* d_cs = comp_total > 0 ? host_view(comp_slot) : nullptr;
  const void* d_q = N > 0 ? host_view(q) : nullptr;
  const void* d_out = N > 0 ? host_view(out) : nullptr;
  if (!d_st || !d_cp || (N > 0 && (!d_ss || !d_sl || !d_sh || !d_q || !d_out)) ||
      (comp_total > 0 && (!d_cb || !d_cs)))
    return SDA_ERR_INVALID_ARG;
  if ((N > 0 && (!aligned(d_q, 16) || !aligned(d_out, 16))) || !aligned(d_st, 4) ||
      !aligned(d_cp, 4) || (N > 0 && (!aligned(d_ss, 4) || !aligned(d_sl, 4) || !aligned(d_sh, 4))) ||
      (comp_total > 0 && (!aligned(d_cb, 4) || !aligned(d_cs, 4))))
    return SDA_ERR_INVALID_ARG;
  size_t dec = 0;
  sda_status r = build_decode_ws(N, H, D, capacity, fp8, &dec);
  if (r != SDA_OK) return r;
  const HostWs w = host_ws_layout(N, H, D, comp_total, capacity, dec);
  if (workspace_bytes < w.total) return SDA_ERR_WORKSPACE;
  char* base = static_cast<char*>(workspace);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if ((int64_t)N * H * D * 2 >= kPipelineBytes && N >= 2)
    return build_decode_host_pipelined(state_slot, swa_len, swa_head, comp_indptr, comp_block,
                                       comp_slot, comp_total, win, k_per_block, swa_pages, capacity,
                                       q, unified_kv, kv_scale, total_pages, attn_sink,
                                       softmax_scale, N, H, D, out, status, base, w, st);
  DeviceCaps caps;
  cudaError_t e = device_caps(&caps);
  const int64_t q_words = (int64_t)N * H * D / 2;
  CopySegments in = {};
  auto add = [](CopySegments& c, const void* src, void* dst, int64_t words) {
    if (words > 0) c.seg[c.n++] = CopySegment{src, dst, words};
  };
  add(in, d_q, base + w.q, q_words);
  add(in, d_ss, base + w.ss, N);
  add(in, d_sl, base + w.sl, N);
  add(in, d_sh, base + w.sh, N);
  add(in, d_cp, base + w.cptr, N + 1);
  add(in, d_cb, base + w.cb, comp_total);
  add(in, d_cs, base + w.cs, comp_total);
  if (e == cudaSuccess) e = launch_gather_copy(in, caps.num_sms, st);
  if (e != cudaSuccess) {
    note_cuda_error(e, "sda_build_decode_host");
    return SDA_ERR_CUDA;
  }
  r = build_decode_impl(reinterpret_cast<const int32_t*>(base + w.ss),
                        reinterpret_cast<const int32_t*>(base + w.sl),
                        reinterpret_cast<const int32_t*>(base + w.sh),
                        reinterpret_cast<const int32_t*>(base + w.cptr),
                        reinterpret_cast<const int32_t*>(base + w.cb),
                        reinterpret_cast<const int32_t*>(base + w.cs), comp_total, win,
                        k_per_block, swa_pages, reinterpret_cast<int32_t*>(base + w.idx), capacity,
                        reinterpret_cast<int32_t*>(base + w.iptr),
                        reinterpret_cast<int32_t*>(base + w.st), base + w.q, unified_kv, kv_scale,
                        total_pages, attn_sink, softmax_scale, N, H, D, base + w.out,
                        base + w.dec, dec > 0 ? dec : 1, stream, "sda_build_decode_host");
  if (r != SDA_OK) return r;
  CopySegments back = {};
  add(back, base + w.out, const_cast<void*>(d_out), q_words);
  add(back, base + w.st, const_cast<void*>(d_st), 1);
  e = launch_gather_copy(back, caps.num_sms, st);
  if (e != cudaSuccess) {
    note_cuda_error(e, "sda_build_decode_host");
    return SDA_ERR_CUDA;
  }
  return SDA_OK;
}

sda_status sda_decode_kernel(int H, int D, int* kernel) {
  if (!kernel) return SDA_ERR_INVALID_ARG;
  if (!shape_supported(H, D)) return SDA_ERR_UNSUPPORTED;
  DeviceCaps caps;
  cudaError_t e = device_caps(&caps);
  if (e != cudaSuccess) {
    note_cuda_error(e, "sda_decode_kernel");
    return SDA_ERR_CUDA;
  }
  LaunchPlan lp;
  choose_plan(H, D, caps, &lp);
  static_assert(SDA_KERNEL_SIMT == kSimt && SDA_KERNEL_ONE_CTA == kUmma, "public kernel codes");
  *kernel = lp.variant;
  return SDA_OK;
}

sda_status sda_debug_wait_fault(int withhold_arrive, uint64_t timeout_ns) {
  if (withhold_arrive != 0 && withhold_arrive != 1) return SDA_ERR_INVALID_ARG;
  g_withhold_arrive.store(withhold_arrive);
  g_wait_timeout_ns.store(timeout_ns);
  return SDA_OK;
}

sda_status sda_set_timing_events(void* before, void* after) {
  if ((before == nullptr) != (after == nullptr)) return SDA_ERR_INVALID_ARG;
  g_ev_before = static_cast<cudaEvent_t>(before);
  g_ev_after = static_cast<cudaEvent_t>(after);
  return SDA_OK;
}

sda_status sda_decode_error_flag(const void* workspace, int32_t* device_flag, void* stream) {
  if (!workspace || !device_flag || !aligned(workspace, 256)) return SDA_ERR_INVALID_ARG;
  const char* src = static_cast<const char*>(workspace) + offsetof(WsHeader, error);
  cudaError_t e = cudaMemcpyAsync(device_flag, src, sizeof(int32_t), cudaMemcpyDeviceToDevice,
                                  static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) {
    note_cuda_error(e, "sda_decode_error_flag");
    return SDA_ERR_CUDA;
  }
  return SDA_OK;
}

sda_status sda_build_indices(const int32_t* state_slot, const int32_t* swa_len,
                             const int32_t* swa_head, const int32_t* comp_indptr,
                             const int32_t* comp_block, const int32_t* comp_slot,
                             int64_t comp_total, int N, int win, int k_per_block,
                             int64_t swa_pages, int64_t total_pages, int32_t* kv_indices,
                             int64_t capacity, int32_t* kv_indptr, int32_t* status,
                             void* stream) {
  if (N < 0 || win <= 0 || k_per_block <= 0 || swa_pages < 0 || total_pages <= 0 ||
      total_pages > 0x7fffffffll || swa_pages > total_pages || capacity < 0 ||
      capacity > 0x7fffffffll || comp_total < 0 || comp_total > 0x7fffffffll)
    return SDA_ERR_INVALID_ARG;
  if (!kv_indptr || !status) return SDA_ERR_INVALID_ARG;
  if (N > 0 && (!state_slot || !swa_len || !swa_head || !comp_indptr)) return SDA_ERR_INVALID_ARG;
  if (comp_total > 0 && (!comp_block || !comp_slot)) return SDA_ERR_INVALID_ARG;
  if (capacity > 0 && !kv_indices) return SDA_ERR_INVALID_ARG;
  cudaError_t e = launch_build_indices(state_slot, swa_len, swa_head, comp_indptr, comp_block,
                                       comp_slot, comp_total, N, win, k_per_block, swa_pages,
                                       total_pages, kv_indices, capacity, kv_indptr, status,
                                       static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) {
    note_cuda_error(e, "sda_build_indices");
    return SDA_ERR_CUDA;
  }
  return SDA_OK;
}

sda_status sda_validate_indices(const int32_t* kv_indices, int64_t total_indices,
                                const int32_t* kv_indptr, int N, int64_t total_pages,
                                int32_t* status, void* stream) {
  if (N < 0 || total_indices < 0 || total_pages <= 0 || !kv_indptr || !status)
    return SDA_ERR_INVALID_ARG;
  if (total_indices > 0 && !kv_indices) return SDA_ERR_INVALID_ARG;
  cudaError_t e = launch_validate(kv_indices, total_indices, kv_indptr, N, total_pages, status,
                                  static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) {
    note_cuda_error(e, "sda_validate_indices");
    return SDA_ERR_CUDA;
  }
  return SDA_OK;
}

sda_status sda_topk_slots(const float* scores, int64_t score_stride, const int32_t* lengths,
                          const int32_t* block_table, int64_t bt_stride, int N, int k,
                          int k_per_block, int32_t* comp_indptr, int32_t* comp_block,
                          int32_t* comp_slot, int64_t capacity, int32_t* status, void* stream) {
  if (N < 0 || k < 0 || k_per_block <= 0 || score_stride < 0 || score_stride > 0x7fffffffll ||
      bt_stride < 0 || bt_stride * static_cast<int64_t>(k_per_block) < score_stride ||
      capacity < 0 || capacity > 0x7fffffffll)
    return SDA_ERR_INVALID_ARG;
  if (!comp_indptr || !status) return SDA_ERR_INVALID_ARG;
  if (N > 0 && !lengths) return SDA_ERR_INVALID_ARG;
  if (N > 0 && k > 0 && score_stride > 0 && (!scores || !block_table)) return SDA_ERR_INVALID_ARG;
  if (capacity > 0 && (!comp_block || !comp_slot)) return SDA_ERR_INVALID_ARG;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaMemsetAsync(status, 0, sizeof(int32_t), st);
  if (e == cudaSuccess && g_ev_before && g_ev_after) e = cudaEventRecord(g_ev_before, st);
  if (e == cudaSuccess)
    e = launch_topk_slots(scores, score_stride, lengths, block_table, bt_stride, N, k,
                          k_per_block, comp_indptr, comp_block, comp_slot, capacity, status, st);
  if (e == cudaSuccess && g_ev_before && g_ev_after) e = cudaEventRecord(g_ev_after, st);
  if (e != cudaSuccess) {
    note_cuda_error(e, "sda_topk_slots");
    return SDA_ERR_CUDA;
  }
  return SDA_OK;
}

static sda_status store_common(const void* q, const void* kv, const void* q_norm_w,
                               const void* kv_norm_w, const float* cos_cache,
                               const float* sin_cache, int max_pos, const int32_t* positions,
                               const int32_t* state_slot, int N, int H, int D, int rope_dim,
                               float eps, int win, int64_t swa_pages, int64_t total_pages,
                               void* q_out, void* pool, uint8_t* pool_fp8, float* pool_scale,
                               int32_t* status, void* stream, const char* who) {
  using namespace sda;
  if (N < 0 || H < 1 || D < 8 || D > 2048 || D % 8 || rope_dim < 0 || rope_dim > D ||
      rope_dim % 8 || max_pos < 0 || win <= 0 || swa_pages < 0 || total_pages <= 0 ||
      swa_pages > total_pages || !(eps >= 0.f) || !std::isfinite(eps))
    return SDA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(N) * (H + 1) > (int64_t{1} << 30)) return SDA_ERR_INVALID_ARG;
  if (!status || !q_norm_w || !kv_norm_w) return SDA_ERR_INVALID_ARG;
  if (N > 0 && (!q || !kv || !positions || !state_slot || !q_out)) return SDA_ERR_INVALID_ARG;
  if (N > 0 && rope_dim > 0 && max_pos > 0 && (!cos_cache || !sin_cache)) return SDA_ERR_INVALID_ARG;
  if (N > 0 && !pool && !pool_fp8) return SDA_ERR_INVALID_ARG;
  if (pool_fp8 && !pool_scale) return SDA_ERR_INVALID_ARG;
  const void* vec16[] = {q, kv, q_norm_w, kv_norm_w, q_out, pool, pool_fp8, cos_cache, sin_cache};
  for (const void* ptr : vec16)
    if (ptr && !aligned(ptr, 16)) return SDA_ERR_INVALID_ARG;
  if (pool_scale && !aligned(pool_scale, 4)) return SDA_ERR_INVALID_ARG;
  // q_out is either q itself (in place) or a disjoint buffer.
  const size_t qbytes = (size_t)N * H * D * 2;
  const uintptr_t a = reinterpret_cast<uintptr_t>(q), b = reinterpret_cast<uintptr_t>(q_out);
  if (N > 0 && a != b && a < b + qbytes && b < a + qbytes) return SDA_ERR_INVALID_ARG;
  DeviceCaps caps;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = device_caps(&caps);
  if (e == cudaSuccess) e = cudaMemsetAsync(status, 0, sizeof(int32_t), st);
  if (e == cudaSuccess && g_ev_before && g_ev_after) e = cudaEventRecord(g_ev_before, st);
  if (e == cudaSuccess)
    e = launch_qk_norm_rope_store(q, kv, q_norm_w, kv_norm_w, cos_cache, sin_cache, max_pos,
                                  positions, state_slot, N, H, D, rope_dim, eps, win, swa_pages,
                                  q_out, pool, pool_fp8, pool_scale, status, caps.num_sms, st);
  if (e == cudaSuccess && g_ev_before && g_ev_after) e = cudaEventRecord(g_ev_after, st);
  if (e != cudaSuccess) {
    note_cuda_error(e, who);
    return SDA_ERR_CUDA;
  }
  return SDA_OK;
}

sda_status sda_qk_norm_rope_swa_store(const void* q, const void* kv, const void* q_norm_w,
                                      const void* kv_norm_w, const float* cos_cache,
                                      const float* sin_cache, int max_pos,
                                      const int32_t* positions, const int32_t* state_slot, int N,
                                      int H, int D, int rope_dim, float eps, int win,
                                      int64_t swa_pages, int64_t total_pages, void* q_out,
                                      void* unified_kv, int32_t* status, void* stream) {
  if (N > 0 && !unified_kv) return SDA_ERR_INVALID_ARG;
  return store_common(q, kv, q_norm_w, kv_norm_w, cos_cache, sin_cache, max_pos, positions,
                      state_slot, N, H, D, rope_dim, eps, win, swa_pages, total_pages, q_out,
                      unified_kv, nullptr, nullptr, status, stream, "sda_qk_norm_rope_swa_store");
}

sda_status sda_qk_norm_rope_swa_store_fp8(const void* q, const void* kv, const void* q_norm_w,
                                          const void* kv_norm_w, const float* cos_cache,
                                          const float* sin_cache, int max_pos,
                                          const int32_t* positions, const int32_t* state_slot,
                                          int N, int H, int D, int rope_dim, float eps, int win,
                                          int64_t swa_pages, int64_t total_pages, void* q_out,
                                          void* kv_fp8, float* kv_scale, int32_t* status,
                                          void* stream) {
  if (N > 0 && (!kv_fp8 || !kv_scale)) return SDA_ERR_INVALID_ARG;
  return store_common(q, kv, q_norm_w, kv_norm_w, cos_cache, sin_cache, max_pos, positions,
                      state_slot, N, H, D, rope_dim, eps, win, swa_pages, total_pages, q_out,
                      nullptr, static_cast<uint8_t*>(kv_fp8), kv_scale, status, stream,
                      "sda_qk_norm_rope_swa_store_fp8");
}

// The checks that the paged-cache operators share; what the kernels trust.
static sda_status chunk_geometry_ok(ChunkGeom& g) {
  if (g.B < 0 || g.T < 0 || g.k_per_block <= 0 || g.max_blocks < 0 || g.window < 0 || g.first < 0)
    return SDA_ERR_INVALID_ARG;
  if (g.total_pages <= 0 || g.total_pages > 0x7fffffffll || g.base < 0 || g.base > g.total_pages)
    return SDA_ERR_INVALID_ARG;
  if (!shape_supported(g.H, g.D)) return SDA_ERR_UNSUPPORTED;
  // rows are counted in 32 bits, 64 of them past the end being addressable
  if (static_cast<int64_t>(g.T) * g.H > 0x7fffffffll - 64 || g.B > (1 << 24))
    return SDA_ERR_INVALID_ARG;
  g.set_h();
  return SDA_OK;
}

static bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return na > 0 && nb > 0 && x < y + nb && y < x + na;
}

// The small arrays that the CTAs of a paged-cache call read at any time.
static bool overlaps_tables(const ChunkGeom& g, const void* p, size_t n) {
  return overlaps(g.block_table, static_cast<size_t>(g.B) * g.max_blocks * 4, p, n) ||
         overlaps(g.q_indptr, (static_cast<size_t>(g.B) + 1) * 4, p, n) ||
         overlaps(g.kv_len, static_cast<size_t>(g.B) * 4, p, n);
}

sda_status sda_paged_error_flag(const void* workspace, int32_t* device_flag, void* stream) {
  if (!workspace || !device_flag || !aligned(workspace, 256) || !aligned(device_flag, 4))
    return SDA_ERR_INVALID_ARG;
  const cudaError_t e = launch_paged_error(workspace, device_flag, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) {
    note_cuda_error(e, "sda_paged_error_flag");
    return SDA_ERR_CUDA;
  }
  return SDA_OK;
}

sda_status sda_chunk_attention_workspace_size(int B, int T, int H, int D, size_t* bytes) {
  if (!bytes) return SDA_ERR_INVALID_ARG;
  ChunkGeom g = {};
  g.B = B, g.T = T, g.H = H, g.D = D, g.k_per_block = 1, g.total_pages = 1;
  const sda_status s = chunk_geometry_ok(g);
  if (s != SDA_OK) return s;
  DeviceCaps caps;
  const cudaError_t e = paged_caps(kOpAttention, &caps);
  if (e != cudaSuccess) {
    note_cuda_error(e, "sda_chunk_attention_workspace_size");
    return SDA_ERR_CUDA;
  }
  *bytes = chunk_layout(g, caps.num_sms).total;
  return SDA_OK;
}

sda_status sda_chunk_attention(const void* q, const void* unified_kv, int64_t total_pages,
                               const int32_t* block_table, int max_blocks, int k_per_block,
                               int64_t base, const int32_t* q_indptr, const int32_t* kv_len,
                               const float* attn_sink, float softmax_scale, int window, int first,
                               int B, int T, int H, int D, void* out, float* lse, void* workspace,
                               size_t workspace_bytes, void* stream) {
  ChunkGeom g{q_indptr, kv_len,      block_table, B,      T,    H, D, max_blocks,
                    k_per_block, base, total_pages, window, first, 0, 0};
  const sda_status s = chunk_geometry_ok(g);
  if (s != SDA_OK) return s;
  if (B == 0 || T == 0) return SDA_OK;
  if (!q || !unified_kv || !q_indptr || !kv_len || !attn_sink || !out || !lse || !workspace)
    return SDA_ERR_INVALID_ARG;
  if (max_blocks > 0 && !block_table) return SDA_ERR_INVALID_ARG;
  for (const void* ptr : {q, unified_kv, static_cast<const void*>(out)})
    if (!aligned(ptr, 16)) return SDA_ERR_INVALID_ARG;
  for (const void* ptr : {static_cast<const void*>(q_indptr), static_cast<const void*>(kv_len),
                          static_cast<const void*>(block_table), static_cast<const void*>(attn_sink),
                          static_cast<const void*>(lse)})
    if (!aligned(ptr, 4)) return SDA_ERR_INVALID_ARG;
  // a unit's out and lse are written while other units still read q and the pool
  const size_t rows = static_cast<size_t>(T) * H, on = rows * D * 2, ln = rows * 4;
  const size_t pn = static_cast<size_t>(total_pages) * D * 2;
  if (overlaps(q, on, out, on) || overlaps(unified_kv, pn, out, on) || overlaps(q, on, lse, ln) ||
      overlaps(unified_kv, pn, lse, ln) || overlaps(out, on, lse, ln))
    return SDA_ERR_INVALID_ARG;
  if (!aligned(workspace, 256)) return SDA_ERR_WORKSPACE;
  const size_t sn = static_cast<size_t>(H) * 4;
  if (overlaps_tables(g, out, on) || overlaps_tables(g, lse, ln) || overlaps(attn_sink, sn, out, on) ||
      overlaps(attn_sink, sn, lse, ln))
    return SDA_ERR_INVALID_ARG;
  DeviceCaps caps;
  cudaError_t e = paged_caps(kOpAttention, &caps);
  if (e != cudaSuccess) {
    note_cuda_error(e, "sda_chunk_attention");
    return SDA_ERR_CUDA;
  }
  const ChunkLayout L = chunk_layout(g, caps.num_sms);
  if (workspace_bytes < L.total) return SDA_ERR_WORKSPACE;
  if (overlaps(q, on, workspace, L.total) || overlaps(unified_kv, pn, workspace, L.total) ||
      overlaps_tables(g, workspace, L.total) || overlaps(attn_sink, sn, workspace, L.total) ||
      overlaps(out, on, workspace, L.total) || overlaps(lse, ln, workspace, L.total))
    return SDA_ERR_INVALID_ARG;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  e = launch_chunk_plan(g, L, workspace, st);
  if (e == cudaSuccess && g_ev_before && g_ev_after) e = cudaEventRecord(g_ev_before, st);
  if (e == cudaSuccess)
    e = launch_chunk_attn(q, unified_kv, g, attn_sink, softmax_scale, out, lse, L, workspace, st);
  if (e == cudaSuccess && g_ev_before && g_ev_after) e = cudaEventRecord(g_ev_after, st);
  if (e == cudaSuccess) e = launch_chunk_combine(attn_sink, g, out, lse, L, workspace, st);
  if (e != cudaSuccess) {
    note_cuda_error(e, "sda_chunk_attention");
    return SDA_ERR_CUDA;
  }
  return SDA_OK;
}

// The mass's score rows span the whole table: S = max_blocks * k_per_block.
static sda_status mass_geometry_ok(ChunkGeom& g) {
  const sda_status s = chunk_geometry_ok(g);
  if (s != SDA_OK) return s;
  const int64_t S = static_cast<int64_t>(g.max_blocks) * g.k_per_block;
  if (S > kMaxLen || (S / 128 + 1) * g.B > (1 << 26)) return SDA_ERR_INVALID_ARG;
  return SDA_OK;
}

sda_status sda_attention_mass_workspace_size(int B, int max_blocks, int k_per_block, size_t* bytes) {
  if (!bytes) return SDA_ERR_INVALID_ARG;
  ChunkGeom g = {};
  g.B = B, g.H = 1, g.D = 64, g.max_blocks = max_blocks, g.k_per_block = k_per_block;
  g.total_pages = 1;
  const sda_status s = mass_geometry_ok(g);
  if (s != SDA_OK) return s;
  DeviceCaps caps;
  const cudaError_t e = paged_caps(kOpMass, &caps);
  if (e != cudaSuccess) {
    note_cuda_error(e, "sda_attention_mass_workspace_size");
    return SDA_ERR_CUDA;
  }
  *bytes = mass_layout(B, static_cast<int64_t>(max_blocks) * k_per_block, caps.num_sms).total;
  return SDA_OK;
}

sda_status sda_attention_mass(const void* q, const void* unified_kv, int64_t total_pages,
                              const int32_t* block_table, int max_blocks, int k_per_block,
                              int64_t base, const int32_t* q_indptr, const int32_t* kv_len,
                              const float* lse, float softmax_scale, int window, int first,
                              const float* prev, float decay, int B, int T, int H, int D,
                              float* out, void* workspace, size_t workspace_bytes, void* stream) {
  ChunkGeom g{q_indptr, kv_len,      block_table, B,      T,    H, D, max_blocks,
                    k_per_block, base, total_pages, window, first, 0, 0};
  const sda_status s = mass_geometry_ok(g);
  if (s != SDA_OK) return s;
  const int64_t S = static_cast<int64_t>(max_blocks) * k_per_block;
  if (B == 0 || S == 0) return SDA_OK;
  if (!unified_kv || !block_table || !q_indptr || !kv_len || !out || !workspace)
    return SDA_ERR_INVALID_ARG;
  if (T > 0 && (!q || !lse)) return SDA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(unified_kv, 16)) return SDA_ERR_INVALID_ARG;
  for (const void* ptr : {static_cast<const void*>(q_indptr), static_cast<const void*>(kv_len),
                          static_cast<const void*>(block_table), static_cast<const void*>(lse),
                          static_cast<const void*>(prev), static_cast<const void*>(out)})
    if (!aligned(ptr, 4)) return SDA_ERR_INVALID_ARG;
  // out is prev itself or apart from it, and apart from what all CTAs read
  const size_t nb = static_cast<size_t>(B) * S * 4, rows = static_cast<size_t>(T) * H;
  if (prev && prev != out && overlaps(prev, nb, out, nb)) return SDA_ERR_INVALID_ARG;
  const size_t qn = rows * D * 2, pn = static_cast<size_t>(total_pages) * D * 2;
  if (overlaps(q, qn, out, nb) || overlaps(lse, rows * 4, out, nb) || overlaps(unified_kv, pn, out, nb) ||
      overlaps_tables(g, out, nb))
    return SDA_ERR_INVALID_ARG;
  if (!aligned(workspace, 256)) return SDA_ERR_WORKSPACE;
  DeviceCaps caps;
  cudaError_t e = paged_caps(kOpMass, &caps);
  if (e != cudaSuccess) {
    note_cuda_error(e, "sda_attention_mass");
    return SDA_ERR_CUDA;
  }
  const MassLayout L = mass_layout(B, S, caps.num_sms);
  if (workspace_bytes < L.total) return SDA_ERR_WORKSPACE;
  if (overlaps(q, qn, workspace, L.total) || overlaps(lse, rows * 4, workspace, L.total) ||
      overlaps(unified_kv, pn, workspace, L.total) || overlaps_tables(g, workspace, L.total) ||
      overlaps(prev, prev ? nb : 0, workspace, L.total) || overlaps(out, nb, workspace, L.total))
    return SDA_ERR_INVALID_ARG;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (g_ev_before && g_ev_after) e = cudaEventRecord(g_ev_before, st);
  if (e == cudaSuccess)
    e = launch_mass(q, unified_kv, g, lse, softmax_scale, prev, decay, out, L, workspace, st);
  if (e == cudaSuccess && g_ev_before && g_ev_after) e = cudaEventRecord(g_ev_after, st);
  if (e != cudaSuccess) {
    note_cuda_error(e, "sda_attention_mass");
    return SDA_ERR_CUDA;
  }
  return SDA_OK;
}

sda_status sda_evict_slots(const float* scores, const int32_t* slot_table, int64_t stride,
                           const int32_t* kv_len, int B, int budget, int first, int recent,
                           float* out_scores, int32_t* out_table, int64_t out_stride,
                           int32_t* out_len, int32_t* freed_slots, int64_t freed_capacity,
                           int32_t* freed_indptr, int32_t* status, void* stream) {
  if (B < 0 || B > (1 << 24) || stride < 0 || stride > kMaxEvictLen || budget < 0 || first < 0 ||
      recent < 0 || out_stride < 0 || out_stride > 0x7fffffffll || freed_capacity < 0)
    return SDA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(first) + recent > budget) return SDA_ERR_INVALID_ARG;
  const int64_t most = stride > budget ? stride - budget : 0;  // slots a sequence can free
  if (out_stride < (stride < budget ? stride : budget)) return SDA_ERR_INVALID_ARG;
  if (most * B > 0x7fffffffll || freed_capacity < most * B) return SDA_ERR_INVALID_ARG;
  if (!freed_indptr || !status || (freed_capacity > 0 && !freed_slots)) return SDA_ERR_INVALID_ARG;
  if (B > 0 && (!kv_len || !out_len)) return SDA_ERR_INVALID_ARG;
  if (B > 0 && stride > 0 && (!scores || !slot_table)) return SDA_ERR_INVALID_ARG;
  if (B > 0 && out_stride > 0 && (!out_scores || !out_table)) return SDA_ERR_INVALID_ARG;
  const void* words[] = {scores, slot_table, kv_len, out_scores, out_table, out_len, freed_slots,
                         freed_indptr, status};
  for (const void* ptr : words)
    if (!aligned(ptr, 4)) return SDA_ERR_INVALID_ARG;
  // what is written is in place (the same array with the same row length) or apart from
  // what is read, and apart from what else is written
  struct Span {
    const void* p;
    size_t n;
    const void* place;  // the input that it may be
  };
  const size_t in = static_cast<size_t>(B) * stride * 4, on = static_cast<size_t>(B) * out_stride * 4;
  const size_t bn = static_cast<size_t>(B) * 4;
  const bool same = stride == out_stride;
  const Span reads[] = {{scores, in, nullptr}, {slot_table, in, nullptr}, {kv_len, bn, nullptr}};
  const Span writes[] = {{out_scores, on, same ? scores : nullptr},
                         {out_table, on, same ? slot_table : nullptr},
                         {out_len, bn, kv_len},
                         {freed_slots, static_cast<size_t>(freed_capacity) * 4, nullptr},
                         {freed_indptr, bn + 4, nullptr},
                         {status, 4, nullptr}};
  for (const Span& w : writes) {
    for (const Span& r : reads)
      if (!(w.p == r.p && w.place == r.p) && overlaps(w.p, w.n, r.p, r.n)) return SDA_ERR_INVALID_ARG;
    for (const Span& o : writes)
      if (&o != &w && overlaps(w.p, w.n, o.p, o.n)) return SDA_ERR_INVALID_ARG;
  }
  const EvictArgs a{scores,  slot_table,  stride,         kv_len,       B,     budget, first, recent,
                    out_scores, out_table, out_stride, out_len, freed_slots, freed_capacity,
                    freed_indptr, status};
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  DeviceCaps caps;
  cudaError_t e = paged_caps(kOpEvict, &caps);
  if (e == cudaSuccess && g_ev_before && g_ev_after) e = cudaEventRecord(g_ev_before, st);
  if (e == cudaSuccess) e = launch_evict(a, st);
  if (e == cudaSuccess && g_ev_before && g_ev_after) e = cudaEventRecord(g_ev_after, st);
  if (e != cudaSuccess) {
    note_cuda_error(e, "sda_evict_slots");
    return SDA_ERR_CUDA;
  }
  return SDA_OK;
}

// The blocks that a pool holds, the last one perhaps in part.
static int64_t pool_blocks(const ChunkGeom& g) {
  return (g.total_pages - g.base + g.k_per_block - 1) / g.k_per_block;
}

// Bytes of workspace that either way of a call needs for itself.
static size_t fp8_own_bytes(const ChunkGeom& g, int num_sms) {
  const size_t a = chunk_fp8_layout(g, num_sms).total, b = chunk_layout(g, num_sms).total;
  return a > b ? a : b;
}

sda_status sda_chunk_attention_fp8_workspace_size(int B, int T, int H, int D, int max_blocks,
                                                  int k_per_block, size_t* bytes) {
  if (!bytes) return SDA_ERR_INVALID_ARG;
  ChunkGeom g = {};
  g.B = B, g.T = T, g.H = H, g.D = D, g.max_blocks = max_blocks, g.k_per_block = k_per_block;
  g.total_pages = 1;
  const sda_status s = chunk_geometry_ok(g);
  if (s != SDA_OK) return s;
  DeviceCaps caps;
  const cudaError_t e = paged_caps(kOpAttentionFp8, &caps);
  if (e != cudaSuccess) {
    note_cuda_error(e, "sda_chunk_attention_fp8_workspace_size");
    return SDA_ERR_CUDA;
  }
  *bytes = spread_layout(g, caps.num_sms, fp8_own_bytes(g, caps.num_sms)).total;
  return SDA_OK;
}

sda_status sda_chunk_attention_fp8(const void* q, const void* kv_fp8, const float* block_scale,
                                   int64_t total_pages, const int32_t* block_table, int max_blocks,
                                   int k_per_block, int64_t base, const int32_t* q_indptr,
                                   const int32_t* kv_len, const float* attn_sink, float softmax_scale,
                                   int window, int first, int B, int T, int H, int D, void* out,
                                   float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  ChunkGeom g{q_indptr, kv_len,      block_table, B,      T,    H, D, max_blocks,
              k_per_block, base, total_pages, window, first, 0, 0};
  const sda_status s = chunk_geometry_ok(g);
  if (s != SDA_OK) return s;
  if (B == 0 || T == 0) return SDA_OK;
  if (!q || !kv_fp8 || !block_scale || !q_indptr || !kv_len || !attn_sink || !out || !lse || !workspace)
    return SDA_ERR_INVALID_ARG;
  if (max_blocks > 0 && !block_table) return SDA_ERR_INVALID_ARG;
  for (const void* ptr : {q, kv_fp8, static_cast<const void*>(out)})
    if (!aligned(ptr, 16)) return SDA_ERR_INVALID_ARG;
  const void* words[] = {block_scale, q_indptr, kv_len, block_table, attn_sink, lse};
  for (const void* ptr : words)
    if (!aligned(ptr, 4)) return SDA_ERR_INVALID_ARG;
  // what is written overlaps neither what other units still read nor what else is written
  struct Span {
    const void* p;
    size_t n;
  };
  const size_t on = static_cast<size_t>(T) * H * D * 2, ln = static_cast<size_t>(T) * H * 4;
  const Span spans[] = {{q, on},
                        {kv_fp8, static_cast<size_t>(total_pages) * D},
                        {block_scale, static_cast<size_t>(pool_blocks(g)) * 4},
                        {attn_sink, static_cast<size_t>(H) * 4},
                        {out, on},
                        {lse, ln}};
  const auto clash = [&](const void* p, size_t n, const Span* self) {
    bool any = overlaps_tables(g, p, n);
    for (const Span& x : spans) any |= &x != self && overlaps(p, n, x.p, x.n);
    return any;
  };
  if (clash(out, on, &spans[4]) || clash(lse, ln, &spans[5])) return SDA_ERR_INVALID_ARG;
  if (!aligned(workspace, 256)) return SDA_ERR_WORKSPACE;
  DeviceCaps caps;
  cudaError_t e = paged_caps(kOpAttentionFp8, &caps);
  if (e != cudaSuccess) {
    note_cuda_error(e, "sda_chunk_attention_fp8");
    return SDA_ERR_CUDA;
  }
  const size_t own = fp8_own_bytes(g, caps.num_sms);
  if (workspace_bytes < own) return SDA_ERR_WORKSPACE;
  const SpreadLayout S = spread_layout(g, caps.num_sms, own);
  const bool spread = S.worth && workspace_bytes >= S.total;
  if (clash(workspace, spread ? S.total : own, nullptr)) return SDA_ERR_INVALID_ARG;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const ChunkGeom sg = spread ? spread_geometry(g, S, workspace) : g;
  const ChunkLayout L = spread ? chunk_layout(sg, caps.num_sms) : chunk_fp8_layout(g, caps.num_sms);
  e = launch_chunk_plan(sg, L, workspace, st);
  if (e == cudaSuccess && g_ev_before && g_ev_after) e = cudaEventRecord(g_ev_before, st);
  if (e == cudaSuccess && spread) e = launch_spread(g, kv_fp8, block_scale, S, workspace, st);
  if (e == cudaSuccess)
    e = spread ? launch_chunk_spread(q, sg, attn_sink, softmax_scale, out, lse, L, S, workspace, st)
               : launch_chunk_fp8(q, kv_fp8, block_scale, g, attn_sink, softmax_scale, out, lse, L, workspace, st);
  if (e == cudaSuccess && g_ev_before && g_ev_after) e = cudaEventRecord(g_ev_after, st);
  if (e == cudaSuccess) e = launch_chunk_combine(attn_sink, sg, out, lse, L, workspace, st);
  if (e != cudaSuccess) {
    note_cuda_error(e, "sda_chunk_attention_fp8");
    return SDA_ERR_CUDA;
  }
  return SDA_OK;
}

static sda_status append_common(AppendParams p, void* stream, const char* who) {
  ChunkGeom& g = p.g;
  const int D = g.D, T = g.T, R = p.R;
  if (g.B < 0 || T < 0 || g.H < 0 || g.k_per_block <= 0 || g.max_blocks < 0 || g.B > (1 << 24) ||
      g.total_pages <= 0 || g.total_pages > 0x7fffffffll || g.base < 0 || g.base > g.total_pages ||
      R < 0 || R > D || R % 8 || p.max_pos < 0 || !(p.eps >= 0.f) || !std::isfinite(p.eps))
    return SDA_ERR_INVALID_ARG;
  if (D < 16 || D > 1024 || D % 16) return SDA_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(T) * (g.H + 1) > 0x7fffffffll) return SDA_ERR_INVALID_ARG;
  if (!p.status || !aligned(p.status, 4)) return SDA_ERR_INVALID_ARG;
  const bool work = g.B > 0 && T > 0;
  if (work) {
    if (!p.kv || !g.q_indptr || !g.kv_len || (!p.pool && !p.codes) || (p.codes && !p.scale) ||
        (g.max_blocks > 0 && !g.block_table) || (g.H > 0 && (!p.q || !p.q_out)) ||
        (R > 0 && p.max_pos > 0 && (!p.cos_cache || !p.sin_cache)))
      return SDA_ERR_INVALID_ARG;
    const void* vec16[] = {p.q, p.kv, p.q_w, p.kv_w, p.cos_cache, p.sin_cache, p.q_out, p.pool, p.codes};
    for (const void* ptr : vec16)
      if (!aligned(ptr, 16)) return SDA_ERR_INVALID_ARG;
    const void* words[] = {g.block_table, g.q_indptr, g.kv_len, p.scale};
    for (const void* ptr : words)
      if (!aligned(ptr, 4)) return SDA_ERR_INVALID_ARG;
    // q_out is q itself or apart from it; else what is written overlaps neither what is
    // read nor what else is written
    struct Span {
      const void* p;
      size_t n;
    };
    const size_t row = static_cast<size_t>(D) * 2, qn = g.H * T * row, cn = static_cast<size_t>(p.max_pos) * R * 2;
    const Span reads[] = {{p.q, qn}, {p.kv, T * row}, {p.q_w, p.q_w ? row : 0}, {p.kv_w, p.kv_w ? row : 0},
                          {p.cos_cache, cn}, {p.sin_cache, cn}};
    const Span writes[] = {{p.q_out, qn},
                           {p.pool, p.pool ? g.total_pages * row : 0},
                           {p.codes, p.codes ? static_cast<size_t>(g.total_pages) * D : 0},
                           {p.scale, p.codes ? static_cast<size_t>(pool_blocks(g)) * 4 : 0},
                           {p.status, 4}};
    for (const Span& w : writes) {
      if (overlaps_tables(g, w.p, w.n)) return SDA_ERR_INVALID_ARG;
      for (const Span& r : reads) {
        // (q_out and q themselves: another array at q's address is read by other warps)
        const bool in_place = &w == &writes[0] && &r == &reads[0] && p.q_out == p.q;
        if (!in_place && overlaps(w.p, w.n, r.p, r.n)) return SDA_ERR_INVALID_ARG;
      }
      for (const Span& o : writes)
        if (&o != &w && overlaps(w.p, w.n, o.p, o.n)) return SDA_ERR_INVALID_ARG;
    }
  }
  DeviceCaps caps;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = device_caps(&caps);
  p.one_status = work && append_one_status(p);
  if (e == cudaSuccess && !p.one_status) e = cudaMemsetAsync(p.status, 0, sizeof(int32_t), st);
  if (e == cudaSuccess && g_ev_before && g_ev_after) e = cudaEventRecord(g_ev_before, st);
  if (e == cudaSuccess && work) e = launch_append(p, caps.num_sms, st);
  if (e == cudaSuccess && g_ev_before && g_ev_after) e = cudaEventRecord(g_ev_after, st);
  if (e != cudaSuccess) {
    note_cuda_error(e, who);
    return SDA_ERR_CUDA;
  }
  return SDA_OK;
}

static AppendParams append_params(const void* q, const void* kv, const void* q_norm_w, const void* kv_norm_w,
                                  const float* cos_cache, const float* sin_cache, int max_pos,
                                  const int32_t* block_table, int max_blocks, int k_per_block, int64_t base,
                                  const int32_t* q_indptr, const int32_t* kv_len, int B, int T, int H, int D,
                                  int rope_dim, float eps, int64_t total_pages, void* q_out, int32_t* status) {
  AppendParams p = {};
  p.q = static_cast<const uint16_t*>(H > 0 ? q : nullptr);
  p.kv = static_cast<const uint16_t*>(kv);
  p.q_w = static_cast<const uint16_t*>(H > 0 ? q_norm_w : nullptr);
  p.kv_w = static_cast<const uint16_t*>(kv_norm_w);
  p.cos_cache = cos_cache;
  p.sin_cache = sin_cache;
  p.g = ChunkGeom{q_indptr, kv_len,      block_table, B, T, H, D, max_blocks,
                  k_per_block, base, total_pages, 0, 0, 0, 0};
  p.R = rope_dim;
  p.max_pos = max_pos;
  p.eps = eps;
  p.inv_d = (D & (D - 1)) == 0 ? 1.f / static_cast<float>(D) : 0.f;
  p.q_out = static_cast<uint16_t*>(H > 0 ? q_out : nullptr);
  p.status = status;
  return p;
}

sda_status sda_append_rows(const void* q, const void* kv, const void* q_norm_w, const void* kv_norm_w,
                           const float* cos_cache, const float* sin_cache, int max_pos,
                           const int32_t* block_table, int max_blocks, int k_per_block, int64_t base,
                           const int32_t* q_indptr, const int32_t* kv_len, int B, int T, int H, int D,
                           int rope_dim, float eps, int64_t total_pages, void* q_out, void* unified_kv,
                           int32_t* status, void* stream) {
  AppendParams p = append_params(q, kv, q_norm_w, kv_norm_w, cos_cache, sin_cache, max_pos, block_table,
                                 max_blocks, k_per_block, base, q_indptr, kv_len, B, T, H, D, rope_dim, eps,
                                 total_pages, q_out, status);
  p.pool = static_cast<uint16_t*>(unified_kv);
  return append_common(p, stream, "sda_append_rows");
}

sda_status sda_append_rows_fp8(const void* q, const void* kv, const void* q_norm_w, const void* kv_norm_w,
                               const float* cos_cache, const float* sin_cache, int max_pos,
                               const int32_t* block_table, int max_blocks, int k_per_block, int64_t base,
                               const int32_t* q_indptr, const int32_t* kv_len, int B, int T, int H, int D,
                               int rope_dim, float eps, int64_t total_pages, void* q_out, void* kv_fp8,
                               float* block_scale, int32_t* status, void* stream) {
  AppendParams p = append_params(q, kv, q_norm_w, kv_norm_w, cos_cache, sin_cache, max_pos, block_table,
                                 max_blocks, k_per_block, base, q_indptr, kv_len, B, T, H, D, rope_dim, eps,
                                 total_pages, q_out, status);
  p.codes = static_cast<uint8_t*>(kv_fp8);
  p.scale = block_scale;
  return append_common(p, stream, "sda_append_rows_fp8");
}

}  // extern "C"
