// Host-side pieces shared by the files that implement the C ABI: the handle,
// the last-error message, the argument checks and the debug kernel timing.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <string>

#include "../../include/tpfuse.h"
#include "tpf_internal.hpp"

namespace tpf {
constexpr int kKernelTimes = 256;   // debug kernel-timing records held per handle
}  // namespace tpf

struct tpf_context {
  int device = 0;
  int num_cus = 0;
  hipStream_t side = nullptr;           // reductions (reducing ops) or gather copies (AllGather)
  hipStream_t gemm2 = nullptr;          // every other chunk's GEMM (two-stream scheduler)
  hipEvent_t ev_fork = nullptr, ev_join = nullptr, ev_join2 = nullptr;
  hipEvent_t ev_chunk[tpf::kMaxChunks] = {};
  hipEvent_t ev_slice[tpf::kMaxShards] = {};
  tpf::Ctrl* ctrl = nullptr;
  int* tile_cnt = nullptr;             // kTileCounters per-output-tile counters (tile scheduler)
  int64_t spin_limit = 0;
  int unreachable = 0;
  tpf::TimelineEvent* timeline = nullptr;   // caller-owned device buffer (debug)
  int timeline_cap = 0;
  // Debug kernel timing: a ring of timing-event pairs around each call's
  // dominant launch.
  bool ktime = false;
  hipEvent_t kt0[tpf::kKernelTimes] = {}, kt1[tpf::kKernelTimes] = {};
  int kt_next = 0;      // ring slot of the next record
  int kt_count = 0;     // records held (<= kKernelTimes)
  int last_sched = -1;  // scheduler the last call ran (AUTO resolved), -1 before any
  void* scratch = nullptr;  // this device's copy of the no-allocation workspace
  tpf::DelayArgs delay{};        // debug: timing perturbation of the producers (tpf_debug_set_delay)
};

namespace tpf {

inline thread_local std::string g_last_error;

inline int fail(int code, const std::string& msg) {
  g_last_error = msg;
  return code;
}

inline int hip_fail(hipError_t e, const char* what) {
  return fail(TPF_ERR_HIP, std::string(what) + ": " + hipGetErrorString(e));
}

#define TPF_HIP(call)                                  \
  do {                                                 \
    hipError_t e_ = (call);                            \
    if (e_ != hipSuccess) return hip_fail(e_, #call);  \
  } while (0)

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool valid_dtype(int d) { return d == TPF_BF16 || d == TPF_F32; }

inline int out_kind(int dtype) { return dtype == TPF_F32 ? OUT_F32 : OUT_BF16; }

inline int check_ptrs(const void* const* arr, int count, const char* name) {
  if (!arr) return fail(TPF_ERR_INVALID_ARG, std::string(name) + " array is NULL");
  for (int i = 0; i < count; ++i) {
    if (!arr[i]) return fail(TPF_ERR_INVALID_ARG, std::string(name) + "[" + std::to_string(i) + "] is NULL");
    if (!aligned16(arr[i]))
      return fail(TPF_ERR_ALIGNMENT, std::string(name) + "[" + std::to_string(i) + "] is not 16-byte aligned");
  }
  return TPF_OK;
}

inline int check_ptr(const void* ptr, const char* name) {
  if (!ptr) return fail(TPF_ERR_INVALID_ARG, std::string(name) + " is NULL");
  if (!aligned16(ptr)) return fail(TPF_ERR_ALIGNMENT, std::string(name) + " is not 16-byte aligned");
  return TPF_OK;
}

inline int check_ws(void* ws, size_t ws_bytes, size_t need) {
  if (need == 0) return TPF_OK;
  if (!ws) return fail(TPF_ERR_WORKSPACE, "workspace is NULL but " + std::to_string(need) + " bytes are needed");
  if (!aligned16(ws)) return fail(TPF_ERR_ALIGNMENT, "workspace is not 16-byte aligned");
  if (ws_bytes < need)
    return fail(TPF_ERR_WORKSPACE, "workspace has " + std::to_string(ws_bytes) + " bytes, needs " + std::to_string(need));
  return TPF_OK;
}

inline int check_handle(tpf_handle h) {
  if (!h) return fail(TPF_ERR_INVALID_ARG, "handle is NULL");
  return TPF_OK;
}

inline int set_device(tpf_handle h) {
  TPF_HIP(hipSetDevice(h->device));
  return TPF_OK;
}

// Debug kernel timing: record the start / stop event of the current call's
// dominant launch on the stream it is launched on.
inline int ktime_start(tpf_handle h, hipStream_t s) {
  if (h->ktime) TPF_HIP(hipEventRecord(h->kt0[h->kt_next], s));
  return TPF_OK;
}
inline int ktime_stop(tpf_handle h, hipStream_t s) {
  if (!h->ktime) return TPF_OK;
  TPF_HIP(hipEventRecord(h->kt1[h->kt_next], s));
  h->kt_next = (h->kt_next + 1) % kKernelTimes;
  h->kt_count = std::min(h->kt_count + 1, kKernelTimes);
  return TPF_OK;
}

#define TPF_TIMED(h, s, launch)      \
  do {                               \
    int st_ = ktime_start((h), (s)); \
    if (st_) return st_;             \
    TPF_HIP(launch);                 \
    st_ = ktime_stop((h), (s));      \
    if (st_) return st_;             \
  } while (0)

}  // namespace tpf
