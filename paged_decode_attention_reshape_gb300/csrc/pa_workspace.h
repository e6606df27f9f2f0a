// pa_workspace.h -- the library-held workspace (host code; no device header, so that a host test can compile it
// against a stand-in of the runtime).
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "../../include/pa.h"

namespace pa {

// One growing allocation per device: an arrival-counter region, then the partial states of
// the call.  The counter region keeps its size between calls (and is zero between them), so
// a call of one shape never leaves its partial states where a call of another shape, with
// more units, looks for its counters.
struct DevWorkspace {
  void *ptr = nullptr;
  size_t bytes = 0;     // the whole allocation
  size_t counters = 0;  // its counter region
  bool captured = false;  // a captured graph holds the address: the allocation outlives its use here
  void *retired = nullptr;  // an allocation that a capture replaced, freed when an eager call next grows
};
inline std::mutex g_ws_mu;
inline DevWorkspace g_ws[64];

// `bytes` of device memory, its first `counters` zero, while a stream is being captured: outside the
// graph, by calls that a capture of the relaxed mode allows.  (Allocated on the captured stream it
// would be memory of that graph, which no other call may use.)  Never freed.
inline void *allocate_beside_capture(size_t bytes, size_t counters) {
  cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
  if (cudaThreadExchangeStreamCaptureMode(&mode) != cudaSuccess) return nullptr;
  void *ptr = nullptr;
  cudaStream_t own = nullptr;
  bool ok = cudaStreamCreateWithFlags(&own, cudaStreamNonBlocking) == cudaSuccess;
  if (ok) {
    ok = cudaMalloc(&ptr, bytes) == cudaSuccess;
    ok = ok && cudaMemsetAsync(ptr, 0, counters, own) == cudaSuccess && cudaStreamSynchronize(own) == cudaSuccess;
    if (!ok && ptr) cudaFree(ptr);
    cudaStreamDestroy(own);
  }
  (void)cudaThreadExchangeStreamCaptureMode(&mode);
  if (!ok) (void)cudaGetLastError();
  return ok ? ptr : nullptr;
}

// The current device's workspace with room for `counters` bytes of arrival counters and `data`
// bytes behind them.  optional: for a call that goes on without it; where there is no memory for more, what is
// held stays (the calls that cannot do without it keep theirs).
inline int internal_workspace(size_t counters, size_t data, cudaStream_t st, DevWorkspace *out, bool optional = false) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return PA_ERR_CUDA;
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(st, &cap) != cudaSuccess) {
    (void)cudaGetLastError();
    return PA_ERR_CUDA;
  }
  const bool capturing = cap != cudaStreamCaptureStatusNone;
  std::lock_guard<std::mutex> g(g_ws_mu);
  DevWorkspace &w = g_ws[dev];
  if (w.counters < counters || w.bytes - w.counters < data) {
    const size_t nc = std::max(w.counters, counters), nd = std::max(w.bytes - w.counters, data);
    DevWorkspace next;
    if (capturing) {
      next.ptr = allocate_beside_capture(nc + nd, nc);
      if (!next.ptr) return PA_ERR_CUDA;  // (the one there is stays)
      next.retired = w.ptr && !w.captured ? w.ptr : w.retired;
    } else {
      auto let_go = [&] {
        if (w.ptr && !w.captured) cudaFreeAsync(w.ptr, st);
        if (w.retired) cudaFreeAsync(w.retired, st);
        w = DevWorkspace{};
      };
      if (!optional) let_go();  // (the new one may take its room)
      if (cudaMallocAsync(&next.ptr, nc + nd, st) != cudaSuccess) {
        (void)cudaGetLastError();  // the failed allocation is reported here, not by a later launch
        return PA_ERR_CUDA;
      }
      if (cudaMemsetAsync(next.ptr, 0, nc, st) != cudaSuccess) {
        cudaFreeAsync(next.ptr, st);
        return PA_ERR_CUDA;
      }
      if (optional) let_go();
    }
    next.bytes = nc + nd;
    next.counters = nc;
    w = next;
  }
  if (capturing) w.captured = true;
  *out = w;
  return PA_OK;
}

}  // namespace pa
