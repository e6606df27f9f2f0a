"""The library-held workspace (csrc/pa_workspace.h) against a stand-in of the CUDA runtime with little memory:
what it holds, frees and zeroes when calls make it grow and when they cannot."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
RUNTIME = r"""
#pragma once
#include <cstddef>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
typedef int cudaError_t;
typedef struct S *cudaStream_t;
enum { cudaSuccess = 0, cudaErrorMemoryAllocation = 2 };
enum cudaStreamCaptureStatus { cudaStreamCaptureStatusNone, cudaStreamCaptureStatusActive };
enum cudaStreamCaptureMode { cudaStreamCaptureModeGlobal, cudaStreamCaptureModeRelaxed = 2 };
enum { cudaStreamNonBlocking = 1 };
inline std::map<void *, size_t> live;  // allocations
inline size_t most = 1000, used = 0;
inline int pending = 0, capturing = 0, frees = 0;
inline cudaError_t cudaMalloc(void **p, size_t n) {
  if (used + n > most) { pending = cudaErrorMemoryAllocation; *p = nullptr; return pending; }
  *p = malloc(n); memset(*p, 0xff, n); live[*p] = n; used += n; return 0;
}
inline cudaError_t cudaFree(void *p) {
  auto at = live.find(p);
  if (at == live.end()) { printf("freed twice\n"); exit(1); }
  used -= at->second; live.erase(at); free(p); ++frees; return 0;
}
inline cudaError_t cudaMallocAsync(void **p, size_t n, cudaStream_t) { return cudaMalloc(p, n); }
inline cudaError_t cudaFreeAsync(void *p, cudaStream_t) { return cudaFree(p); }
inline cudaError_t cudaMemsetAsync(void *p, int v, size_t n, cudaStream_t) { memset(p, v, n); return 0; }
inline cudaError_t cudaGetLastError() { int e = pending; pending = 0; return e; }
inline cudaError_t cudaGetDevice(int *d) { *d = 0; return 0; }
inline cudaError_t cudaStreamIsCapturing(cudaStream_t, cudaStreamCaptureStatus *s) {
  *s = capturing ? cudaStreamCaptureStatusActive : cudaStreamCaptureStatusNone; return 0;
}
inline cudaError_t cudaThreadExchangeStreamCaptureMode(cudaStreamCaptureMode *) { return 0; }
inline cudaError_t cudaStreamCreateWithFlags(cudaStream_t *s, int) { *s = nullptr; return 0; }
inline cudaError_t cudaStreamDestroy(cudaStream_t) { return 0; }
inline cudaError_t cudaStreamSynchronize(cudaStream_t) { return 0; }
"""
MAIN = r"""
#include "pa_workspace.h"
using namespace pa;
#define CHECK(x) do { if (!(x)) { printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)
static bool zero(const DevWorkspace &w) {
  for (size_t i = 0; i < w.counters; ++i) if (static_cast<char *>(w.ptr)[i]) return false;
  return true;
}
int main() {
  DevWorkspace a, b, c;
  for (capturing = 0; capturing < 2; ++capturing) {
    g_ws[0] = DevWorkspace{};
    live.clear(), used = 0, most = 1000;
    // a call that needs it, then one that would like more than there is: the first one's stays, untouched
    CHECK(internal_workspace(100, 200, nullptr, &a) == PA_OK && a.ptr && a.counters == 100 && a.bytes >= 300 && zero(a));
    frees = 0;
    CHECK(internal_workspace(0, 5000, nullptr, &b, true) == PA_ERR_CUDA);
    CHECK(pending == 0 && frees == 0 && g_ws[0].ptr == a.ptr && live.count(a.ptr));
    CHECK(internal_workspace(100, 200, nullptr, &b) == PA_OK && b.ptr == a.ptr && frees == 0);
    // and where there is room for both at once, the larger one takes its place, with as many counters
    CHECK(internal_workspace(0, 500, nullptr, &b, true) == PA_OK && b.counters == 100 && b.bytes >= 600 && zero(b));
    CHECK(internal_workspace(100, 200, nullptr, &c) == PA_OK && c.ptr == b.ptr);
    CHECK(live.count(b.ptr) && live.count(a.ptr) == (capturing ? 1u : 0u) && frees == (capturing ? 0 : 1));
  }
  // a call that cannot do without it may have the old one's room
  capturing = 0;
  g_ws[0] = DevWorkspace{};
  live.clear(), used = 0;
  CHECK(internal_workspace(100, 500, nullptr, &a) == PA_OK);
  CHECK(internal_workspace(100, 800, nullptr, &b) == PA_OK && live.size() == 1 && zero(b));
  // a graph holds an address: it outlives larger ones
  capturing = 1;
  CHECK(internal_workspace(100, 800, nullptr, &a) == PA_OK && a.ptr == b.ptr);
  capturing = 0;
  most = 10000;
  CHECK(internal_workspace(0, 2000, nullptr, &c, true) == PA_OK && c.ptr != a.ptr && live.count(a.ptr));
  printf("ok\n");
  return 0;
}
"""


def test_growth_and_refusal(tmp_path):
    (tmp_path / "cuda_runtime.h").write_text(RUNTIME)
    (tmp_path / "main.cpp").write_text(MAIN)
    exe = str(tmp_path / "main")
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-pthread", "-I", str(tmp_path), "-I",
                           os.path.join(ROOT, "paged_decode_attention_reshape_gb300", "csrc"), str(tmp_path / "main.cpp"), "-o", exe])
    r = subprocess.run([exe], capture_output=True, text=True)
    assert (r.returncode, r.stdout) == (0, "ok\n")
