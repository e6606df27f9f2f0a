// pa_validate.h -- descriptor checks shared by the entry points (host code).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <utility>

#include "pa_internal.h"

namespace pa {

inline int elem_bytes(int dt) {
  switch (dt) {
    case PA_F32: case PA_I32: return 4;
    case PA_BF16: case PA_F16: return 2;
    case PA_FP8_E4M3: case PA_FP4_E2M1: return 1;  // (an E2M1 cache is given as its page bytes)
    case PA_I64: return 8;
    default: return 0;
  }
}

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Whether a tensor's elements lie on multiples of their size.
inline bool on_elements(const pa_tensor *t) {
  return reinterpret_cast<uintptr_t>(t->data) % static_cast<uintptr_t>(elem_bytes(t->dtype)) == 0;
}

// Whether rows of `len` elements of an output [n0, n1, ...] share memory (a broadcast one's do): written
// side by side, and read before they are added to, they would hold whichever came last.
inline bool rows_overlap(const pa_tensor *t, int64_t len) {
  int64_t n = t->shape[0], a = t->stride[0], m = t->shape[1], b = t->stride[1];  // a <= b
  if (a > b) {
    std::swap(n, m);
    std::swap(a, b);
  }
  if (n < 1 || m < 1 || len < 1) return false;
  return (n > 1 && a < len) || (m > 1 && b < (n > 1 ? (n - 1) * a : 0) + len);
}

// Rows [T, H, D] whose every 32-byte piece is 32-byte aligned (element size eb).
inline bool rows_aligned32(const pa_tensor *t, int eb) {
  return (reinterpret_cast<uintptr_t>(t->data) & 31u) == 0 && (t->stride[0] * eb) % 32 == 0 && (t->stride[1] * eb) % 32 == 0;
}

// Descriptor sanity: non-null, rank, element type, positive extents.
inline int check_desc(const pa_tensor *t, int ndim) {
  if (!t || t->ndim != ndim) return PA_ERR_INVALID_ARG;
  for (int i = 0; i < ndim; ++i)
    if (t->shape[i] < 0 || t->stride[i] < 0) return PA_ERR_INVALID_ARG;
  if (elem_bytes(t->dtype) == 0) return PA_ERR_UNSUPPORTED_DTYPE;
  return PA_OK;
}

inline int device_sm_count() {
  static int cache[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev >= 0 && dev < 64 && cache[dev]) return cache[dev];
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (dev >= 0 && dev < 64) cache[dev] = n;
  return n;
}

// The cache pair of a call: [NB, Hkv, 16, D], or for a 4-bit cache [NB, Hkv, 9 D] page bytes.
inline int validate_cache_pair(const pa_tensor *kc, const pa_tensor *vc, int *NB, int *Hkv, int *D) {
  int r;
  const bool fp4 = kc && kc->dtype == PA_FP4_E2M1;
  const int rank = fp4 ? 3 : 4;
  if ((r = check_desc(kc, rank)) || (r = check_desc(vc, rank))) return r;
  for (int i = 0; i < rank; ++i)
    if (kc->shape[i] != vc->shape[i]) return PA_ERR_INVALID_ARG;
  if (kc->dtype != vc->dtype) return PA_ERR_INVALID_ARG;
  if (fp4) {
    if (kc->shape[2] != 9 * 64 && kc->shape[2] != 9 * 128 && kc->shape[2] != 9 * 256) return PA_ERR_UNSUPPORTED_SHAPE;
  } else if (kc->shape[2] != kBlock) {
    return PA_ERR_UNSUPPORTED_SHAPE;
  }
  if (kc->stride[rank - 1] != 1 || vc->stride[rank - 1] != 1) return PA_ERR_INVALID_ARG;
  if (!kc->data || !vc->data) return PA_ERR_INVALID_ARG;
  const int eb = elem_bytes(kc->dtype);
  if (!aligned16(kc->data) || !aligned16(vc->data)) return PA_ERR_ALIGNMENT;
  for (int i = 0; i < rank - 1; ++i)
    if ((kc->stride[i] * eb) % 16 || (vc->stride[i] * eb) % 16) return PA_ERR_ALIGNMENT;
  if (kc->shape[0] > INT32_MAX || kc->shape[1] > 65535) return PA_ERR_UNSUPPORTED_SHAPE;
  *NB = static_cast<int>(kc->shape[0]);
  *Hkv = static_cast<int>(kc->shape[1]);
  *D = static_cast<int>(fp4 ? kc->shape[2] / 9 : kc->shape[3]);
  return PA_OK;
}

}  // namespace pa
