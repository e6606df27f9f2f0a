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

// Whether a row of a tensor x [T, H, D] shares memory with a row of an output [T, H', D] (elements of eb bytes;
// the output's own rows do not overlap, see rows_overlap).  Views of one buffer, like heads side by side, do not.
// Equal strides take a few divisions; others a step for each run of x's rows, where the two spans meet at all.
inline bool rows_shared(const pa_tensor *x, const pa_tensor *out, int eb) {
  struct Axis {
    int64_t n, step;  // (step 0: one row, wherever it would go on)
  };
  struct Rows {
    Axis big, small;
    int64_t row;
    int64_t span() const { return (big.n - 1) * big.step + (small.n - 1) * small.step + row; }
  };
  const int64_t row = x->shape[2] * eb;
  if (!x->data || !out->data || row < 1) return false;
  auto rows = [&](const pa_tensor *t) {
    Rows r{{t->shape[0], t->stride[0] * eb}, {t->shape[1], t->stride[1] * eb}, row};
    for (Axis *a : {&r.big, &r.small})
      if (a->n <= 1) a->step = 0;
    if (r.big.step < r.small.step) std::swap(r.big, r.small);
    return r;
  };
  const Rows a = rows(x), b = rows(out);
  if (a.big.n < 1 || a.small.n < 1 || b.big.n < 1 || b.small.n < 1) return false;
  // where x's rows start, seen from the output's first
  const int64_t away = static_cast<int64_t>(reinterpret_cast<intptr_t>(x->data) - reinterpret_cast<intptr_t>(out->data));
  if (away >= b.span() || -away >= a.span()) return false;
  auto floor_div = [](int64_t p, int64_t q) { return p >= 0 ? p / q : -((-p + q - 1) / q); };

  const bool alike = x->stride[0] == out->stride[0] && x->stride[1] == out->stride[1];
  if (alike && !rows_overlap(x, x->shape[2])) {
    // Some difference of (t, h) must bring the starts within a row.  Neither tensor's rows overlap, so its heads of
    // a token (or tokens of a head) end within the larger step, and only the nearest multiples come into question.
    const bool heads_big = x->stride[1] > x->stride[0];
    const int big = heads_big ? 1 : 0, small = 1 - big;
    auto axis = [&](int i, int64_t from, auto &&each) {  // every difference i of that axis near `from` bytes
      const int64_t n = x->shape[i], m = out->shape[i], step = n > 1 || m > 1 ? x->stride[i] * eb : 0;
      const int64_t at = step > 0 ? floor_div(from, step) : 0;
      for (int64_t d = at - 1; d <= at + 2; ++d)  // d = (the output's index) - (x's)
        if (d < m && -d < n && (step > 0 || d == 0) && each(from - d * step)) return true;
      return false;
    };
    return axis(big, away, [&](int64_t left) {
      return axis(small, left, [&](int64_t apart) { return apart < row && -apart < row; });
    });
  }

  // The first row of the output that ends behind `at`: whether it starts before at + len.
  auto met = [&](int64_t at, int64_t len) {
    const int64_t block = (b.small.n - 1) * b.small.step + row;
    int64_t i = b.big.n > 1 ? floor_div(at - block, b.big.step) + 1 : at < block ? 0 : 1;
    if (i < 0) i = 0;
    if (i >= b.big.n) return false;
    const int64_t left = at - i * b.big.step;
    int64_t j = b.small.n > 1 ? floor_div(left - row, b.small.step) + 1 : 0;
    if (j < 0) j = 0;
    return i * b.big.step + j * b.small.step < at + len;
  };
  // x's rows in runs: those of the smaller step as one where they lie side by side (or are one and the same)
  const bool joined = a.small.step <= row;
  const int64_t run = joined ? (a.small.n - 1) * a.small.step + row : row;
  const int64_t bigs = a.big.step > 0 ? a.big.n : 1, smalls = joined ? 1 : a.small.n;
  for (int64_t i = 0; i < bigs; ++i)
    for (int64_t j = 0; j < smalls; ++j)
      if (met(away + i * a.big.step + j * a.small.step, run)) return true;
  return false;
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
