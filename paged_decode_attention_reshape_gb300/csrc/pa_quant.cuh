// pa_quant.cuh -- input rows as fp32 values and the quotients that quantisation takes, shared
// by the cache writes (pa_write.cu, pa_fp4.cu).
#pragma once

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

__device__ __forceinline__ uint4 ld_once(const void *p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// Element type codes for the template (match pa_dtype values).
template <int DT> struct In;
template <> struct In<PA_F32> { static constexpr int bytes = 4; };
template <> struct In<PA_BF16> { static constexpr int bytes = 2; };
template <> struct In<PA_F16> { static constexpr int bytes = 2; };

template <int DT>
__device__ __forceinline__ void unpack8(const uint4 &v, float (&x)[16 / In<DT>::bytes]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if constexpr (DT == PA_F32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = (DT == PA_BF16) ? unpack_bf16(w[i]) : unpack_f16(w[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}

// The correctly rounded quotient x / s for one divisor s shared by a whole tensor.
// With y = RN(1/s): q0 = RN(x y) is within 1.5 ulp of x/s; one correction
// q1 = RN(q0 + (x - q0 s) y) brings it within 1 ulp, and then (Markstein's theorem:
// y within half an ulp of 1/s, q1 within one ulp of x/s, residual x - q1 s exact by
// FMA) q2 = RN(q1 + (x - q1 s) y) is RN(x/s).  The theorem needs the operands and the
// residuals away from underflow and overflow, so zero, tiny, huge, infinite or NaN x
// (and divisors outside [2^-40, 2^40]) take the general IEEE division instead.
struct Divisor {
  float s, y;
  bool fast;
  __device__ __forceinline__ static bool in_range(float x) {
    const float ax = fabsf(x);
    return ax >= 0x1p-80f && ax <= 0x1p80f;  // false for zero, subnormals, inf, NaN
  }
  __device__ __forceinline__ float div(float x) const {
    if (fast && in_range(x)) {
      float q = __fmul_rn(x, y);
      float r = __fmaf_rn(-q, s, x);
      q = __fmaf_rn(r, y, q);
      r = __fmaf_rn(-q, s, x);
      return __fmaf_rn(r, y, q);
    }
    return __fdiv_rn(x, s);
  }
  // The same correctly rounded steps on two operands at once (packed fp32x2 operations,
  // each lane an IEEE round-to-nearest multiply / fused multiply-add); the caller has
  // checked fast and in_range for both.
  __device__ __forceinline__ float2 div2_fast(float a, float b) const {
    uint64_t x, sy, ns, q, r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a), "f"(b));
    asm("mov.b64 %0, {%1, %1};" : "=l"(sy) : "f"(y));
    asm("mov.b64 %0, {%1, %1};" : "=l"(ns) : "f"(-s));
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(q) : "l"(x), "l"(sy));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(q), "l"(ns), "l"(x));
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(q) : "l"(r), "l"(sy));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(q), "l"(ns), "l"(x));
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(q) : "l"(r), "l"(sy));
    float2 o;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(o.x), "=f"(o.y) : "l"(q));
    return o;
  }
  // The first correction only: within one ulp, and exact where the quotient is an fp32 number.
  __device__ __forceinline__ float2 div2_near(float a, float b) const {
    uint64_t x, sy, ns, q, r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a), "f"(b));
    asm("mov.b64 %0, {%1, %1};" : "=l"(sy) : "f"(y));
    asm("mov.b64 %0, {%1, %1};" : "=l"(ns) : "f"(-s));
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(q) : "l"(x), "l"(sy));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(q), "l"(ns), "l"(x));
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(q) : "l"(r), "l"(sy));
    float2 o;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(o.x), "=f"(o.y) : "l"(q));
    return o;
  }
};

__device__ __forceinline__ Divisor make_divisor(float s) {
  Divisor d;
  d.s = s;
  d.y = __frcp_rn(s);
  const float as = fabsf(s);
  d.fast = as >= 0x1p-40f && as <= 0x1p40f;
  return d;
}

// min(|x|, 2^80), NaN for a NaN x.
__device__ __forceinline__ float clamp_mag(float x) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(x)), "f"(0x1p80f));
  return r;
}

}  // namespace pa
