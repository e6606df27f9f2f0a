// pa_fp4_quant.cuh -- a group of 16 elements to its E2M1 codes and E4M3 scale (the definition is in
// pa_fp4.cu), shared by the 4-bit cache writes (pa_fp4.cu, pa_rotary.cuh).
#pragma once

#include "pa_fp4.cuh"
#include "pa_quant.cuh"

namespace pa {

// 16 elements of a row as its bytes (32 of a 16-bit row, 64 of an fp32 one).  wide: 32-byte aligned.
template <int DT>
__device__ __forceinline__ void load_group(const char *src, bool wide, uint32_t (&w)[4 * In<DT>::bytes]) {
#pragma unroll
  for (int i = 0; i < In<DT>::bytes / 2; ++i) {
    uint32_t v[8];
    if (wide) {
      ld32_once(src + 32 * i, v);
    } else {
      const uint4 a = ld_once(src + 32 * i), b = ld_once(src + 32 * i + 16);
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
      v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) w[8 * i + j] = v[j];
  }
}
template <int DT>
__device__ __forceinline__ void group_values(const uint32_t (&w)[4 * In<DT>::bytes], float (&x)[16]) {
  if constexpr (DT == PA_F32) {
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 f = DT == PA_BF16 ? unpack_bf16(w[i]) : unpack_f16(w[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}

__device__ __forceinline__ float with_sign(float mag, float sign_of) {
  return __uint_as_float((__float_as_uint(mag) & 0x7fffffffu) | (__float_as_uint(sign_of) & 0x80000000u));
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Two E2M1 codes in a byte: low half = a.
__device__ __forceinline__ uint32_t e2m1x8(const float (&q)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 x0, x1, x2, x3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 x0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 x1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 x2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 x3, %8, %7;\n\t"
      "mov.b32 %0, {x0, x1, x2, x3};\n\t}"
      : "=r"(r)
      : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
  return r;
}

// The group's codes and scale, by the definition's own quotients (every one an IEEE division): for a
// group with a NaN, an infinity or a value above 2^80, and for head scales s outside [2^-40, 2^40].
static __device__ __noinline__ uint3 quantise_exact(const float (&x)[16], float s) {
  float y[16], top = 0.f;
  bool bad = false;
#pragma unroll 1
  for (int i = 0; i < 16; ++i) {
    y[i] = __fdiv_rn(x[i], s);
    bad |= y[i] != y[i];
    top = fmaxf(top, fabsf(y[i]));
  }
  if (bad) return make_uint3(0u, 0u, 0x7Fu);
  const uint32_t scale =
      static_cast<uint32_t>(__nv_cvt_float_to_fp8(fmaxf(__fdiv_rn(top, 6.f), 0x1p-9f), __NV_SATFINITE, __NV_E4M3));
  const float sg = unpack_f16(e4m3x2_to_f16x2(scale)).x;
  const uint32_t flip = s < 0.f ? 0x80000000u : 0u;  // (a quotient that is zero has lost its sign for a zero x)
  uint32_t w[2] = {0u, 0u};
#pragma unroll 1
  for (int i = 0; i < 16; i += 8) {
    float q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      q[j] = with_sign(fabsf(__fdiv_rn(y[i + j], sg)), __uint_as_float(__float_as_uint(x[i + j]) ^ flip));
    w[i >> 3] = e2m1x8(q);
  }
  return make_uint3(w[0], w[1], scale);
}

__device__ __forceinline__ uint3 settle(const float (&x)[16], float s) {
  float y[16];  // (a copy: the call takes an address, and x stays in registers)
#pragma unroll
  for (int i = 0; i < 16; ++i) y[i] = x[i];
  return quantise_exact(y, s);
}

// The same in registers, the quotients by Markstein's steps (Divisor), for top = max |x| <= 2^80 and |s|
// in [2^-40, 2^40]: a group whose border cases the brackets below leave open.  Where a step leaves the
// range in which it is exact, the code is the same all the same: a |y| above 2^80 saturates, one below
// 2^-80 is far under the smallest code's border.
__device__ __forceinline__ uint3 quantise_divided(const float (&x)[16], float s, float top) {
  const Divisor by_s = make_divisor(fabsf(s));
  const Divisor by_six{6.f, 1.f / 6.f, true};
  const float y_top = by_s.div2_fast(top, top).x;  // (rounding keeps the order: the largest |y|)
  const uint32_t scale = static_cast<uint32_t>(
      __nv_cvt_float_to_fp8(fmaxf(by_six.div2_fast(y_top, y_top).x, 0x1p-9f), __NV_SATFINITE, __NV_E4M3));
  const Divisor by_sg = make_divisor(unpack_f16(e4m3x2_to_f16x2(scale)).x);
  const uint32_t flip = s < 0.f ? 0x80000000u : 0u;
  float q[16];
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    const float2 y = by_s.div2_fast(fabsf(x[i]), fabsf(x[i + 1]));
    const float2 r = by_sg.div2_fast(y.x, y.y);
    q[i] = with_sign(r.x, __uint_as_float(__float_as_uint(x[i]) ^ flip));
    q[i + 1] = with_sign(r.y, __uint_as_float(__float_as_uint(x[i + 1]) ^ flip));
  }
  return make_uint3(e2m1x8(reinterpret_cast<float(&)[8]>(q[0])), e2m1x8(reinterpret_cast<float(&)[8]>(q[8])), scale);
}

__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float b) {
  uint64_t x, y;
  float2 o;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %1};" : "=l"(y) : "f"(b));
  asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(x) : "l"(y));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(o.x), "=f"(o.y) : "l"(x));
  return o;
}

// The same without a division.  Rounding never falls as its argument grows, so if a value a little
// below the quotient and one a little above it have the same code, the quotient has it too.  With
// r = (1 / s) (1 / sg) from two approximate reciprocals (2^-23 each) and three rounded products
// (2^-24 each), x r is within 2^-21.1 of x / (s sg), and the definition's twice rounded quotient
// within 2^-23: the codes of x r (1 - kNear) and x r (1 + kNear) enclose its code and, where they
// agree, are it; the group's scale is settled alike from its largest |x|.  Products keep the signs
// of zeros.  What stays open is divided (quantise_divided): of normal bf16 rows one group in four at a
// power of two, one in five at 0.75, so nearly every warp, but few at a scale of many bits (8192 rows of
// 8 x 128 in states beyond L2: 16.8 us at 0.5 and 0.75 against 11.8; 170 when those groups went through
// quantise_exact, and 92 against 11.4 with no scale, below).
// UNIT16: a 16-bit x and s = 1, where borders are hit often (the group's scale for 8 of the 128 bf16
// significands of its largest element): x has at most 11 significant bits, a border of the code 3, of
// the scale 5, 6 two and sg 4, so x / sg and x / 6 are a border or 2^-18 of themselves away from it, and
// a quotient corrected once (exact where the true one is an fp32 number, else within 2^-22) decides.
constexpr float kNear = 0x1p-20f;
template <bool UNIT16>
__device__ __forceinline__ uint3 quantise_group(const float (&x)[16], float s, float rs) {
  float top = fabsf(x[0]);
#pragma unroll
  for (int i = 1; i < 16; ++i) top = max_nan(top, fabsf(x[i]));
  // (false for a NaN; the bounds keep every product below from overflow, and a head scale whose
  // reciprocal is not a plain number out of here)
  if (!(top <= 0x1p80f && fabsf(rs) <= 0x1p40f && fabsf(rs) >= 0x1p-40f)) return settle(x, s);
  float q[16];
  uint2 codes;
  uint32_t scale;
  if constexpr (UNIT16) {
    const Divisor by_six{6.f, 1.f / 6.f, true};
    scale = static_cast<uint32_t>(
        __nv_cvt_float_to_fp8(fmaxf(by_six.div2_near(top, top).x, 0x1p-9f), __NV_SATFINITE, __NV_E4M3));
    const float sg = unpack_f16(e4m3x2_to_f16x2(scale)).x;
    const Divisor d{sg, rcp_approx(sg), true};
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      const float2 r = d.div2_near(x[i], x[i + 1]);  // (drops the sign of a zero)
      q[i] = with_sign(r.x, x[i]);
      q[i + 1] = with_sign(r.y, x[i + 1]);
    }
    codes.x = e2m1x8(reinterpret_cast<float(&)[8]>(q[0]));
    codes.y = e2m1x8(reinterpret_cast<float(&)[8]>(q[8]));
  } else {
    const float want = top * fabsf(rs) * (1.f / 6.f);
    const uint32_t two = static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(
        make_float2(fmaxf(want * (1.f - kNear), 0x1p-9f), fmaxf(want * (1.f + kNear), 0x1p-9f)), __NV_SATFINITE,
        __NV_E4M3));
    scale = two & 0xffu;
    const float r = rs * rcp_approx(unpack_f16(e4m3x2_to_f16x2(scale)).x);
    uint2 above;
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      const float2 v = mul2(make_float2(x[i], x[i + 1]), r * (1.f - kNear));
      q[i] = v.x;
      q[i + 1] = v.y;
    }
    codes.x = e2m1x8(reinterpret_cast<float(&)[8]>(q[0]));
    codes.y = e2m1x8(reinterpret_cast<float(&)[8]>(q[8]));
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      const float2 v = mul2(make_float2(x[i], x[i + 1]), r * (1.f + kNear));
      q[i] = v.x;
      q[i + 1] = v.y;
    }
    above.x = e2m1x8(reinterpret_cast<float(&)[8]>(q[0]));
    above.y = e2m1x8(reinterpret_cast<float(&)[8]>(q[8]));
    if (scale != two >> 8 || codes.x != above.x || codes.y != above.y) return quantise_divided(x, s, top);
  }
  return make_uint3(codes.x, codes.y, scale);
}

}  // namespace pa
