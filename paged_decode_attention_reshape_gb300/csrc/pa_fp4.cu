// pa_fp4.cu -- the 4-bit cache write, and the read back of rows of any cache.
//
// Write.  For each group of 16 elements x of a (token, kv head) row, with the head's scale s
// (every operation one IEEE fp32 operation, rounded to nearest):
//   y = x / s,  sg = E4M3(max(max |y| / 6, 2^-9)),  code = E2M1(y / sg)
// E4M3 and E2M1 rounding to nearest even, saturating.  6 is the largest E2M1 value, so the
// group's largest element uses the top of the code's range; 2^-9 is the smallest E4M3 value
// above zero, so sg is never zero and the quotient always exists (a group of zeros gets codes
// of zero).  A group that holds a NaN gets scale NaN (0x7F) and codes 0.
//
// Work split: one thread per group, K and V together (16 elements are 32 bytes of a 16-bit row, one
// 32-byte load where it is aligned, and 8 bytes of codes).  Bound by the bytes (2 read and 9/16
// written an element) and by the arithmetic when T is large, by the launch when it is small, so the
// quotients are bracketed instead of taken (quantise_group): two products and two conversions an
// element, and the definition's divisions only for a group that the bracket does not settle.
//
// Read back.  value = code * sg * s: code * sg has at most 6 significant bits (exact in f16),
// the product with s and the conversion to the output's type round once each.  The same
// kernel copies or widens rows of the other caches.
#include "pa_fp4.cuh"
#include "pa_quant.cuh"

namespace pa {
namespace {

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
__device__ __noinline__ uint3 quantise_exact(const float (&x)[16], float s) {
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

// A product of an index and a stride, in one widening multiply when both are below 2^31 (I32).
template <bool I32>
__device__ __forceinline__ int64_t times(int64_t i, int64_t stride) {
  if constexpr (I32) return static_cast<int64_t>(static_cast<uint64_t>(static_cast<uint32_t>(i)) * static_cast<uint32_t>(stride));
  else return i * stride;
}

// Blocks of (groups of a row, heads, tokens) threads: no thread divides to find its place.
template <int DT, bool I32>
__global__ void __launch_bounds__(256) write_fp4_kernel(const Fp4WriteParams p) {
  // the decode that usually follows waits for this grid's completion before its first read
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int IB = In<DT>::bytes;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.z + threadIdx.z;
  if (t >= p.T) return;
  const int64_t slot = __ldg(p.slot_mapping + t);  // (not waited for before the rows are asked for)
  const char *key = static_cast<const char *>(p.key) + times<I32>(t, p.key_ts), *value = static_cast<const char *>(p.value) + times<I32>(t, p.val_ts);
#pragma unroll 1  // (one turn for most shapes)
  for (int h = threadIdx.y; h < p.Hkv; h += blockDim.y) {
#pragma unroll 1
    for (int gi = threadIdx.x; gi < p.D >> 4; gi += blockDim.x) {
      uint32_t wk[4 * IB], wv[4 * IB];
      load_group<DT>(key + times<I32>(h, p.key_hs) + gi * (16 * IB), p.wide, wk);
      load_group<DT>(value + times<I32>(h, p.val_hs) + gi * (16 * IB), p.wide, wv);
      const float ks = p.k_scale ? __ldg(p.k_scale + h * p.scale_stride) : 1.f;
      const float vs = p.v_scale ? __ldg(p.v_scale + h * p.scale_stride) : 1.f;
      if (slot < 0) return;  // padding row: no destination
      if (slot >= p.num_slots) {
        if (p.err && threadIdx.x == 0 && threadIdx.y == 0) atomicOr(p.err, kErrSlot);
        return;
      }
      const int64_t blk = slot >> 4;
      const int off = static_cast<int>(slot) & (kBlock - 1);
      const int co = fp4_code_off(p.D, off, gi * 8), so = fp4_scale_off(p.D, off, gi);
      auto store = [&](char *page, const uint3 &c) {
        *reinterpret_cast<uint2 *>(page + co) = make_uint2(c.x, c.y);
        *reinterpret_cast<uint8_t *>(page + so) = static_cast<uint8_t>(c.z);
      };
      auto quantised = [&](const uint32_t (&w)[4 * IB], float s) {
        float x[16];
        group_values<DT>(w, x);
        if (DT != PA_F32 && s == 1.f) return quantise_group<true>(x, 1.f, 1.f);
        return quantise_group<false>(x, s, rcp_approx(s));
      };
      store(p.k_cache + times<I32>(blk, p.kc_s0) + times<I32>(h, p.kc_s1), quantised(wk, ks));
      store(p.v_cache + times<I32>(blk, p.vc_s0) + times<I32>(h, p.vc_s1), quantised(wv, vs));
    }
  }
}

// ------------------------------------------------------------------- read back

// One group of 16 elements of a cache row as it lies there (OB: bytes of an element of a 16- or
// 32-bit cache), and as fp32 values, its head's scale times theirs.
template <int CT>
struct Cached {
  static constexpr int N = CT == PA_FP4_E2M1 || CT == PA_FP8_E4M3 ? 1 : In<CT == PA_FP4_E2M1 || CT == PA_FP8_E4M3 ? PA_F32 : CT>::bytes;
  uint4 w[N];  // (4-bit: x, y the codes, z the scale)
  // src: the row's start (4-bit: its page's)
  __device__ __forceinline__ void load(const char *src, int D, int off, int gi) {
    if constexpr (CT == PA_FP4_E2M1) {
      const char *page = src;
      const uint2 v = *reinterpret_cast<const uint2 *>(page + fp4_code_off(D, off, gi * 8));
      const uint32_t s = *reinterpret_cast<const uint8_t *>(page + fp4_scale_off(D, off, gi));
      w[0] = make_uint4(v.x, v.y, s, 0u);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] = *reinterpret_cast<const uint4 *>(src + gi * (16 * N) + 16 * i);
    }
  }
  __device__ __forceinline__ void values(float scale, float (&x)[16]) const {
    if constexpr (CT == PA_FP4_E2M1) {
      const uint32_t sg = e4m3x2_to_f16x2(w[0].z | (w[0].z << 8));
      uint32_t v[8];
      e2m1x8_to_f16x2x4(w[0].x, v[0], v[1], v[2], v[3]);
      e2m1x8_to_f16x2x4(w[0].y, v[4], v[5], v[6], v[7]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 f = mul2(unpack_f16(mul_f16x2(v[i], sg)), scale);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
      }
    } else if constexpr (CT == PA_FP8_E4M3) {
      const uint32_t ww[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t lo, hi;
        e4m3x4_to_f16x2x2(ww[i], lo, hi);
        const float2 a = mul2(unpack_f16(lo), scale), b = mul2(unpack_f16(hi), scale);
        x[4 * i] = a.x;
        x[4 * i + 1] = a.y;
        x[4 * i + 2] = b.x;
        x[4 * i + 3] = b.y;
      }
    }
  }
};

// N packs of 16 bytes (2 of a 16-bit group, 4 of an fp32 one).  wide: 32-byte aligned.
template <int N>
__device__ __forceinline__ void store_packs(char *dst, bool wide, const uint32_t (&w)[4 * N]) {
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    if (wide) {
      const uint32_t v[8] = {w[8 * i],     w[8 * i + 1], w[8 * i + 2], w[8 * i + 3],
                             w[8 * i + 4], w[8 * i + 5], w[8 * i + 6], w[8 * i + 7]};
      st32(dst + 32 * i, v);
    } else {
      *reinterpret_cast<uint4 *>(dst + 32 * i) = make_uint4(w[8 * i], w[8 * i + 1], w[8 * i + 2], w[8 * i + 3]);
      *reinterpret_cast<uint4 *>(dst + 32 * i + 16) = make_uint4(w[8 * i + 4], w[8 * i + 5], w[8 * i + 6], w[8 * i + 7]);
    }
  }
}
template <int OT>
__device__ __forceinline__ void store_group(char *dst, bool wide, const float (&x)[16]) {
  constexpr int N = In<OT>::bytes;
  uint32_t w[4 * N];
  if constexpr (OT == PA_F32) {
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(x[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = OT == PA_BF16 ? pack_bf16(x[2 * i], x[2 * i + 1]) : pack_f16(x[2 * i], x[2 * i + 1]);
  }
  store_packs<N>(dst, wide, w);
}

// CT == OT (a cache of the output's own type): bit copies.  A thread keeps its group of a row and
// goes over tokens, K and V, the next token's bytes and the slot after that in flight while it
// widens and stores: a slot and then a row are two trips to memory, and 9 bytes a group keep too
// little of it busy when every thread makes them once.  32768 rows of 8 x 128 at random slots: 34.6 us;
// 64 bytes of codes and 8 of scales a row are two bursts of memory, 201 MB in all, 30 us at its rate.
constexpr int kGatherCtas = 3;  // per SM (4 or 5: 39.1, 37.6 us against 34.6)
template <int CT, int OT, bool I32>
__global__ void __launch_bounds__(256, kGatherCtas) gather_kernel(const GatherParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int OB = In<OT>::bytes;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.z;
#pragma unroll 1  // (one turn for most shapes)
  for (int h = threadIdx.y; h < p.Hkv; h += blockDim.y) {
#pragma unroll 1
    for (int gi = threadIdx.x; gi < p.D >> 4; gi += blockDim.x) {
      const char *const kc = p.k_cache + times<I32>(h, p.kc_s1), *const vc = p.v_cache + times<I32>(h, p.vc_s1);
      char *const key = p.key + times<I32>(h, p.key_hs) + gi * (16 * OB);
      char *const value = p.value + times<I32>(h, p.val_hs) + gi * (16 * OB);
      float ks = 1.f, vs = 1.f;
      if constexpr (CT != OT) {
        if (p.k_scale) ks = __ldg(p.k_scale + h * p.scale_stride);
        if (p.v_scale) vs = __ldg(p.v_scale + h * p.scale_stride);
      }
      auto slot_of = [&](int64_t t) {  // -1: nothing to read (the output row keeps what it holds)
        if (t >= p.T) return static_cast<int64_t>(-1);
        const int64_t slot = __ldg(p.slot_mapping + t);
        if (slot < p.num_slots) return slot;
        if (p.err && h == 0 && gi == 0) atomicOr(p.err, kErrSlot);
        return static_cast<int64_t>(-1);
      };
      auto load = [&](int64_t slot, Cached<CT> &ck, Cached<CT> &cv) {
        if (slot < 0) return;
        const int64_t blk = slot >> 4;
        const int off = static_cast<int>(slot) & (kBlock - 1);
        ck.load(kc + times<I32>(blk, p.kc_s0) + times<I32>(off, p.kc_s2), p.D, off, gi);
        cv.load(vc + times<I32>(blk, p.vc_s0) + times<I32>(off, p.vc_s2), p.D, off, gi);
      };
      int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.z + threadIdx.z;
      int64_t slot = slot_of(t), slot1 = slot_of(t + stride);
      Cached<CT> ck, cv;
      load(slot, ck, cv);
      for (; t < p.T; t += stride) {
        const int64_t slot2 = slot_of(t + 2 * stride);
        Cached<CT> nk = ck, nv = cv;
        load(slot1, nk, nv);
        if (slot >= 0) {
          char *kd = key + times<I32>(t, p.key_ts), *vd = value + times<I32>(t, p.val_ts);
          if constexpr (CT == OT) {
            store_packs<OB>(kd, p.wide, reinterpret_cast<const uint32_t(&)[4 * OB]>(ck.w));
            store_packs<OB>(vd, p.wide, reinterpret_cast<const uint32_t(&)[4 * OB]>(cv.w));
          } else {
            float x[16];
            ck.values(ks, x);
            store_group<OT>(kd, p.wide, x);
            cv.values(vs, x);
            store_group<OT>(vd, p.wide, x);
          }
        }
        slot = slot1;
        slot1 = slot2;
        ck = nk;
        cv = nv;
      }
    }
  }
}

// Blocks of 256 threads or fewer: groups of a row, heads, tokens; at most `most` of them (0: any).
template <auto kern, typename P>
cudaError_t launch_tokens(const P &p, int64_t most, cudaStream_t st) {
  const int x = p.D / 16 < 32 ? p.D / 16 : 32, y = p.Hkv < 256 / x ? p.Hkv : 256 / x, fit = 256 / (x * y);
  const int z = fit < 64 ? fit : 64;
  int64_t blocks = (p.T + z - 1) / z;
  if (most > 0 && blocks > most) blocks = most;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  // the SM's shared / L1 split stays what the decode kernels ask for (see pa_write.cu)
  static std::atomic<uint64_t> done{0};
  cudaError_t e = once_per_device(done, [] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
  });
  if (e != cudaSuccess) return e;
  kern<<<static_cast<unsigned>(blocks), dim3(x, y, z), 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

template <int DT>
cudaError_t launch_write_one(const Fp4WriteParams &p, cudaStream_t st) {
  return p.i32 ? launch_tokens<write_fp4_kernel<DT, true>>(p, 0, st) : launch_tokens<write_fp4_kernel<DT, false>>(p, 0, st);
}

template <int CT, int OT>
cudaError_t launch_gather_one(const GatherParams &p, int sm_count, cudaStream_t st) {
  const int64_t wave = static_cast<int64_t>(sm_count) * kGatherCtas;
  return p.i32 ? launch_tokens<gather_kernel<CT, OT, true>>(p, wave, st)
               : launch_tokens<gather_kernel<CT, OT, false>>(p, wave, st);
}

cudaError_t launch_write_fp4(const Fp4WriteParams &p, int in_dtype, cudaStream_t st) {
  switch (in_dtype) {
    case PA_F32: return launch_write_one<PA_F32>(p, st);
    case PA_BF16: return launch_write_one<PA_BF16>(p, st);
    case PA_F16: return launch_write_one<PA_F16>(p, st);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_gather(const GatherParams &p, int cache_dtype, int out_dtype, int sm_count, cudaStream_t st) {
  auto by_out = [&](auto ct) -> cudaError_t {
    constexpr int CT = decltype(ct)::value;
    switch (out_dtype) {
      case PA_F32: return launch_gather_one<CT, PA_F32>(p, sm_count, st);
      case PA_BF16: return launch_gather_one<CT, PA_BF16>(p, sm_count, st);
      case PA_F16: return launch_gather_one<CT, PA_F16>(p, sm_count, st);
      default: return cudaErrorInvalidValue;
    }
  };
  if (cache_dtype == PA_FP4_E2M1) return by_out(std::integral_constant<int, PA_FP4_E2M1>{});
  if (cache_dtype == PA_FP8_E4M3) return by_out(std::integral_constant<int, PA_FP8_E4M3>{});
  if (cache_dtype != out_dtype) return cudaErrorInvalidValue;
  switch (out_dtype) {
    case PA_F32: return launch_gather_one<PA_F32, PA_F32>(p, sm_count, st);
    case PA_BF16: return launch_gather_one<PA_BF16, PA_BF16>(p, sm_count, st);
    case PA_F16: return launch_gather_one<PA_F16, PA_F16>(p, sm_count, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pa
