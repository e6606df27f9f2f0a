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
// Work split: one thread per group, K and V together (16 elements are 32 bytes of a 16-bit
// row, two 16-byte loads, and 8 bytes of codes), a CTA over whole tokens, adjacent threads
// on adjacent groups.  Bound by the bytes (2 read and 9/16 written an element) when T is
// large, by the launch when it is small.  Both quotients of an element are the correctly
// rounded ones of pa_quant.cuh (one reciprocal per scale, packed fused steps), about 12
// operations an element.
//
// Read back.  value = code * sg * s: code * sg has at most 6 significant bits (exact in f16),
// the product with s and the conversion to the output's type round once each.  The same
// kernel copies or widens rows of the other caches.
#include "pa_fp4.cuh"
#include "pa_quant.cuh"

namespace pa {
namespace {

// Element i of the group: x[i] as fp32.
template <int DT>
__device__ __forceinline__ void load_group(const char *src, float (&x)[16]) {
  if constexpr (DT == PA_F32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 v = ld_once(src + 16 * i);
      x[4 * i] = __uint_as_float(v.x);
      x[4 * i + 1] = __uint_as_float(v.y);
      x[4 * i + 2] = __uint_as_float(v.z);
      x[4 * i + 3] = __uint_as_float(v.w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float h[8];
      unpack8<DT>(ld_once(src + 16 * i), h);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[8 * i + j] = h[j];
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

// The group's codes and scale.  `dv` divides by the head's scale; `unit` when that is 1.
// Magnitudes are clamped to 2^80 and signs put back at the end, so the fused quotient steps
// hold for every input (see store_fp8 in pa_write.cu): a larger magnitude saturates all the
// same, a magnitude too small for exact steps rounds to code 0 under any scale >= 2^-9.
__device__ __forceinline__ void quantise_group(float (&x)[16], const Divisor &dv, bool unit, uint2 &codes,
                                               uint32_t &scale) {
  float y[16];
  if (unit) {
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = clamp_mag(x[i]);
  } else if (dv.fast) {
    const Divisor da{fabsf(dv.s), fabsf(dv.y), true};
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      const float2 r = da.div2_fast(clamp_mag(x[i]), clamp_mag(x[i + 1]));
      y[i] = r.x;
      y[i + 1] = r.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = clamp_mag(__fdiv_rn(x[i], fabsf(dv.s)));
  }
  float top = y[0];
#pragma unroll
  for (int i = 1; i < 16; ++i) top = max_nan(top, y[i]);
  const float want = max_nan(__fdiv_rn(top, 6.f), 0x1p-9f);
  scale = static_cast<uint32_t>(__nv_cvt_float_to_fp8(want, __NV_SATFINITE, __NV_E4M3));
  if (top != top) {
    codes = make_uint2(0u, 0u);
    return;
  }
  const uint32_t wide = e4m3x2_to_f16x2(scale);
  const Divisor dg = make_divisor(unpack_f16(wide).x);  // in [2^-9, 448]
  const float flip = dv.s < 0.f ? -1.f : 1.f;  // (the scale's sign: unit and zero scales have none)
  float q[16];
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    const float2 r = dg.div2_fast(y[i], y[i + 1]);
    q[i] = with_sign(r.x, x[i] * flip);
    q[i + 1] = with_sign(r.y, x[i + 1] * flip);
  }
  codes.x = e2m1x8(reinterpret_cast<float(&)[8]>(q[0]));
  codes.y = e2m1x8(reinterpret_cast<float(&)[8]>(q[8]));
}

template <int DT>
__global__ void __launch_bounds__(256) write_fp4_kernel(const Fp4WriteParams p) {
  // the decode that usually follows waits for this grid's completion before its first read
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int IB = In<DT>::bytes;
  const int per_row = p.D >> 4;           // groups per (token, head) row
  const int per_tok = p.Hkv * per_row;    // groups per token
  const int width = min(per_tok, 256);
  const int rows = 256 / width;
  const int tl = threadIdx.x / width;
  const int j0 = threadIdx.x - tl * width;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * rows + tl;
  if (tl >= rows || t >= p.T) return;
  const int64_t slot = __ldg(p.slot_mapping + t);
  if (slot < 0) return;  // padding row: no destination
  if (slot >= p.num_slots) {
    if (p.err && j0 == 0) atomicOr(p.err, kErrSlot);
    return;
  }
  const int64_t blk = slot / kBlock;
  const int off = static_cast<int>(slot % kBlock);
  for (int j = j0; j < per_tok; j += 256) {  // one turn unless a token is wider than the block
    const int h = j / per_row, gi = j - h * per_row;
    const float ks = p.k_scale ? __ldg(p.k_scale + h * p.scale_stride) : 1.f;
    const float vs = p.v_scale ? __ldg(p.v_scale + h * p.scale_stride) : 1.f;
    float xk[16], xv[16];
    load_group<DT>(static_cast<const char *>(p.key) + (t * p.key_ts + h * p.key_hs + gi * 16) * IB, xk);
    load_group<DT>(static_cast<const char *>(p.value) + (t * p.val_ts + h * p.val_hs + gi * 16) * IB, xv);
    const int co = fp4_code_off(p.D, off, gi * 8), so = fp4_scale_off(p.D, off, gi);
    uint2 codes;
    uint32_t sc;
    quantise_group(xk, make_divisor(ks), ks == 1.f, codes, sc);
    char *page = p.k_cache + blk * p.kc_s0 + h * p.kc_s1;
    *reinterpret_cast<uint2 *>(page + co) = codes;
    *reinterpret_cast<uint8_t *>(page + so) = static_cast<uint8_t>(sc);
    quantise_group(xv, make_divisor(vs), vs == 1.f, codes, sc);
    page = p.v_cache + blk * p.vc_s0 + h * p.vc_s1;
    *reinterpret_cast<uint2 *>(page + co) = codes;
    *reinterpret_cast<uint8_t *>(page + so) = static_cast<uint8_t>(sc);
  }
}

// ------------------------------------------------------------------- read back

// One group of 16 elements of a cache row -> fp32 values (without the head's scale).
template <int CT>
__device__ __forceinline__ void load_cached(const char *c, int64_t s0, int64_t s1, int64_t s2, int D, int64_t blk,
                                            int off, int h, int gi, float (&x)[16]) {
  if constexpr (CT == PA_FP4_E2M1) {
    const char *page = c + blk * s0 + h * s1;
    const uint2 w = *reinterpret_cast<const uint2 *>(page + fp4_code_off(D, off, gi * 8));
    const uint32_t s = *reinterpret_cast<const uint8_t *>(page + fp4_scale_off(D, off, gi));
    const uint32_t sg = e4m3x2_to_f16x2(s | (s << 8));
    uint32_t v[8];
    e2m1x8_to_f16x2x4(w.x, v[0], v[1], v[2], v[3]);
    e2m1x8_to_f16x2x4(w.y, v[4], v[5], v[6], v[7]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 f = unpack_f16(mul_f16x2(v[i], sg));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  } else if constexpr (CT == PA_FP8_E4M3) {
    const uint4 w = *reinterpret_cast<const uint4 *>(c + blk * s0 + h * s1 + off * s2 + gi * 16);
    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t lo, hi;
      e4m3x4_to_f16x2x2(ww[i], lo, hi);
      const float2 a = unpack_f16(lo), b = unpack_f16(hi);
      x[4 * i] = a.x;
      x[4 * i + 1] = a.y;
      x[4 * i + 2] = b.x;
      x[4 * i + 3] = b.y;
    }
  }
}

template <int OT>
__device__ __forceinline__ void store_group(char *dst, const float (&x)[16]) {
  if constexpr (OT == PA_F32) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<float4 *>(dst + 16 * i) = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
  } else {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = OT == PA_BF16 ? pack_bf16(x[2 * i], x[2 * i + 1]) : pack_f16(x[2 * i], x[2 * i + 1]);
    *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4 *>(dst + 16) = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// CT == OT (a cache of the output's own type): bit copies.
template <int CT, int OT>
__global__ void __launch_bounds__(256) gather_kernel(const GatherParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int OB = In<OT>::bytes;
  const int per_row = p.D >> 4, per_tok = p.Hkv * per_row;
  const int width = min(per_tok, 256);
  const int rows = 256 / width;
  const int tl = threadIdx.x / width;
  const int j0 = threadIdx.x - tl * width;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * rows + tl;
  if (tl >= rows || t >= p.T) return;
  const int64_t slot = __ldg(p.slot_mapping + t);
  if (slot < 0) return;  // no source: the output row keeps what it holds
  if (slot >= p.num_slots) {
    if (p.err && j0 == 0) atomicOr(p.err, kErrSlot);
    return;
  }
  const int64_t blk = slot / kBlock;
  const int off = static_cast<int>(slot % kBlock);
  for (int j = j0; j < per_tok; j += 256) {
    const int h = j / per_row, gi = j - h * per_row;
    char *kd = p.key + (t * p.key_ts + h * p.key_hs + gi * 16) * OB;
    char *vd = p.value + (t * p.val_ts + h * p.val_hs + gi * 16) * OB;
    if constexpr (CT == OT) {
      const char *ks = p.k_cache + blk * p.kc_s0 + h * p.kc_s1 + off * p.kc_s2 + gi * 16 * OB;
      const char *vs = p.v_cache + blk * p.vc_s0 + h * p.vc_s1 + off * p.vc_s2 + gi * 16 * OB;
      uint4 a[OB], b[OB];  // 16 elements of OB bytes are OB packs of 16 bytes
#pragma unroll
      for (int i = 0; i < OB; ++i) {
        a[i] = *reinterpret_cast<const uint4 *>(ks + 16 * i);
        b[i] = *reinterpret_cast<const uint4 *>(vs + 16 * i);
      }
#pragma unroll
      for (int i = 0; i < OB; ++i) {
        *reinterpret_cast<uint4 *>(kd + 16 * i) = a[i];
        *reinterpret_cast<uint4 *>(vd + 16 * i) = b[i];
      }
    } else {
      const float ks = p.k_scale ? __ldg(p.k_scale + h * p.scale_stride) : 1.f;
      const float vs = p.v_scale ? __ldg(p.v_scale + h * p.scale_stride) : 1.f;
      float xk[16], xv[16];
      load_cached<CT>(p.k_cache, p.kc_s0, p.kc_s1, p.kc_s2, p.D, blk, off, h, gi, xk);
      load_cached<CT>(p.v_cache, p.vc_s0, p.vc_s1, p.vc_s2, p.D, blk, off, h, gi, xv);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        xk[i] *= ks;
        xv[i] *= vs;
      }
      store_group<OT>(kd, xk);
      store_group<OT>(vd, xv);
    }
  }
}

// Grid of a kernel whose CTAs take whole tokens of `per_tok` groups.
cudaError_t token_grid(int64_t T, int per_tok, unsigned *blocks) {
  const int rows = 256 / (per_tok < 256 ? per_tok : 256);
  const int64_t n = (T + rows - 1) / rows;
  if (n > INT32_MAX) return cudaErrorInvalidValue;
  *blocks = static_cast<unsigned>(n);
  return cudaSuccess;
}

template <typename P>
cudaError_t launch_tokens(void (*kern)(P), const P &p, cudaStream_t st) {
  unsigned blocks = 0;
  cudaError_t e = token_grid(p.T, p.Hkv * (p.D / 16), &blocks);
  if (e != cudaSuccess) return e;
  // the SM's shared / L1 split stays what the decode kernels ask for (see pa_write.cu)
  e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
  if (e != cudaSuccess) return e;
  kern<<<blocks, 256, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_write_fp4(const Fp4WriteParams &p, int in_dtype, cudaStream_t st) {
  switch (in_dtype) {
    case PA_F32: return launch_tokens(write_fp4_kernel<PA_F32>, p, st);
    case PA_BF16: return launch_tokens(write_fp4_kernel<PA_BF16>, p, st);
    case PA_F16: return launch_tokens(write_fp4_kernel<PA_F16>, p, st);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_gather(const GatherParams &p, int cache_dtype, int out_dtype, cudaStream_t st) {
  auto by_out = [&](auto ct) -> cudaError_t {
    constexpr int CT = decltype(ct)::value;
    switch (out_dtype) {
      case PA_F32: return launch_tokens(gather_kernel<CT, PA_F32>, p, st);
      case PA_BF16: return launch_tokens(gather_kernel<CT, PA_BF16>, p, st);
      case PA_F16: return launch_tokens(gather_kernel<CT, PA_F16>, p, st);
      default: return cudaErrorInvalidValue;
    }
  };
  if (cache_dtype == PA_FP4_E2M1) return by_out(std::integral_constant<int, PA_FP4_E2M1>{});
  if (cache_dtype == PA_FP8_E4M3) return by_out(std::integral_constant<int, PA_FP8_E4M3>{});
  if (cache_dtype != out_dtype) return cudaErrorInvalidValue;
  switch (out_dtype) {
    case PA_F32: return launch_tokens(gather_kernel<PA_F32, PA_F32>, p, st);
    case PA_BF16: return launch_tokens(gather_kernel<PA_BF16, PA_BF16>, p, st);
    case PA_F16: return launch_tokens(gather_kernel<PA_F16, PA_F16>, p, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pa
