// pa_fp4.cuh -- the 4-bit (E2M1) cache page: where its bytes are, and how codes become f16.
//
// One page, of one (block, kv head), is 9 D contiguous bytes: 8 D bytes of E2M1 codes (16
// tokens x D / 2 bytes; byte b of a token holds elements 2b, low half, and 2b + 1), then D
// bytes of E4M3 scales (16 tokens x D / 16; scale j belongs to elements 16 j .. 16 j + 15).
// One contiguous run per page means one bulk copy per page and tensor, and a page size that
// is a multiple of 64 bytes for every head size.
//
// Code bytes lie in sections of 16 x min(64, D / 2) bytes (head size 256: two, elements
// 0..127 and 128..255), token by token, with bits 5 and 6 of the offset XORed by bits 7 and
// 8.  Both readers of a page in shared memory are then free of bank conflicts: the score
// fragments (lane (r, c) reads a run of token r, 16 bytes at D >= 128, 8 at D = 64) and the
// P.V fragments (lane (r, c) reads run r, 8 or 4 bytes, of token 2c + {0, 1, 8, 9}), which
// without the XOR would meet in one quarter of the banks (4-way).
#pragma once

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

__host__ __device__ constexpr int fp4_page_bytes(int D) { return 9 * D; }

// Offset in its page of code byte `b` of token `t`.
__host__ __device__ __forceinline__ int fp4_code_off(int D, int t, int b) {
  const int row = D >= 128 ? 64 : D / 2;
  const int lin = t * row + (b & 63);
  return (b >> 6) * 1024 + (lin ^ (((lin >> 7) & 3) << 5));
}
// Offset in its page of the scale of elements 16 j .. 16 j + 15 of token `t`.
__host__ __device__ __forceinline__ int fp4_scale_off(int D, int t, int j) { return 8 * D + t * (D / 16) + j; }

// Four code bytes (byte 0 first) -> four f16x2, each with its byte's low code in the low
// half.  Exact: every E2M1 value is an f16.
__device__ __forceinline__ void e2m1x8_to_f16x2x4(uint32_t eight_codes, uint32_t &a, uint32_t &b, uint32_t &c,
                                                  uint32_t &d) {
  asm("{\n\t.reg .b8 x0, x1, x2, x3;\n\t"
      "mov.b32 {x0, x1, x2, x3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, x0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, x1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, x2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, x3;\n\t}"
      : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
      : "r"(eight_codes));
}

// Two E4M3 codes (low byte first) -> f16x2.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two_codes) {
  uint32_t r;
  asm("{\n\t.reg .b16 l;\n\tcvt.u16.u32 l, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(two_codes));
  return r;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// What one lane reads of a page, from shared address `at` = the page's address plus the lane's own
// offset.  The XOR takes its bits from lin / 128, which is t / 2 at head sizes 128 and 256 (rows of
// 64 bytes) and t / 4 at 64 (rows of 32).  8 tokens on is 8 rows on at 128 and 256, for every
// lane; at 64 it is 256 bytes on with bit 6 flipped.  The token after an even one, a row on, has
// the row's bit (6 or 5) flipped.  A lane keeps those steps (`on8`, `odd`) as numbers.
//
// Lane (r, c) of a score fragment: elements 128 b + 32 c .. + 31 (head size 64: 16 c .. + 15)
// of tokens r and r + 8.
template <int D>
struct Fp4Rows {
  static constexpr int ROWB = D >= 128 ? 64 : 32;   // code bytes of a token in a section
  static constexpr int NW = D >= 128 ? 4 : 2;       // words of eight codes
  static constexpr int NS = NW / 2;                 // scales
  static __device__ __forceinline__ int code_lane(int r, int c) { return fp4_code_off(D, r, 4 * NW * c); }
  static __device__ __forceinline__ int scale_lane(int r, int c) { return fp4_scale_off(D, r, NS * c); }
  static __device__ __forceinline__ int on8(int code_lane) {
    return D >= 128 ? 8 * ROWB : 256 + ((code_lane & 64) ? -64 : 64);
  }
  // at: token r's, or on8 behind it token r + 8's
  static __device__ __forceinline__ void codes(uint32_t at, int b, uint32_t (&w)[NW]) {
    const uint32_t a = at + b * 1024;
    if constexpr (D >= 128) {
      const uint4 v = lds128(a);
      w[0] = v.x;
      w[1] = v.y;
      w[2] = v.z;
      w[3] = v.w;
    } else {
      const uint2 v = lds64(a);
      w[0] = v.x;
      w[1] = v.y;
    }
  }
  // the scales of those elements, each in both halves of an f16x2
  static __device__ __forceinline__ void scales(uint32_t at, bool second, int b, uint32_t (&s)[NS]) {
    const uint32_t a = at + (second ? 8 * (D / 16) : 0) + b * 8;
    if constexpr (D >= 128) {
      const uint32_t two = e4m3x2_to_f16x2(lds_u16(a));
      s[0] = __byte_perm(two, two, 0x1010);
      s[1] = __byte_perm(two, two, 0x3232);
    } else {
      const uint32_t one = lds_u8(a);
      s[0] = e4m3x2_to_f16x2(one | (one << 8));
    }
  }
};

// Lane (r, c) of a P.V fragment: run r, elements 128 b + 16 r .. + 15 (head size 64: 8 r .. + 7), of
// tokens 2c + {0, 1, 8, 9}.
template <int D>
struct Fp4Runs {
  static constexpr int NW = D >= 128 ? 2 : 1;       // words of eight codes
  static __device__ __forceinline__ int code_lane(int r, int c) { return fp4_code_off(D, 2 * c, 4 * NW * r); }
  static __device__ __forceinline__ int scale_lane(int r, int c) {
    return fp4_scale_off(D, 2 * c, D == 64 ? r >> 1 : r);
  }
  static __device__ __forceinline__ int odd(int code_lane) {
    constexpr int R = Fp4Rows<D>::ROWB;
    return (code_lane & R) ? -R : R;
  }
  // at: token 2c's; on8 and odd behind it the others'
  static __device__ __forceinline__ void codes(uint32_t at, int b, uint32_t (&w)[NW]) {
    const uint32_t a = at + b * 1024;
    if constexpr (D >= 128) {
      const uint2 v = lds64(a);
      w[0] = v.x;
      w[1] = v.y;
    } else {
      w[0] = lds32(a);
    }
  }
  // E4M3 codes of tokens 2c + 8 i and 2c + 1 + 8 i
  static __device__ __forceinline__ uint32_t scale_pair(uint32_t at, int i, int b) {
    const uint32_t a = at + i * 8 * (D / 16) + b * 8;
    return lds_u8(a) | (lds_u8(a + D / 16) << 8);
  }
};

}  // namespace pa
