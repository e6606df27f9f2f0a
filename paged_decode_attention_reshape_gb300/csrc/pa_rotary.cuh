// pa_rotary.cuh -- rotary positions of query and key rows, with a norm of every head before the rotation
// and the cache write behind it (instantiated per element type in pa_rotary_*.cu).
//
// For a row x [D] of a head at position t:
//   norm (with a weight w):  x <- x (mean(x^2) + eps)^(-1/2) w
//   rotation of pair i < R/2 (elements i and i + R/2, or interleaved 2i and 2i + 1; R <= D):
//     a <- m (a cos f_i t - b sin f_i t),  b <- m (b cos f_i t + a sin f_i t)
// Elements from R on pass.  Sums and products are fp32, the row is rounded to its type once; a key
// goes to the cache from there (copied, or quantised as pa_reshape_and_cache does, bit for bit), so a
// key read back is the one pa_rotary gives.
//
// Angles.  A frequency is held as turns per position in units of 2^-64, so the angle in turns is the
// 64-bit product position * frequency with its whole turns dropped by the arithmetic itself: exact
// for every position, negative ones included, where a product in fp32 has lost the angle's last bits
// from a few thousand positions on (and one in fp64 costs this GPU's scarce fp64 units).  What is left
// after the nearest quarter turn is at most pi / 4, 31 bits of it go to fp32, and the quarter turns
// pick and negate the two results of sincospif.
//
// Work split.  A warp takes a token at a time: the sines of its position, once per pair, through a table of its own
// in shared memory into registers (a lane needs the same eight pairs of every row), then the token's
// rows, queries, keys, values, 32 / (D / 16) of them at a time.  D / 16 lanes take a row, 16 elements a
// lane: eight of each half of the pairs (half layout: two runs of eight elements, side by side in
// neighbouring lanes) or 16 side by side (interleaved); the eight pairs are the same numbers in both.
// The grid is one resident wave; the tokens that do not fill a whole round of its warps (a few tokens, or the
// last ones) are cut by groups of rows, each token into the same number of pieces where that takes no more
// groups a warp than equal shares of all would, else into those shares (which may hold the end of one token and
// the start of the next): 8192 tokens of 40 rows, 2.2 rounds, 30 us, in whole tokens 32; 5001 of 80, 1.4
// rounds, 38 us, in whole tokens 42.
// Warps wait for nothing but their own loads, which run kAhead groups of rows ahead.
// Bound: HBM, each row once in and once out, as long as the instructions per row stay few: fp32 pairs go
// through the two-lane operations, what a token's rows share is worked out once, and queries, keys and values
// have loops of their own with a pointer each way.  Bf16, heads of 128, normalised, into a bf16 cache, 32768
// tokens of 32/8 heads: 142 us, 5.7 TB/s, 0.83 of the copy peak (a CTA per range of rows of any tokens, with the
// sines in shared memory for every row: 199 us and 406 warp instructions per 16 elements a lane, here 196).
#pragma once

#include <algorithm>
#include <type_traits>

#include "pa_fp4_quant.cuh"

namespace pa {

// What becomes of the keys and values.
enum RotaryMode : int { ROTARY_ROWS = 0, ROTARY_COPY = 1, ROTARY_E4M3 = 2, ROTARY_E2M1 = 3 };

// Warps of a CTA (at most), CTAs resident per SM (16-bit rows: 2 / 3 / 4 with 3 / 2 / 2 groups on their way,
// 32768 tokens of 48 rows: 156 / 142 / 161 us; at 3, 80 registers, the copy mode spills nothing to 4 bytes, rows 0 to
// 32, E4M3 4 to 40, 4-bit 40 to 52), groups of rows that a warp has on their way (3: 144 us).
constexpr int kRotaryWarps = 8;
template <int DT> constexpr int kRotaryCtas = DT == PA_F32 ? 2 : 3;
constexpr int kAhead = 2;

// Eight elements in place: 16 bytes of a 16-bit row, 32 of an fp32 one.  (Rows may be rotated in
// place, so not through the read-only path.)
__device__ __forceinline__ uint4 ld_row16(const char *p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}
__device__ __forceinline__ void ld_row32(const char *p, uint32_t *v) {
  asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
               : "l"(p)
               : "memory");
}
// 32 bytes, 32-byte aligned (wide) or 16.
__device__ __forceinline__ void load32(const char *p, bool wide, uint32_t *w) {
  if (wide) {
    ld_row32(p, w);
  } else {
    const uint4 a = ld_row16(p), b = ld_row16(p + 16);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
    w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  }
}
__device__ __forceinline__ void store32(char *p, bool wide, const uint32_t *w) {
  if (wide) {
    const uint32_t v[8] = {w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]};
    st32(p, v);
  } else {
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4 *>(p + 16) = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// A lane's 16 elements of a row: two runs of eight, from elements e0 and e1 on, as their bytes.
// INTER: e1 = e0 + 8.  As values they are eight pairs: elements e0 + i and e1 + i, or (INTER) e0 + 2i and
// e0 + 2i + 1.
template <int DT, bool INTER>
struct Unit {
  static constexpr int IB = In<DT>::bytes, N = 4 * IB;  // words
  uint32_t w[N];
  // from the first run's address and, `on` bytes behind it, the second's
  __device__ __forceinline__ void load(const char *at, int on, bool wide) {
    if constexpr (IB == 4) {
      load32(at, wide, w);
      load32(at + on, wide, w + 8);
    } else if constexpr (INTER) {
      load32(at, wide, w);
    } else {
      const uint4 a = ld_row16(at), b = ld_row16(at + on);
      w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
      w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
    }
  }
  __device__ __forceinline__ void store(char *at, int on, bool wide) const {
    if constexpr (IB == 4) {
      store32(at, wide, w);
      store32(at + on, wide, w + 8);
    } else if constexpr (INTER) {
      store32(at, wide, w);
    } else {
      *reinterpret_cast<uint4 *>(at) = make_uint4(w[0], w[1], w[2], w[3]);
      *reinterpret_cast<uint4 *>(at + on) = make_uint4(w[4], w[5], w[6], w[7]);
    }
  }
  __device__ __forceinline__ float2 two(int i) const {  // elements 2i and 2i + 1 of the 16
    if constexpr (IB == 4) return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    else return DT == PA_BF16 ? unpack_bf16(w[i]) : unpack_f16(w[i]);
  }
  __device__ __forceinline__ void pairs(float (&a)[8], float (&b)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 f = two(i);
      if constexpr (INTER) {
        a[i] = f.x;
        b[i] = f.y;
      } else {
        (i < 4 ? a : b)[2 * (i & 3)] = f.x;
        (i < 4 ? a : b)[2 * (i & 3) + 1] = f.y;
      }
    }
  }
  __device__ __forceinline__ void set(const float (&a)[8], const float (&b)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = INTER ? a[i] : (i < 4 ? a : b)[2 * (i & 3)], y = INTER ? b[i] : (i < 4 ? a : b)[2 * (i & 3) + 1];
      if constexpr (IB == 4) {
        w[2 * i] = __float_as_uint(x);
        w[2 * i + 1] = __float_as_uint(y);
      } else {
        w[i] = DT == PA_BF16 ? pack_bf16(x, y) : pack_f16(x, y);
      }
    }
  }
};

// cos and sin of position * frequency, `frequency` in 2^-64 turns per position.
__device__ __forceinline__ float2 turned(int64_t position, uint64_t frequency) {
  const uint64_t phase = static_cast<uint64_t>(position) * frequency;
  const uint32_t quarter = static_cast<uint32_t>((phase + (1ull << 61)) >> 62);  // (4 wraps to 0)
  const int32_t rest = static_cast<int32_t>(static_cast<int64_t>(phase - (static_cast<uint64_t>(quarter) << 62)) >> 30);
  float s, c;
  sincospif(static_cast<float>(rest) * 0x1p-33f, &s, &c);
  const float x = quarter & 1 ? s : c, y = quarter & 1 ? c : s;
  return make_float2(((quarter + 1) & 2) ? -x : x, (quarter & 2) ? -y : y);
}

__device__ __forceinline__ float weight_at(const void *w, int dtype, int i) {
  return dtype == PA_F32    ? __ldg(static_cast<const float *>(w) + i)
         : dtype == PA_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(w)[i])
                            : __half2float(static_cast<const __half *>(w)[i]);
}

template <int DT, int D, int MODE, bool INTER>
__global__ void __launch_bounds__(kRotaryWarps * 32, kRotaryCtas<DT>) rotary_kernel(const RotaryParams p) {
  // the decode that usually follows waits for this grid's completion before its first read
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  using U = Unit<DT, INTER>;
  constexpr int LANES = D / 16, RW = 32 / LANES;  // lanes of a row, rows of a group
  constexpr uint32_t ALL = 0xffffffffu;
  __shared__ float4 weights[2][4][LANES];              // queries', keys': [a lo, a hi, b lo, b hi]
  __shared__ float4 tables[kRotaryWarps][4][LANES];    // the warp's token: [cos lo, cos hi, sin lo, sin hi]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int u = lane % LANES, sub = lane / LANES;
  const int RU = p.R >> 4;  // lanes with pairs
  // a lane's runs of eight in a row that is rotated, and in a value
  auto run0 = [&](int i) {
    if constexpr (INTER) return 16 * i;
    else return i < RU ? 8 * i : p.R + 8 * (i - RU);
  };
  auto run1 = [&](int i) {
    if constexpr (INTER) return 16 * i + 8;
    else return run0(i) + 8 * (i < RU ? RU : LANES - RU);
  };
  const int e0 = run0(u), e1 = run1(u), f0 = INTER ? e0 : 8 * u, f1 = INTER ? e1 : 8 * (u + LANES);

  // Launched as a programmatic dependent of the preceding work: nothing is read or written before its end.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (p.q_weight || p.k_weight) {
    for (int j = threadIdx.x; j < D; j += blockDim.x) {
      const int i = j / 4 % LANES, part = j / (4 * LANES), n = 4 * (part & 1) + (j & 3);
      const int e = INTER ? 16 * i + 2 * n + (part >> 1) : (part >> 1 ? run1(i) : run0(i)) + n;
      if (p.q_weight) reinterpret_cast<float *>(weights[0])[j] = weight_at(p.q_weight, p.q_weight_dtype, e);
      if (p.k_weight) reinterpret_cast<float *>(weights[1])[j] = weight_at(p.k_weight, p.k_weight_dtype, e);
    }
    __syncthreads();
  }

  U x[kAhead];
#pragma unroll
  for (int j = 0; j < kAhead; ++j)
#pragma unroll
    for (int i = 0; i < U::N; ++i) x[j].w[i] = 0u;  // (lanes without a row go along with what they hold)

  // groups of RW rows: the queries', the keys', the values'
  const int IK = p.groups_q, IV = IK + p.groups_k, IE = IV + p.groups_v;
  // This warp's share: a token of each whole round, then groups n0 .. n1 - 1 of the remaining tokens.
  const int w = blockIdx.x * warps + warp, all_warps = gridDim.x * warps;
  int n0, n1;
  if (p.pieces > 0) {
    const int token = w / p.pieces;
    n0 = token < p.extra ? token * IE + (w - token * p.pieces) * p.share : 0;
    n1 = token < p.extra ? min(n0 + p.share, (token + 1) * IE) : 0;
  } else {
    n0 = w * p.share + min(w, p.extra);
    n1 = n0 + p.share + (w < p.extra ? 1 : 0);
  }
  for (int round = 0;; ++round) {
    int t, it = 0, end = IE;
    if (round < p.rounds) {
      t = round * all_warps + w;
    } else {
      if (n0 >= n1) return;
      const int token = n0 / IE;
      t = p.rounds * all_warps + token;
      it = n0 - token * IE;
      end = min(IE, it + n1 - n0);
      n0 += end - it;
    }
    uint64_t c[4], s[4];  // of pairs 2i and 2i + 1 of the lane's eight
    const bool turn = u < RU;

    auto rotate = [&](U &unit, auto kind) {
      constexpr int KIND = decltype(kind)::value;
      const bool norm = KIND == 0 ? p.q_weight != nullptr : p.k_weight != nullptr;
      float a[8], b[8];
      unit.pairs(a, b);
      uint64_t x[4], y[4];  // pairs 2i and 2i + 1: their a, their b
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        x[n] = f2pack(a[2 * n], a[2 * n + 1]);
        y[n] = f2pack(b[2 * n], b[2 * n + 1]);
      }
      if (norm) {
        auto sum_of_squares = [&]() {
          uint64_t f = f2mul(x[0], x[0]), g = f2mul(y[0], y[0]);
#pragma unroll
          for (int n = 1; n < 4; ++n) {
            f = f2fma(x[n], x[n], f);
            g = f2fma(y[n], y[n], g);
          }
          const float2 e = f2unpack(f2add(f, g));
          float v = e.x + e.y;
#pragma unroll
          for (int o = 1; o < LANES; o <<= 1) v += __shfl_xor_sync(ALL, v, o);
          return v;
        };
        auto times = [&](float f) {
          const uint64_t ff = f2pack(f, f);
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            x[n] = f2mul(x[n], ff);
            y[n] = f2mul(y[n], ff);
          }
        };
        float ms = fmaf(sum_of_squares(), 1.f / D, p.eps);
        // squares that overflow, or vanish: those rows once more by a power of two (2^100: an fp32 row's largest
        // element is then at most 2^56, its sum 2^120, and the square of the smallest number there is 2^-98)
        if (__any_sync(ALL, !(ms <= 0x1p120f) || ms < 0x1p-96f)) {
          const float by = ms < 0x1p-96f ? 0x1p100f : ms <= 0x1p120f ? 1.f : 0x1p-70f;
          times(by);
          ms = fmaf(sum_of_squares(), 1.f / D, p.eps * by * by);
        }
        times(__frsqrt_rn(ms));
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const float4 f = weights[KIND][n][u], g = weights[KIND][2 + n][u];
          x[2 * n] = f2mul(x[2 * n], f2pack(f.x, f.y));
          x[2 * n + 1] = f2mul(x[2 * n + 1], f2pack(f.z, f.w));
          y[2 * n] = f2mul(y[2 * n], f2pack(g.x, g.y));
          y[2 * n + 1] = f2mul(y[2 * n + 1], f2pack(g.z, g.w));
        }
      }
      if (turn) {
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const float2 ac = f2unpack(f2mul(x[n], c[n])), bb = f2unpack(y[n]), sf = f2unpack(s[n]);
          y[n] = f2fma(x[n], s[n], f2mul(y[n], c[n]));
          x[n] = f2pack(__fmaf_rn(-bb.x, sf.x, ac.x), __fmaf_rn(-bb.y, sf.y, ac.y));
        }
      }
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const float2 f = f2unpack(x[n]), g = f2unpack(y[n]);
        a[2 * n] = f.x, a[2 * n + 1] = f.y;
        b[2 * n] = g.x, b[2 * n + 1] = g.y;
      }
      unit.set(a, b);
    };

    int off = 0;  // 4-bit: the token within its page
    // Groups i0 .. i1 - 1 of one kind of rows (0 queries, 1 keys, 2 values), `heads` a token: from src to dst,
    // both the token's row of head 0.
    auto section = [&](auto kind, int i0, int i1, int heads, const char *src, int64_t src_hs, char *dst, int64_t dst_hs,
                       auto before) {
      constexpr int KIND = decltype(kind)::value;
      constexpr bool CACHED = MODE != ROTARY_ROWS && KIND > 0;
      const int a0 = KIND == 2 ? f0 : e0, a1 = KIND == 2 ? f1 : e1;
      const int head0 = i0 * RW + sub;
      const char *from = src + head0 * src_hs + a0 * U::IB;
      int rows = heads - head0;  // > 0: this lane has a row of the group
      auto fetch = [&](U &y) {
        if (rows > 0) y.load(from, (a1 - a0) * U::IB, p.wide);
        rows -= RW;
        from += RW * src_hs;
      };
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        if (i0 + j < i1) fetch(x[j]);
      before();  // (while they come)
      char *to = dst + head0 * dst_hs + (CACHED && MODE != ROTARY_COPY ? 0 : a0 * U::IB);
      int left = heads - head0;
      auto process = [&](U &unit) {
        if constexpr (KIND < 2) rotate(unit, kind);
        const bool live = left > 0;
        const int h = heads - left;
        char *const at = to;
        left -= RW;
        to += RW * dst_hs;
        if constexpr (!CACHED || MODE == ROTARY_COPY) {
          if (live) unit.store(at, (a1 - a0) * U::IB, p.wide);
        } else if constexpr (MODE == ROTARY_E4M3) {
          if (!live) return;
          const float *const scales = KIND == 2 ? p.v_scale : p.k_scale;
          const Divisor dv = make_divisor(scales ? __ldg(scales + h * p.scale_stride) : 1.f);
#pragma unroll
          for (int n = 0; n < U::N / 4; ++n) {  // 16 bytes of the row: 8 or 4 elements
            const int first = n * (16 / U::IB);
            store_fp8<DT>(at + (first < 8 ? a0 : a1 - 8) + first,
                          make_uint4(unit.w[4 * n], unit.w[4 * n + 1], unit.w[4 * n + 2], unit.w[4 * n + 3]), dv);
          }
        } else {
          // lane u quantises elements 16 u .. 16 u + 15: runs 2u and 2u + 1 of eight, wherever they were
          uint32_t v[U::N];
          if constexpr (INTER) {
#pragma unroll
            for (int n = 0; n < U::N; ++n) v[n] = unit.w[n];
          } else {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int run = 2 * u + j;
              // the lane that holds it, and whether as its first or second run
              const int base = KIND == 2 || run < 2 * RU ? 0 : RU, n_lanes = KIND == 2 ? LANES : run < 2 * RU ? RU : LANES - RU;
              const int place = run - 2 * base;
              const bool second = place >= n_lanes;
              const int lane_of = base + (second ? place - n_lanes : place);
#pragma unroll
              for (int n = 0; n < U::N / 2; ++n) {
                const uint32_t v0 = __shfl_sync(ALL, unit.w[n], lane_of, LANES);
                const uint32_t v1 = __shfl_sync(ALL, unit.w[U::N / 2 + n], lane_of, LANES);
                v[j * (U::N / 2) + n] = second ? v1 : v0;
              }
            }
          }
          if (!live) return;
          float y[16];
          group_values<DT>(v, y);
          const float *const scales = KIND == 2 ? p.v_scale : p.k_scale;
          const float scale = scales ? __ldg(scales + h * p.scale_stride) : 1.f;
          const uint3 q = DT != PA_F32 && scale == 1.f ? quantise_group<true>(y, 1.f, 1.f)
                                                       : quantise_group<false>(y, scale, rcp_approx(scale));
          *reinterpret_cast<uint2 *>(at + fp4_code_off(D, off, u * 8)) = make_uint2(q.x, q.y);
          *reinterpret_cast<uint8_t *>(at + fp4_scale_off(D, off, u)) = static_cast<uint8_t>(q.z);
        }
      };
      for (int i = i0; i < i1; i += kAhead) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          if (i + j >= i1) break;
          process(x[j]);
          if (i + j + kAhead < i1) fetch(x[j]);
        }
      }
    };
    auto sines = [&] {  // of the token's position, into c and s
      if (p.R == 0) return;
      const int64_t pos = p.pos64 ? __ldg(static_cast<const int64_t *>(p.positions) + t)
                                  : static_cast<int64_t>(__ldg(static_cast<const int32_t *>(p.positions) + t));
      float *const table = reinterpret_cast<float *>(tables[warp]);
      __syncwarp();  // (the last token's are read)
      for (int i = lane; i < p.R >> 1; i += 32) {
        const float2 cs = turned(pos, __ldg(p.frequencies + i));
        // pair i is the i % 8-th of lane i / 8
        const int place = (((i >> 2) & 1) * LANES + (i >> 3)) * 4 + (i & 3);
        table[place] = cs.x * p.magnitude;
        table[place + 2 * LANES * 4] = cs.y * p.magnitude;
      }
      __syncwarp();
      if (turn) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float4 cc = tables[warp][i][u], ss = tables[warp][2 + i][u];
          c[2 * i] = f2pack(cc.x, cc.y), c[2 * i + 1] = f2pack(cc.z, cc.w);
          s[2 * i] = f2pack(ss.x, ss.y), s[2 * i + 1] = f2pack(ss.z, ss.w);
        }
      }
    };
    auto nothing = [] {};
    int64_t slot = -1;
    if constexpr (MODE != ROTARY_ROWS) slot = __ldg(p.slots + t);
    bool turned_yet = false;
    auto once = [&] {
      if (!turned_yet) sines();
      turned_yet = true;
    };
    if (it < IK)
      section(std::integral_constant<int, 0>{}, it, min(end, IK), p.Hq, p.q + t * p.q_ts, p.q_hs, p.q_out + t * p.qo_ts,
              p.qo_hs, once);
    if (end <= IK) continue;
    if constexpr (MODE == ROTARY_ROWS) {
      section(std::integral_constant<int, 1>{}, max(it, IK) - IK, end - IK, p.Hk, p.key + t * p.key_ts, p.key_hs,
              p.k_out + t * p.ko_ts, p.ko_hs, once);
    } else {
      if (slot >= p.num_slots) {
        if (p.err && lane == 0) atomicOr(p.err, kErrSlot);
        continue;
      }
      if (slot < 0) continue;  // a padding row: no destination
      const int64_t blk = slot >> 4;
      off = static_cast<int>(slot) & (kBlock - 1);
      if (it < IV)
        section(std::integral_constant<int, 1>{}, max(it, IK) - IK, min(end, IV) - IK, p.Hk, p.key + t * p.key_ts, p.key_hs,
                p.k_cache + blk * p.kc_s0 + off * p.kc_s2, p.kc_s1, once);
      if (end > IV)
        section(std::integral_constant<int, 2>{}, max(it, IV) - IV, end - IV, p.Hv, p.value + t * p.val_ts, p.val_hs,
                p.v_cache + blk * p.vc_s0 + off * p.vc_s2, p.vc_s1, nothing);
    }
  }
}

template <int DT, int D, int MODE, bool INTER>
cudaError_t launch_rotary_one(RotaryParams p, int sm_count, cudaStream_t st) {
  constexpr int RW = 32 / (D / 16);
  p.groups_q = (p.Hq + RW - 1) / RW;
  p.groups_k = (p.Hk + RW - 1) / RW;
  p.groups_v = (p.Hv + RW - 1) / RW;
  const int64_t groups = p.groups_q + p.groups_k + p.groups_v;
  const int64_t all = p.T < INT64_MAX / groups ? p.T * groups : INT64_MAX;
  // one resident wave of CTAs; smaller ones where there are few groups, so that every SM has some
  int warps = kRotaryWarps;
  while (warps > 1 && all < static_cast<int64_t>(sm_count) * warps) warps >>= 1;
  const int64_t blocks = std::min<int64_t>((all + warps - 1) / warps, static_cast<int64_t>(sm_count) * kRotaryCtas<DT>);
  const int64_t wave = blocks * warps;
  p.rounds = static_cast<int>(p.T / wave);
  const int64_t tokens = p.T - p.rounds * wave, rest = tokens * groups;  // (below wave * groups: 2^31)
  const int64_t per = std::max<int64_t>((rest + wave - 1) / wave, 1), pieces = (groups + per - 1) / per;
  p.pieces = tokens * pieces <= wave ? static_cast<int>(pieces) : 0;
  p.share = static_cast<int>(p.pieces > 0 ? (groups + pieces - 1) / pieces : rest / wave);
  p.extra = static_cast<int>(p.pieces > 0 ? tokens : rest % wave);
  auto kern = rotary_kernel<DT, D, MODE, INTER>;
  static std::atomic<uint64_t> done{0};
  // the SM's shared / L1 split stays what the decode kernels ask for (see pa_write.cu)
  cudaError_t e = once_per_device(done, [kern] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
  });
  if (e != cudaSuccess) return e;
  // (its start overlaps the end of what runs before it: a call among others 32.8 -> 30.4 us on 8192 x 40 rows)
  e = launch_pdl(kern, dim3(static_cast<unsigned>(blocks)), dim3(warps * 32), 0, st, 1, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int DT, int MODE>
cudaError_t launch_rotary_mode(const RotaryParams &p, int sm_count, cudaStream_t st) {
  switch (p.D * 2 + (p.interleaved ? 1 : 0)) {
    case 128: return launch_rotary_one<DT, 64, MODE, false>(p, sm_count, st);
    case 129: return launch_rotary_one<DT, 64, MODE, true>(p, sm_count, st);
    case 256: return launch_rotary_one<DT, 128, MODE, false>(p, sm_count, st);
    case 257: return launch_rotary_one<DT, 128, MODE, true>(p, sm_count, st);
    case 512: return launch_rotary_one<DT, 256, MODE, false>(p, sm_count, st);
    case 513: return launch_rotary_one<DT, 256, MODE, true>(p, sm_count, st);
    default: return cudaErrorInvalidValue;
  }
}

template <int DT>
cudaError_t launch_rotary_type(const RotaryParams &p, int cache_dtype, int sm_count, cudaStream_t st) {
  if (!p.k_cache) return launch_rotary_mode<DT, ROTARY_ROWS>(p, sm_count, st);
  if (cache_dtype == PA_FP8_E4M3) return launch_rotary_mode<DT, ROTARY_E4M3>(p, sm_count, st);
  if (cache_dtype == PA_FP4_E2M1) return launch_rotary_mode<DT, ROTARY_E2M1>(p, sm_count, st);
  return launch_rotary_mode<DT, ROTARY_COPY>(p, sm_count, st);
}

}  // namespace pa
