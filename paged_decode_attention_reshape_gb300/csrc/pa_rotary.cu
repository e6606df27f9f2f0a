// pa_rotary.cu -- rotary positions of query and key rows, with a norm of every head before the rotation
// and the cache write behind it.
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
// Work split.  The rows of all tokens (queries, then keys, then values), concatenated, are cut into
// equal ranges, one per CTA, whatever the numbers of tokens and heads.  D / 16 lanes take a row, 16
// elements a lane: eight of each half of the pairs (half layout: two runs of eight elements, 8-element
// runs of a row side by side in neighbouring lanes) or 16 side by side (interleaved); the lane's
// eight pairs are the same numbers in both.  A thread first asks for its share of all its rows, and
// while they come the CTA works out the sines of its tokens, once per (token, pair), into shared
// memory.  Bound: HBM, each row once in and once out.
#include "pa_fp4_quant.cuh"

namespace pa {
namespace {

// What becomes of the keys and values.
enum RotaryMode : int { ROWS = 0, COPY = 1, E4M3 = 2, E2M1 = 3 };

constexpr int kThreads = 256;
// rows a thread asks for at once (32 bytes each, 64 of fp32 rows)
template <int DT> constexpr int kRowsAtOnce = DT == PA_F32 ? 2 : 4;

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
// INTER: e1 = e0 + 8.
template <int DT, bool INTER>
struct Unit {
  static constexpr int IB = In<DT>::bytes, N = 4 * IB;  // words
  uint32_t w[N];
  __device__ __forceinline__ void load(const char *row, int e0, int e1, bool wide) {
    if constexpr (IB == 4) {
      load32(row + e0 * 4, wide, w);
      load32(row + e1 * 4, wide, w + 8);
    } else if constexpr (INTER) {
      load32(row + e0 * 2, wide, w);
    } else {
      const uint4 a = ld_row16(row + e0 * 2), b = ld_row16(row + e1 * 2);
      w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
      w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
    }
  }
  __device__ __forceinline__ void store(char *row, int e0, int e1, bool wide) const {
    if constexpr (IB == 4) {
      store32(row + e0 * 4, wide, w);
      store32(row + e1 * 4, wide, w + 8);
    } else if constexpr (INTER) {
      store32(row + e0 * 2, wide, w);
    } else {
      *reinterpret_cast<uint4 *>(row + e0 * 2) = make_uint4(w[0], w[1], w[2], w[3]);
      *reinterpret_cast<uint4 *>(row + e1 * 2) = make_uint4(w[4], w[5], w[6], w[7]);
    }
  }
  __device__ __forceinline__ void values(float (&x)[16]) const {
    if constexpr (IB == 4) {
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
  __device__ __forceinline__ void set(const float (&x)[16]) {
    if constexpr (IB == 4) {
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(x[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        w[i] = DT == PA_BF16 ? pack_bf16(x[2 * i], x[2 * i + 1]) : pack_f16(x[2 * i], x[2 * i + 1]);
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

template <int DT, int MODE, bool INTER>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotaryParams p) {
  // the decode that usually follows waits for this grid's completion before its first read
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  using U = Unit<DT, INTER>;
  constexpr int IB = U::IB, K = kRowsAtOnce<DT>;
  extern __shared__ float4 smem[];
  float *const weights = reinterpret_cast<float *>(smem);  // queries' [D], keys' [D]
  float4 *const turns = smem + p.D / 2;                    // [tokens][cos lo, cos hi, sin lo, sin hi][R / 16]

  const int lanes = p.D >> 4, u = threadIdx.x & (lanes - 1), group = threadIdx.x / lanes, groups = kThreads / lanes;
  const int RU = p.R >> 4;  // lanes with pairs
  const uint32_t mask = (lanes == 32 ? 0xffffffffu : (1u << lanes) - 1) << ((threadIdx.x & 31) & ~(lanes - 1));
  const int NR = p.Hq + p.Hk + p.Hv;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * p.rows_per_cta;
  const int64_t t0 = n0 / NR;
  const int r0 = static_cast<int>(n0 - t0 * NR);
  // the lane's runs of eight in a row that is rotated, and in a value
  int e0, e1, f0, f1;
  if constexpr (INTER) {
    e0 = f0 = 16 * u;
    e1 = f1 = 16 * u + 8;
  } else {
    const int base = u < RU ? 0 : p.R, n = u < RU ? RU : lanes - RU, i = u < RU ? u : u - RU;
    e0 = base + 8 * i;
    e1 = e0 + 8 * n;
    f0 = 8 * u;
    f1 = f0 + 8 * lanes;
  }

  U unit[K];
  int64_t tok[K], slot[K];
  int row[K];  // -1: none
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int off = k * groups + group;
    row[k] = -1;
    slot[k] = -1;
    tok[k] = 0;
    if (off < p.rows_per_cta) {
      const uint32_t at = static_cast<uint32_t>(r0) + off;
      // at / NR: below two for a row count past the range's, else by the host's reciprocal
      const uint32_t dt = p.magic ? __umulhi(at, p.magic) : NR == 1 ? at : at >= static_cast<uint32_t>(NR);
      const int64_t t = t0 + dt;
      if (t < p.T) {
        const int r = static_cast<int>(at - dt * NR);
        tok[k] = t;
        row[k] = r;
        if (r < p.Hq) {
          unit[k].load(p.q + t * p.q_ts + r * p.q_hs, e0, e1, p.wide);
        } else {
          if constexpr (MODE != ROWS) slot[k] = __ldg(p.slots + t);
          if (r < p.Hq + p.Hk) unit[k].load(p.key + t * p.key_ts + (r - p.Hq) * p.key_hs, e0, e1, p.wide);
          else unit[k].load(p.value + t * p.val_ts + (r - p.Hq - p.Hk) * p.val_hs, f0, f1, p.wide);
        }
      }
    }
  }

  // ---- sines of the CTA's tokens, norm weights
  if (p.R > 0) {
    const int half = p.R >> 1;
    const int64_t last = min(p.T - 1, (n0 + p.rows_per_cta - 1) / NR);
    const int count = static_cast<int>(last - t0 + 1) * half;
    float *const table = reinterpret_cast<float *>(turns);
    for (int j = threadIdx.x; j < count; j += kThreads) {
      const int dt = j / half, i = j - dt * half;
      const int64_t pos = p.pos64 ? __ldg(static_cast<const int64_t *>(p.positions) + t0 + dt)
                                  : static_cast<int64_t>(__ldg(static_cast<const int32_t *>(p.positions) + t0 + dt));
      const float2 cs = turned(pos, __ldg(p.frequencies + i));
      // pair i is element i % 8 of lane i / 8
      const int place = ((dt * 4 + ((i >> 2) & 1)) * RU + (i >> 3)) * 4 + (i & 3);
      table[place] = cs.x * p.magnitude;
      table[place + 2 * RU * 4] = cs.y * p.magnitude;
    }
  }
  if (p.q_weight || p.k_weight) {
    for (int i = threadIdx.x; i < p.D; i += kThreads) {
      if (p.q_weight) weights[i] = weight_at(p.q_weight, p.q_weight_dtype, i);
      if (p.k_weight) weights[p.D + i] = weight_at(p.k_weight, p.k_weight_dtype, i);
    }
  }
  __syncthreads();

#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int r = row[k];
    if (r < 0) continue;
    const int64_t t = tok[k];
    const bool is_q = r < p.Hq, is_v = r >= p.Hq + p.Hk;
    if (!is_v) {
      float x[16];
      unit[k].values(x);
      if (is_q ? p.q_weight != nullptr : p.k_weight != nullptr) {
        auto sum_of_squares = [&](float by) {
          float s = 0.f;
#pragma unroll
          for (int i = 0; i < 16; ++i) s = fmaf(x[i] * by, x[i] * by, s);
          for (int o = 1; o < lanes; o <<= 1) s += __shfl_xor_sync(mask, s, o);
          return s;
        };
        const float inv_d = 1.f / static_cast<float>(p.D);
        float by = 1.f, ms = fmaf(sum_of_squares(1.f), inv_d, p.eps);
        // squares that overflow, or vanish: once more by a power of two
        if (!(ms <= 0x1p120f)) {
          by = 0x1p-70f;
          ms = fmaf(sum_of_squares(by), inv_d, p.eps * by * by);
        } else if (ms < 0x1p-96f) {
          by = 0x1p64f;
          ms = fmaf(sum_of_squares(by), inv_d, p.eps * by * by);
        }
        const float rs = __frsqrt_rn(ms);
        const float *w = weights + (is_q ? 0 : p.D);
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const float4 f = *reinterpret_cast<const float4 *>(w + (i < 8 ? e0 : e1 - 8) + i);
          x[i] = x[i] * by * rs * f.x;
          x[i + 1] = x[i + 1] * by * rs * f.y;
          x[i + 2] = x[i + 2] * by * rs * f.z;
          x[i + 3] = x[i + 3] * by * rs * f.w;
        }
      }
      if (u < RU) {
        const float4 *cs = turns + static_cast<int>(t - t0) * 4 * RU + u;
        float c[8], s[8];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float4 a = cs[i * RU], b = cs[(2 + i) * RU];
          c[4 * i] = a.x, c[4 * i + 1] = a.y, c[4 * i + 2] = a.z, c[4 * i + 3] = a.w;
          s[4 * i] = b.x, s[4 * i + 1] = b.y, s[4 * i + 2] = b.z, s[4 * i + 3] = b.w;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float &a = x[INTER ? 2 * i : i], &b = x[INTER ? 2 * i + 1 : i + 8];
          const float a0 = a, b0 = b;
          // (written out: the same rounding in every variant)
          a = __fmaf_rn(-b0, s[i], __fmul_rn(a0, c[i]));
          b = __fmaf_rn(a0, s[i], __fmul_rn(b0, c[i]));
        }
      }
      unit[k].set(x);
    }
    if (is_q) {
      unit[k].store(p.q_out + t * p.qo_ts + r * p.qo_hs, e0, e1, p.wide);
      continue;
    }
    const int h = r - p.Hq - (is_v ? p.Hk : 0);
    const int g0 = is_v ? f0 : e0, g1 = is_v ? f1 : e1;
    if constexpr (MODE == ROWS) {
      unit[k].store(p.k_out + t * p.ko_ts + h * p.ko_hs, g0, g1, p.wide);
    } else {
      if (slot[k] < 0) continue;  // padding row: no destination
      if (slot[k] >= p.num_slots) {
        if (p.err && u == 0) atomicOr(p.err, kErrSlot);
        continue;
      }
      const int64_t blk = slot[k] >> 4;
      const int off = static_cast<int>(slot[k]) & (kBlock - 1);
      char *const dst = is_v ? p.v_cache + blk * p.vc_s0 + h * p.vc_s1 + off * p.vc_s2
                             : p.k_cache + blk * p.kc_s0 + h * p.kc_s1 + off * p.kc_s2;
      const float *const scales = is_v ? p.v_scale : p.k_scale;
      if constexpr (MODE == COPY) {
        unit[k].store(dst, g0, g1, p.wide);
      } else if constexpr (MODE == E4M3) {
        const Divisor dv = make_divisor(scales ? __ldg(scales + h * p.scale_stride) : 1.f);
#pragma unroll
        for (int i = 0; i < U::N / 4; ++i) {  // 16 bytes of the row: 8 or 4 elements
          constexpr int E = 16 / IB;
          const int first = i * E;
          store_fp8<DT>(dst + (first < 8 ? g0 : g1 - 8) + first,
                        make_uint4(unit[k].w[4 * i], unit[k].w[4 * i + 1], unit[k].w[4 * i + 2], unit[k].w[4 * i + 3]), dv);
        }
      } else {
        // lane u quantises elements 16 u .. 16 u + 15: runs 2u and 2u + 1 of eight, wherever they were
        uint32_t w[U::N];
        if constexpr (INTER) {
#pragma unroll
          for (int i = 0; i < U::N; ++i) w[i] = unit[k].w[i];
        } else {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int run = 2 * u + j;
            // the lane that holds it, and whether as its first or second run
            const int base = is_v || run < 2 * RU ? 0 : RU, n = is_v ? lanes : run < 2 * RU ? RU : lanes - RU;
            const int at = run - 2 * base;
            const bool second = at >= n;
            const int from = base + (second ? at - n : at);
#pragma unroll
            for (int i = 0; i < U::N / 2; ++i) {
              const uint32_t a = __shfl_sync(mask, unit[k].w[i], from, lanes);
              const uint32_t b = __shfl_sync(mask, unit[k].w[U::N / 2 + i], from, lanes);
              w[j * (U::N / 2) + i] = second ? b : a;
            }
          }
        }
        float x[16];
        group_values<DT>(w, x);
        const float s = scales ? __ldg(scales + h * p.scale_stride) : 1.f;
        const uint3 c = DT != PA_F32 && s == 1.f ? quantise_group<true>(x, 1.f, 1.f)
                                                 : quantise_group<false>(x, s, rcp_approx(s));
        char *const page = dst;  // (kc_s2 = 0)
        *reinterpret_cast<uint2 *>(page + fp4_code_off(p.D, off, u * 8)) = make_uint2(c.x, c.y);
        *reinterpret_cast<uint8_t *>(page + fp4_scale_off(p.D, off, u)) = static_cast<uint8_t>(c.z);
      }
    }
  }
}

template <int DT, int MODE, bool INTER>
cudaError_t launch_one(RotaryParams p, int sm_count, cudaStream_t st) {
  const int groups = kThreads / (p.D / 16);
  const int64_t NR = static_cast<int64_t>(p.Hq) + p.Hk + p.Hv, rows = p.T * NR;
  // rows per CTA: as many as a thread asks for at once, fewer where that leaves SMs without a CTA
  int k = kRowsAtOnce<DT>;
  while (k > 1 && (rows + groups * k - 1) / (groups * k) < 2 * sm_count) k >>= 1;
  p.rows_per_cta = groups * k;
  p.magic = NR > 1 && NR <= p.rows_per_cta ? static_cast<uint32_t>(((1ull << 32) + NR - 1) / NR) : 0;
  const int64_t blocks = (rows + p.rows_per_cta - 1) / p.rows_per_cta;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  const int64_t tokens = (p.rows_per_cta + NR - 2) / NR + 1;  // tokens that a range touches, at most
  const size_t smem = 2 * p.D * sizeof(float) + static_cast<size_t>(tokens) * p.R * sizeof(float);
  auto kern = rotary_kernel<DT, MODE, INTER>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = once_per_device(done, [kern] {
    cudaError_t r = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRotarySmem);
    // the SM's shared / L1 split stays what the decode kernels ask for (see pa_write.cu)
    return r != cudaSuccess ? r : cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout,
                                                       cudaSharedmemCarveoutMaxShared);
  });
  if (e != cudaSuccess) return e;
  kern<<<static_cast<unsigned>(blocks), kThreads, smem, st>>>(p);
  return cudaGetLastError();
}

template <int DT>
cudaError_t launch_type(const RotaryParams &p, int mode, int sm_count, cudaStream_t st) {
  switch (mode * 2 + (p.interleaved ? 1 : 0)) {
    case 0: return launch_one<DT, ROWS, false>(p, sm_count, st);
    case 1: return launch_one<DT, ROWS, true>(p, sm_count, st);
    case 2: return launch_one<DT, COPY, false>(p, sm_count, st);
    case 3: return launch_one<DT, COPY, true>(p, sm_count, st);
    case 4: return launch_one<DT, E4M3, false>(p, sm_count, st);
    case 5: return launch_one<DT, E4M3, true>(p, sm_count, st);
    case 6: return launch_one<DT, E2M1, false>(p, sm_count, st);
    case 7: return launch_one<DT, E2M1, true>(p, sm_count, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_rotary(const RotaryParams &p, int dtype, int cache_dtype, int sm_count, cudaStream_t st) {
  const int mode = !p.k_cache ? ROWS : cache_dtype == PA_FP8_E4M3 ? E4M3 : cache_dtype == PA_FP4_E2M1 ? E2M1 : COPY;
  switch (dtype) {
    case PA_F32: return launch_type<PA_F32>(p, mode, sm_count, st);
    case PA_BF16: return launch_type<PA_BF16>(p, mode, sm_count, st);
    case PA_F16: return launch_type<PA_F16>(p, mode, sm_count, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pa
