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
#include "pa_fp4_quant.cuh"

namespace pa {
namespace {

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

// A CTA per (page number, sequence): every head's page of K and V, a group of 16 elements a thread.  Codes
// (4-bit: times their group's scale, 6 bits) are 16-bit numbers exactly; the heads' scales go into the
// attention's own.  Bound by the bytes, a third read and the rest written: 16 chunks of 256..512 tokens, window
// 1024, 8 heads of 128, E4M3: 23 us for 132 MB, 5.7 TB/s (the attention behind it 188 us).
template <int CT, int OT>
__global__ void __launch_bounds__(256) widen_kernel(const WidenParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int v = blockIdx.x, s = blockIdx.y;
  const int len = __ldg(p.seq_lens + s), a = __ldg(p.qsl + s), b = __ldg(p.qsl + s + 1), nq = b - a;
  // (sequences that the attention refuses, and those without a query)
  if (len < 0 || len > p.max_blocks * kBlock || a < 0 || b > p.Tq || nq <= 0 || nq > p.nq_max || nq > len) return;
  const Window win = make_window(p.window, p.sinks, len - nq);
  if (v >= (len + kBlock - 1) / kBlock - win.skip || v >= p.pages) return;
  const int page = win.page(v);
  const int blk = __ldg(p.block_table + s * p.bt_ss + page);
  const bool bad = blk < 0 || blk >= p.num_blocks;
  if (threadIdx.x == 0) {
    p.table[static_cast<int64_t>(s) * p.max_blocks + page] = bad ? -1 : s * p.pages + v;
    if (bad && p.err) atomicOr(p.err, kErrBlock);
  }
  if (bad) return;
  const int groups = p.D / 16, per = p.Hkv * kBlock * groups;  // groups of a block of K
  char *const out0 = p.k_out + static_cast<int64_t>(s * static_cast<int64_t>(p.pages) + v) * per * 32;
  char *const out1 = p.v_out + static_cast<int64_t>(s * static_cast<int64_t>(p.pages) + v) * per * 32;
  for (int i = threadIdx.x; i < 2 * per; i += 256) {
    const bool second = i >= per;
    const int j = second ? i - per : i, gi = j % groups, t = j / groups % kBlock, h = j / groups / kBlock;
    const char *src = second ? p.v_cache + blk * p.vc_s0 + h * p.vc_s1 + t * p.vc_s2
                             : p.k_cache + blk * p.kc_s0 + h * p.kc_s1 + t * p.kc_s2;
    Cached<CT> c;
    c.load(src, p.D, t, gi);
    float x[16];
    c.values(1.f, x);
    store_group<OT>((second ? out1 : out0) + static_cast<int64_t>(j) * 32, p.wide, x);
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

cudaError_t launch_widen(const WidenParams &p, int cache_dtype, int out_dtype, cudaStream_t st) {
  const dim3 grid(p.pages, p.S), block(256);
  const bool fp4 = cache_dtype == PA_FP4_E2M1;
  cudaError_t e;
  if (out_dtype == PA_BF16)
    e = fp4 ? launch_pdl(widen_kernel<PA_FP4_E2M1, PA_BF16>, grid, block, 0, st, 1, p)
            : launch_pdl(widen_kernel<PA_FP8_E4M3, PA_BF16>, grid, block, 0, st, 1, p);
  else
    e = fp4 ? launch_pdl(widen_kernel<PA_FP4_E2M1, PA_F16>, grid, block, 0, st, 1, p)
            : launch_pdl(widen_kernel<PA_FP8_E4M3, PA_F16>, grid, block, 0, st, 1, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace pa
