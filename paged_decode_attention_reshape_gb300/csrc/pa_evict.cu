// pa_evict.cu -- eviction from the paged cache by accumulated attention weight.
//
// Of every sequence s longer than the budget B and every KV head g, the last R tokens stay
// and, of the others, the B - R of largest weight (pa_decode_accumulate's array), equal
// weights by lowest position.  They keep their order and move to positions 0 .. B - 1 of the
// sequence's own blocks; the blocks behind are free afterwards.  Each KV head keeps its own
// tokens: a head's rows of a block are its own, so only the count has to agree.
//
// Two kernels.
//
// select_kernel, one CTA (of 256 threads; 1024 for few long rows) per (s, g): the weight of the last token to stay is found digit by
// digit (radix select on the floats' ordered bit patterns, 11 + 11 + 10 bits: a histogram in
// shared memory, then the digit in which the count from the top passes what is still wanted),
// which is exact for any distribution and needs no sort; then every warp counts and writes its own
// stretch of the kept positions and their weights, in order.  The passes work on registers for
// the first 16 a thread, on L2 behind them.  Bound: 4 bytes a token from HBM once; in fact the
// passes' latency.
//
// move_kernel, one or more CTAs per (s, g) and cache: rows p_0 < p_1 < ... move to rows
// 0, 1, ....  p_i >= i, so in ascending order a row is only ever overwritten after it has been
// read, and rows of a later stretch never lie where an earlier one writes: a CTA reads a stretch
// into registers, meets at a barrier, and writes it, with the next one's reads in flight.  Rows at the front that stay where they
// are (p_i = i) are not touched.  CTAs of one (s, g) take different bytes of the rows.  Bound:
// every kept row read and written once.
#include "pa_fp4.cuh"
#include "pa_internal.h"
#include "pa_merge.cuh"
#include "pa_validate.h"

#define PA_API extern "C" __attribute__((visibility("default")))

namespace pa {
namespace {

struct EvictParams {
  char *cache[2];              // K, V
  int64_t s0[2], s1[2], s2[2]; // bytes (s2 not used by 4-bit pages)
  const int32_t *block_table;
  int64_t bt_ss;
  const int32_t *seq_lens;
  const float *weights;
  float *new_weights;
  int64_t w_ss, w_hs, nw_ss, nw_hs;
  int32_t *kept;
  int64_t k_ss, k_hs;
  int32_t *new_lens;
  int Hkv, D, num_blocks, max_blocks, W, budget, recent;
  int pieces, slices;          // pieces of a row; CTAs that share a row's pieces
  int *err;
};

constexpr int kBins = 2048;
constexpr int kHeld = 16;  // tiles of 32 weights that a warp keeps in registers (16 T tokens a CTA)

// Bit patterns that order as the floats do (-0 as +0, NaN below everything).
__device__ __forceinline__ uint32_t ordered_bits(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

template <int T>
__global__ void __launch_bounds__(T, T == 256 ? 4 : 1) select_kernel(const EvictParams p) {
  constexpr int kWarps = T / 32, kPerThread = kBins / T;
  __shared__ uint32_t hist[kBins];
  __shared__ uint32_t s_sum[kWarps], s_above[kWarps], s_equal[kWarps];
  __shared__ uint32_t s_digit, s_left;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = blockIdx.x, s = blockIdx.y, tid = threadIdx.x;
  grid_dependency_wait();
  const int len = __ldg(p.seq_lens + s);
  const float *w = p.weights + s * p.w_ss + g * p.w_hs;
  float *nw = p.new_weights + s * p.nw_ss + g * p.nw_hs;
  int32_t *kept = p.kept + s * p.k_ss + g * p.k_hs;
  const bool len_ok = len >= 0 && len <= p.max_blocks * kBlock;
  bool bad = !len_ok;
  if (len_ok) {
    const int32_t *bt = p.block_table + s * p.bt_ss;
    for (int b = tid; b < (len + kBlock - 1) / kBlock; b += T) {
      const int id = __ldg(bt + b);
      bad |= id < 0 || id >= p.num_blocks;
    }
  }
  bad = __syncthreads_or(bad);
  if (bad && g == 0 && tid == 0 && p.err) atomicOr(p.err, len_ok ? kErrBlock : kErrSeqLen);
  if (bad || len <= p.budget) {  // nothing to evict, or nothing that may be touched
    for (int i = tid; i < p.budget; i += T) kept[i] = !bad && i < len ? i : -1;
    for (int i = tid; i < p.W; i += T) nw[i] = bad || i < len ? __ldg(w + i) : 0.f;
    if (g == 0 && tid == 0) p.new_lens[s] = len;
    return;
  }
  const int tail = min(p.recent, p.budget);
  const int cand = len - tail;             // candidates: positions 0 .. cand - 1
  const uint32_t want = p.budget - tail;   // of which this many stay (< cand)
  // Warp w has the candidates [w per, (w + 1) per): `tiles` rows of 32, the first kHeld of them in
  // registers as ordered bits, the others read again by each pass.
  const int per = ((cand + kWarps - 1) / kWarps + 31) / 32 * 32, tiles = per / 32;
  const int first = warp * per + lane;
  uint32_t held[kHeld];
#pragma unroll
  for (int j = 0; j < kHeld; ++j)
    held[j] = j < tiles && first + 32 * j < cand ? ordered_bits(__ldg(w + first + 32 * j)) : 0u;
  auto each = [&](auto f) {  // f(position, ordered bits, a candidate), whole warps
#pragma unroll
    for (int j = 0; j < kHeld; ++j)
      if (j < tiles) f(first + 32 * j, held[j], first + 32 * j < cand);
    for (int j = kHeld; j < tiles; ++j) {
      const int t = first + 32 * j;
      f(t, t < cand ? ordered_bits(__ldg(w + t)) : 0u, t < cand);
    }
  };
  // the threshold: `prefix` holds its leading `done` bits, `left` of the candidates that share
  // them are still wanted
  uint32_t prefix = 0, left = want;
  if (want > 0) {
    int done = 0;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int bits = pass < 2 ? 11 : 10, shift = 32 - done - bits;
      for (int i = tid; i < kBins; i += T) hist[i] = 0;
      __syncthreads();
      each([&](int, uint32_t u, bool in) {
        if (in && (done == 0 || (u >> (32 - done)) == prefix)) atomicAdd(&hist[(u >> shift) & ((1u << bits) - 1)], 1u);
      });
      __syncthreads();
      // counts from the top: thread i holds the kPerThread bins from the i-th group down
      uint32_t c[kPerThread], sum = 0;
#pragma unroll
      for (int j = 0; j < kPerThread; ++j) {
        c[j] = hist[kBins - 1 - kPerThread * tid - j];
        sum += c[j];
      }
      uint32_t before = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t t = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += t;
      }
      if (lane == 31) s_sum[warp] = before;
      before -= sum;
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kWarps; ++k) before += k < warp ? s_sum[k] : 0u;
#pragma unroll
      for (int j = 0; j < kPerThread; ++j) {
        if (before < left && left <= before + c[j]) {
          s_digit = kBins - 1 - kPerThread * tid - j;
          s_left = left - before;
        }
        before += c[j];
      }
      __syncthreads();
      prefix = (prefix << bits) | s_digit;
      left = s_left;
      done += bits;
    }
    // kept candidates in order: all above the threshold, and the first `left` equal to it.  Counts per
    // warp first, then every warp writes its own.
    uint32_t above = 0, equal = 0;
    each([&](int, uint32_t u, bool in) {
      above += __popc(__ballot_sync(0xffffffffu, in && u > prefix));
      equal += __popc(__ballot_sync(0xffffffffu, in && u == prefix));
    });
    if (lane == 0) {
      s_above[warp] = above;
      s_equal[warp] = equal;
    }
    __syncthreads();
    above = equal = 0;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      above += k < warp ? s_above[k] : 0u;
      equal += k < warp ? s_equal[k] : 0u;
    }
    each([&](int t, uint32_t u, bool in) {
      const bool gt = in && u > prefix, eq = in && u == prefix;
      const uint32_t mg = __ballot_sync(0xffffffffu, gt), me = __ballot_sync(0xffffffffu, eq);
      const uint32_t lower = (1u << lane) - 1;
      const uint32_t e = equal + __popc(me & lower);
      if (gt || (eq && e < left)) {
        const uint32_t at = above + __popc(mg & lower) + min(e, left);
        if (at < want) {  // always, unless the weights change during the call
          kept[at] = t;
          nw[at] = __ldg(w + t);
        }
      }
      above += __popc(mg);
      equal += __popc(me);
    });
  }
  for (int i = tid; i < tail; i += T) {
    kept[want + i] = cand + i;
    nw[want + i] = __ldg(w + cand + i);
  }
  for (int i = p.budget + tid; i < p.W; i += T) nw[i] = 0.f;
  if (g == 0 && tid == 0) p.new_lens[s] = p.budget;
}

constexpr int kMoveUnroll = 4;     // rows of a thread in a stretch

// V: the piece of a row that one thread moves at a time (16 bytes, or D / 16 of a 4-bit page: 8
// pieces of a token's codes and its scales as the ninth).  The next stretch is read while the
// last one is written, and its positions one stretch ahead of that.
template <typename V, bool FP4, int T>
__global__ void __launch_bounds__(T) move_kernel(const EvictParams p) {
  const int which = blockIdx.x / p.slices, slice = blockIdx.x - which * p.slices;
  const int g = blockIdx.y, s = blockIdx.z;
  grid_dependency_wait();
  const int32_t *kept = p.kept + s * p.k_ss + g * p.k_hs;
  const int len = __ldg(p.seq_lens + s);
  if (len <= p.budget || __ldcg(kept) < 0) return;  // nothing moves (kept[0] < 0: a fault)
  // Positions and blocks are select_kernel's, checked there.  A caller that writes the inputs during
  // the call gets wrong rows, but none outside the caches: what is read again is bounded again.
  const unsigned last_block = p.num_blocks - 1;
  if (len > p.max_blocks * kBlock || p.num_blocks <= 0) return;
  const int32_t *bt = p.block_table + s * p.bt_ss;
  char *base = p.cache[which] + g * p.s1[which];
  const int64_t s0 = p.s0[which], s2 = p.s2[which];
  const int rows = blockDim.y, r = threadIdx.y, q = slice * blockDim.x + threadIdx.x;
  auto place = [&](int pos) {
    const int64_t blk = min(static_cast<unsigned>(__ldg(bt + pos / kBlock)), last_block);
    const int t = pos % kBlock;
    if constexpr (FP4) {
      const int off = q < 8 ? fp4_code_off(p.D, t, q * static_cast<int>(sizeof(V))) : fp4_scale_off(p.D, t, 0);
      return reinterpret_cast<V *>(base + blk * s0 + off);
    } else {
      return reinterpret_cast<V *>(base + blk * s0 + t * s2 + q * 16);
    }
  };
  // the first row that moves: kept[i] - i never falls
  int lo = 0, hi = p.budget;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldcg(kept + mid) == mid) lo = mid + 1;
    else hi = mid;
  }
  const int stretch = rows * kMoveUnroll;
  V v[kMoveUnroll], next[kMoveUnroll];
  int pos[kMoveUnroll];
  auto positions = [&](int i0) {
#pragma unroll
    for (int k = 0; k < kMoveUnroll; ++k) {
      const int i = i0 + k * rows + r;
      pos[k] = i < p.budget ? __ldcg(kept + i) : -1;
      if (pos[k] >= len) pos[k] = -1;
    }
  };
  auto read = [&](V (&to)[kMoveUnroll]) {
#pragma unroll
    for (int k = 0; k < kMoveUnroll; ++k)
      if (pos[k] >= 0) to[k] = __ldcg(place(pos[k]));
  };
  positions(lo);
  read(v);
  positions(lo + stretch);
  for (int i0 = lo; i0 < p.budget; i0 += stretch) {
    read(next);  // of rows behind everything this stretch writes
    positions(i0 + 2 * stretch);
    __syncthreads();  // every read of this stretch is done before its first write
#pragma unroll
    for (int k = 0; k < kMoveUnroll; ++k) {
      const int i = i0 + k * rows + r;
      if (i < p.budget) *place(i) = v[k];
      v[k] = next[k];
    }
  }
}

template <typename V, bool FP4>
cudaError_t launch_move(const EvictParams &p, int S, bool wide, cudaStream_t st) {
  const int x = p.pieces / p.slices;
  const dim3 grid(2 * p.slices, p.Hkv, S);
  return wide ? launch_pdl(move_kernel<V, FP4, 1024>, grid, dim3(x, 1024 / x), 0, st, 1, p)
                     : launch_pdl(move_kernel<V, FP4, 256>, grid, dim3(x, 256 / x), 0, st, 1, p);
}

}  // namespace
}  // namespace pa

using namespace pa;

PA_API int pa_evict(pa_tensor *k_cache, pa_tensor *v_cache, const pa_tensor *block_table, const pa_tensor *seq_lens,
                    const pa_tensor *weights, int budget, int recent, pa_tensor *kept, pa_tensor *new_seq_lens,
                    pa_tensor *new_weights, int *device_error, pa_stream_t stream) {
  int r;
  if ((r = check_desc(block_table, 2)) || (r = check_desc(seq_lens, 1)) || (r = check_desc(weights, 3)) ||
      (r = check_desc(kept, 3)) || (r = check_desc(new_seq_lens, 1)) || (r = check_desc(new_weights, 3)))
    return r;
  int NB, Hkv, D;
  if ((r = validate_cache_pair(k_cache, v_cache, &NB, &Hkv, &D))) return r;
  if (budget < 1 || recent < 0) return PA_ERR_INVALID_ARG;
  if (block_table->dtype != PA_I32 || seq_lens->dtype != PA_I32 || kept->dtype != PA_I32 ||
      new_seq_lens->dtype != PA_I32 || weights->dtype != PA_F32 || new_weights->dtype != PA_F32)
    return PA_ERR_UNSUPPORTED_DTYPE;
  const int cdt = k_cache->dtype;
  const bool fp4 = cdt == PA_FP4_E2M1;
  if (cdt != PA_F32 && cdt != PA_BF16 && cdt != PA_F16 && cdt != PA_FP8_E4M3 && !fp4) return PA_ERR_UNSUPPORTED_DTYPE;
  const int64_t S = seq_lens->shape[0], MB = block_table->shape[1], W = weights->shape[2];
  if (block_table->shape[0] != S || weights->shape[0] != S || kept->shape[0] != S || new_seq_lens->shape[0] != S ||
      new_weights->shape[0] != S)
    return PA_ERR_INVALID_ARG;
  if (weights->shape[1] != Hkv || kept->shape[1] != Hkv || new_weights->shape[1] != Hkv) return PA_ERR_INVALID_ARG;
  if (kept->shape[2] != budget || new_weights->shape[2] != W) return PA_ERR_INVALID_ARG;
  // (the kernels count positions in 32 bits, to less than 4096 past the last)
  if (S > 65535 || MB > INT32_MAX / kBlock || W > INT32_MAX - 4096 || budget > (1 << 30)) return PA_ERR_UNSUPPORTED_SHAPE;
  if (W < MB * kBlock) return PA_ERR_INVALID_ARG;
  if (block_table->stride[1] != 1 || seq_lens->stride[0] != 1 || weights->stride[2] != 1 || kept->stride[2] != 1 ||
      new_seq_lens->stride[0] != 1 || new_weights->stride[2] != 1)
    return PA_ERR_INVALID_ARG;
  if (rows_overlap(kept, budget) || rows_overlap(new_weights, W)) return PA_ERR_INVALID_ARG;
  const int eb = elem_bytes(cdt);
  if (!fp4 && (D <= 0 || (static_cast<int64_t>(D) * eb) % 16 || static_cast<int64_t>(D) * eb > 16 * 256))
    return PA_ERR_UNSUPPORTED_SHAPE;
  if (S == 0 || Hkv == 0) return PA_OK;
  if ((MB > 0 && !block_table->data) || !seq_lens->data || !kept->data || !new_seq_lens->data) return PA_ERR_INVALID_ARG;
  if (W > 0 && (!weights->data || !new_weights->data)) return PA_ERR_INVALID_ARG;
  for (const pa_tensor *t : {block_table, seq_lens, weights, static_cast<const pa_tensor *>(kept),
                             static_cast<const pa_tensor *>(new_seq_lens), static_cast<const pa_tensor *>(new_weights)})
    if (!on_elements(t)) return PA_ERR_ALIGNMENT;
  if (!aligned4(device_error)) return PA_ERR_ALIGNMENT;
  // read by every CTA of a sequence while others write the new ones
  if ((W > 0 && new_weights->data == weights->data) || new_seq_lens->data == seq_lens->data) return PA_ERR_INVALID_ARG;

  EvictParams p{};
  const pa_tensor *c[2] = {k_cache, v_cache};
  for (int i = 0; i < 2; ++i) {
    p.cache[i] = static_cast<char *>(c[i]->data);
    p.s0[i] = c[i]->stride[0] * eb;
    p.s1[i] = c[i]->stride[1] * eb;
    p.s2[i] = fp4 ? 0 : c[i]->stride[2] * eb;
  }
  p.block_table = static_cast<const int32_t *>(block_table->data);
  p.bt_ss = block_table->stride[0];
  p.seq_lens = static_cast<const int32_t *>(seq_lens->data);
  p.weights = static_cast<const float *>(weights->data);
  p.new_weights = static_cast<float *>(new_weights->data);
  p.w_ss = weights->stride[0];
  p.w_hs = weights->stride[1];
  p.nw_ss = new_weights->stride[0];
  p.nw_hs = new_weights->stride[1];
  p.kept = static_cast<int32_t *>(kept->data);
  p.k_ss = kept->stride[0];
  p.k_hs = kept->stride[1];
  p.new_lens = static_cast<int32_t *>(new_seq_lens->data);
  p.Hkv = Hkv;
  p.D = D;
  p.num_blocks = NB;
  p.max_blocks = static_cast<int>(MB);
  p.W = static_cast<int>(W);
  p.budget = budget;
  p.recent = recent;
  p.err = device_error;
  p.pieces = fp4 ? 9 : D * eb / 16;
  const int sm = device_sm_count();
  if (sm <= 0) return PA_ERR_CUDA;
  // Few (sequence, head) pairs: several CTAs share their rows, down to 64 bytes of a row each, or 32
  // where even so the CTAs are few (1 x 32768 tokens, one head, 16384 to stay: 57.2 us against 65.1;
  // with 8 heads 74.7 against 83.4; but 8 x 8..16k, 8 heads, 128 against 109).  There a CTA of 1024
  // threads moves longer stretches (64-byte slices, 256 threads: 82.9 and 108.6 us), and where there are no more pairs
  // than SMs, selects faster from more tokens than 256 threads hold (with 256: 118.7 and 161.3).
  const int64_t units = S * Hkv * 2;
  p.slices = 1;
  for (int n = 2; n * (fp4 ? 3 : 4) <= p.pieces && units * p.slices < 4 * sm; ++n)
    if (p.pieces % n == 0) p.slices = n;
  if (!fp4 && p.pieces % (2 * p.slices) == 0 && units * p.slices * 2 <= 2 * sm) p.slices *= 2;
  const bool wide_select = S * Hkv <= sm && MB * kBlock > 4096;
  const bool wide_move = units * p.slices <= 2 * sm && budget > 1024;

  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const dim3 grid(Hkv, static_cast<unsigned>(S));
  cudaError_t e = wide_select ? launch_pdl(select_kernel<1024>, grid, dim3(1024), 0, st, 1, p)
                              : launch_pdl(select_kernel<256>, grid, dim3(256), 0, st, 1, p);
  if (e == cudaSuccess) {
    const int n = static_cast<int>(S);
    e = !fp4 ? launch_move<uint4, false>(p, n, wide_move, st)
        : D == 64  ? launch_move<uint32_t, true>(p, n, wide_move, st)
        : D == 128 ? launch_move<uint2, true>(p, n, wide_move, st)
                   : launch_move<uint4, true>(p, n, wide_move, st);
  }
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
