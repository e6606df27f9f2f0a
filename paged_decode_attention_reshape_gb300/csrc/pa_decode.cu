// pa_decode.cu -- the fp32 decode path (CUDA cores), and the accumulation of attention weights.
#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_merge.cuh"

namespace pa {

// ---------------------------------------------------------------- fp32 path
//
// CUDA-core decode for fp32 caches (exact fp32 products; no 16-bit operand).
// Same work unit and merge as the tensor-core kernel.  Each warp walks its pages
// token by token: the 32 lanes hold D/32 strided elements of the K/V rows
// (coalesced 128-byte loads), one butterfly reduction per (token, head) gives
// the score, and the per-head online-softmax state is kept in registers.

// ACC: scores and softmax sums kept for pa_decode_accumulate.
template <int D, int W, bool ACC>
__global__ void __launch_bounds__(W * 32) decode_f32_kernel(const DecodeParams p) {
  constexpr int PER = D / 32;
  __shared__ float sm[W][8][D + 2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int s = blockIdx.z, part = blockIdx.x;
  const int g = blockIdx.y / p.HG, hg = blockIdx.y - g * p.HG;
  const int v0 = hg * 8;  // first column (virtual head) of this CTA, see DecodeParams
  int ng = min(8, p.VH - v0);
  const bool split = p.max_parts > 1;
  grid_dependency_wait();
  const int len = __ldg(p.seq_lens + s);
  if (len < 0 || len > p.max_blocks * kBlock) {
    if (threadIdx.x == 0 && part == 0 && blockIdx.y == 0 && p.err) atomicOr(p.err, kErrSeqLen);
    return;
  }
  int64_t row0 = s;  // the sequence's query tokens: one (decode) or rows qsl[s] .. qsl[s+1]-1
  int nq = 1;
  if (p.qsl) {
    const int a = __ldg(p.qsl + s), b = __ldg(p.qsl + s + 1);
    row0 = a;
    nq = b - a;
    if (a < 0 || b > p.Tq || nq < 0 || nq > p.nq_max || nq > len) {  // rows outside q / out, or too many
      if (threadIdx.x == 0 && part == 0 && blockIdx.y == 0 && p.err) atomicOr(p.err, kErrSeqLen);
      return;
    }
  }
  ng = min(ng, nq * p.G - v0);
  if (ng <= 0) return;
  const Cols cm{row0, p.G, g, v0};
  const int pos0 = len - nq;  // column hh sees the tokens up to pos0 + (v0 + hh) / G
  const int npages = (pos0 + (v0 + ng - 1) / p.G + 1 + kBlock - 1) / kBlock;
  const bool clustered = p.cluster > 1;  // rank `part` of a cluster splitting the unit equally
  const int pb = clustered ? static_cast<int>(static_cast<int64_t>(part) * npages / p.cluster) : part * p.pages_per_part;
  const int pe = clustered ? static_cast<int>(static_cast<int64_t>(part + 1) * npages / p.cluster)
                           : min(npages, pb + p.pages_per_part);
  if (pb >= pe && !clustered) {
    if (npages == 0 && part == 0)  // empty sequence (any split): zero output rows
      for (int i = threadIdx.x; i < ng * D; i += W * 32) static_cast<float *>(p.out)[cm.out_off(p, i / D) + i % D] = 0.f;
    return;
  }
  float q[8][PER], acc[8][PER], m[8], l[8], ab[8];
  int pos[8];
#pragma unroll
  for (int hh = 0; hh < 8; ++hh) {
    // last visible position (causal) and ALiBi slope in log2 units (0 without ALiBi):
    // logit += slope * (t - pos)
    pos[hh] = hh < ng ? pos0 + (v0 + hh) / p.G : -1;
    ab[hh] = (p.alibi && hh < ng) ? __ldg(p.alibi + cm.head(hh)) * 1.4426950408889634f : 0.f;
    const float *qr = static_cast<const float *>(p.q) + cm.q_off(p, min(hh, ng - 1));
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      q[hh][i] = hh < ng ? __ldg(qr + lane + 32 * i) : 0.f;
      acc[hh][i] = 0.f;
    }
    m[hh] = -INFINITY;
    l[hh] = 0.f;
  }
  bool bad = false;
  const int32_t *bt = p.block_table + static_cast<int64_t>(s) * p.bt_ss;
  for (int page = pb + warp; page < pe; page += W) {
    const int pid = __ldg(bt + page);
    if (pid < 0 || pid >= p.num_blocks) {
      bad = true;
      if (lane == 0 && p.err) atomicOr(p.err, kErrBlock);
      continue;
    }
    const int nv = min(kBlock, len - page * kBlock);
    const float *kbase = p.kc + static_cast<int64_t>(pid) * p.kc_s0 + static_cast<int64_t>(g) * p.kc_s1;
    const float *vbase = p.vc + static_cast<int64_t>(pid) * p.vc_s0 + static_cast<int64_t>(g) * p.vc_s1;
    for (int t = 0; t < nv; ++t) {
      float kr[PER], vr[PER];
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        kr[i] = __ldg(kbase + t * p.kc_s2 + lane + 32 * i);
        vr[i] = __ldg(vbase + t * p.vc_s2 + lane + 32 * i);
      }
      const int tt = page * kBlock + t;  // the token's position
#pragma unroll
      for (int hh = 0; hh < 8; ++hh) {
        if (tt <= pos[hh]) {  // visible to this column (never for hh >= ng)
          float z = 0.f;
#pragma unroll
          for (int i = 0; i < PER; ++i) z = fmaf(q[hh][i], kr[i], z);
#pragma unroll
          for (int off = 16; off > 0; off >>= 1) z += __shfl_xor_sync(0xffffffffu, z, off);
          z = fmaf(ab[hh], static_cast<float>(tt - pos[hh]), z * p.scale_log2);
          if (ACC && lane == 0)
            p.scores[((static_cast<int64_t>(s) * gridDim.y + blockIdx.y) * p.max_blocks * kBlock + tt) * p.score_cols + hh] = z;
          const float mn = fmaxf(m[hh], z);
          const float al = ex2(m[hh] - mn);
          const float pz = ex2(z - mn);
          l[hh] = l[hh] * al + pz;
#pragma unroll
          for (int i = 0; i < PER; ++i) acc[hh][i] = acc[hh][i] * al + pz * vr[i];
          m[hh] = mn;
        }
      }
    }
  }
#pragma unroll
  for (int hh = 0; hh < 8; ++hh) {
#pragma unroll
    for (int i = 0; i < PER; ++i) sm[warp][hh][lane + 32 * i] = acc[hh][i];
    if (lane == 0) {
      sm[warp][hh][D] = m[hh];
      sm[warp][hh][D + 1] = l[hh];
    }
  }
  const bool any_bad = __syncthreads_or(bad);
  if (clustered) {
    // CTA state in place over warp 0's slots (each element is read and overwritten by one thread)
    __shared__ float2 cmd[8];
    __shared__ int cbad;
    if (!any_bad) {
      for (int i = threadIdx.x; i < ng * D; i += W * 32) {
        const int hh = i / D, d = i - hh * D;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < W; ++w) M = fmaxf(M, sm[w][hh][D]);
        float num = 0.f, den = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const float mw = sm[w][hh][D];
          const float sc = (mw == -INFINITY) ? 0.f : ex2(mw - M);
          den += sc * sm[w][hh][D + 1];
          num += sc * sm[w][hh][d];
        }
        sm[0][hh][d] = num;
        if (d == 0) cmd[hh] = make_float2(M, den);
      }
    }
    cluster_merge_write<float, D>(p, cm, ng, 1.f, any_bad, &sm[0][0][0], D + 2, cmd, &cbad, W * 32);
    return;
  }
  const int nparts = split ? (npages + p.pages_per_part - 1) / p.pages_per_part : 1;
  const bool direct = nparts == 1;
  const FixedRows rows{(static_cast<int64_t>(s) * p.Hkv + g) * p.VH + v0, p.max_parts};
  if (!any_bad) {
    for (int i = threadIdx.x; i < ng * D; i += W * 32) {
      const int hh = i / D, d = i - hh * D;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < W; ++w) M = fmaxf(M, sm[w][hh][D]);
      float num = 0.f, den = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float mw = sm[w][hh][D];
        const float sc = (mw == -INFINITY) ? 0.f : ex2(mw - M);
        den += sc * sm[w][hh][D + 1];
        num += sc * sm[w][hh][d];
      }
      if (direct) {
        static_cast<float *>(p.out)[cm.out_off(p, hh) + d] = den > 0.f ? num / den : 0.f;
        if (ACC && d == 0) p.lse[cm.row(hh) * p.Hq + cm.head(hh)] = log_total(M, den);
      } else {
        const int64_t row = rows(hh, part);
        p.part_acc[row * D + d] = num;
        if (d == 0) p.part_ml[row] = make_float2(M, den);
      }
    }
  }
  if (ACC && any_bad && direct) drop_lse(p, cm, ng);
  static_assert(sizeof(sm) >= 8 * kMergeSmemParts * 4, "merge weights reuse sm");
  if (!direct)
    merge_if_last<float, D, ACC>(p, cm, static_cast<int>(blockIdx.y) + p.Hkv * p.HG * s, ng, nparts, 1.f, any_bad,
                            W * 32, &sm[0][0][0], rows);
}

namespace {
template <bool ACC>
cudaError_t launch_f32(const DecodeParams &p, cudaStream_t st) {
  const dim3 grid(p.max_parts, p.Hkv * p.HG, p.S);
  cudaError_t e;
  switch (p.D) {
    case 64: e = launch_pdl(decode_f32_kernel<64, 4, ACC>, grid, dim3(128), 0, st, p.cluster, p); break;
    case 128: e = launch_pdl(decode_f32_kernel<128, 4, ACC>, grid, dim3(128), 0, st, p.cluster, p); break;
    case 256: e = launch_pdl(decode_f32_kernel<256, 2, ACC>, grid, dim3(64), 0, st, p.cluster, p); break;
    default: return cudaErrorInvalidValue;
  }
  return e != cudaSuccess ? e : cudaGetLastError();
}
}  // namespace

cudaError_t launch_decode_f32(const DecodeParams &p, cudaStream_t st) {
  return p.scores ? launch_f32<true>(p, st) : launch_f32<false>(p, st);
}

// ------------------------------------------------- accumulated attention weights
//
// weights[s, g, t] += sum over the query heads h of KV head g of 2^(score_h,t - lse_h), the
// attention weight of token t: the decode kernels have left every score (log2 units) and
// every head's log2 of the softmax sum, which is known only after the last page, in the
// workspace (+inf for a head without a positive sum, which adds nothing; NaN for one whose unit set an
// error, as a timed-out wait may in one KV head alone: the sequence adds nothing).  Scores are stored
// token by token, the group's columns together, so a thread reads one 16- or 32-byte run per token and
// adjacent threads adjacent runs.  Keeping the
// scores costs 4 bytes a (query head, token) each way, mostly served by L2, against a second
// read of every K page (2 D bytes a (KV head, token) for a 16-bit cache).
constexpr int kWeightTokens = 4;  // tokens in flight per thread (one: 32 us on 64 x 1k..8k tokens, 8 KV heads)
template <int CW>
__global__ void __launch_bounds__(256) weights_kernel(const WeightsParams p) {
  const int s = blockIdx.z, g = blockIdx.y;
  grid_dependency_wait();
  const int len = __ldg(p.seq_lens + s);
  if (len <= 0 || len > p.max_tokens) return;  // (out of range: reported by the decode)
  const float *row = p.lse + static_cast<int64_t>(s) * p.Hkv * p.G;
  bool failed = false;
  for (int h = threadIdx.x; h < p.Hkv * p.G; h += 256) {
    const float x = __ldcg(row + h);
    failed |= x != x;
  }
  float *w = p.weights + s * p.w_ss + g * p.w_hs;
  const int64_t unit0 = (static_cast<int64_t>(s) * p.Hkv + g) * p.HG;
  const int first = blockIdx.x * (256 * kWeightTokens);
  for (int b0 = first; b0 < len; b0 += gridDim.x * (256 * kWeightTokens)) {
    const int t0 = b0 + threadIdx.x;
    float sum[kWeightTokens], old[kWeightTokens];
#pragma unroll
    for (int k = 0; k < kWeightTokens; ++k) {
      sum[k] = 0.f;
      old[k] = t0 + 256 * k < len ? w[t0 + 256 * k] : 0.f;
    }
    for (int hg = 0; hg < p.HG; ++hg) {
      const float *sc = p.scores + (unit0 + hg) * p.max_tokens * CW;
      const float *lse = row + g * p.G + hg * 8;
      const int n = min(CW, p.G - hg * 8);
      float v[kWeightTokens][CW], ls[CW];
#pragma unroll
      for (int k = 0; k < kWeightTokens; ++k) {
        if (t0 + 256 * k >= len) continue;
        const float *x = sc + static_cast<int64_t>(t0 + 256 * k) * CW;
        if constexpr (CW >= 4) {
#pragma unroll
          for (int i = 0; i < CW / 4; ++i) {
            const float4 f = __ldcg(reinterpret_cast<const float4 *>(x) + i);
            v[k][4 * i] = f.x;
            v[k][4 * i + 1] = f.y;
            v[k][4 * i + 2] = f.z;
            v[k][4 * i + 3] = f.w;
          }
        } else {
#pragma unroll
          for (int i = 0; i < CW; ++i) v[k][i] = __ldcg(x + i);
        }
      }
#pragma unroll
      for (int i = 0; i < CW; ++i) ls[i] = i < n ? __ldcg(lse + i) : INFINITY;
      // a column without a sum is left out here, not by the exponent: its scores may be NaN or +inf
#pragma unroll
      for (int k = 0; k < kWeightTokens; ++k)
#pragma unroll
        for (int i = 0; i < CW; ++i)
          if (ls[i] < INFINITY && t0 + 256 * k < len) sum[k] += ex2(v[k][i] - ls[i]);
    }
    if (b0 == first && __syncthreads_or(failed)) return;  // (here: behind the loads)
#pragma unroll
    for (int k = 0; k < kWeightTokens; ++k)
      if (t0 + 256 * k < len) w[t0 + 256 * k] = old[k] + sum[k];
  }
}

cudaError_t launch_weights(const WeightsParams &p, int cols, cudaStream_t st) {
  const int64_t blocks = (static_cast<int64_t>(p.max_tokens) + 256 * kWeightTokens - 1) / (256 * kWeightTokens);
  const dim3 grid(static_cast<unsigned>(blocks < 65535 ? blocks : 65535), p.Hkv, p.S);
  switch (cols) {
    case 1: return launch_pdl(weights_kernel<1>, grid, dim3(256), 0, st, 1, p);
    case 2: return launch_pdl(weights_kernel<2>, grid, dim3(256), 0, st, 1, p);
    case 4: return launch_pdl(weights_kernel<4>, grid, dim3(256), 0, st, 1, p);
    case 8: return launch_pdl(weights_kernel<8>, grid, dim3(256), 0, st, 1, p);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pa
