// pa_decode_fp4_warps.cuh -- single-query decode over 4-bit pages, split evenly over the warps of
// one resident wave.
//
// A 4-bit page pair takes an SM 100 clocks at HBM rate, so a CTA per (sequence, KV head) spends
// much of its life not reading: waiting for its length, its table and its first pages, and
// leaving its slot to the next (304 x 256 tokens, 8 KV heads of 128, eight waves of CTAs: 42.1 us,
// where HBM alone takes 14).  Here every warp works by itself.  The stages (pa_decode_fp4.cuh) of all sequences,
// concatenated, are cut into equal ranges, one per warp of each head row (KV head and group of 8
// query heads); a range may begin and end inside sequences.  Copies run ahead over the whole
// range, across sequences, so they never pause; nothing waits for another warp.
//
// A sequence that one warp holds whole is written from its registers.  The parts of a cut one are
// merged, in order, by the warp that arrives last at the unit's counter (so the result does not
// depend on which it is).  The warps of a CTA have neighbouring ranges, and where all of a unit's
// parts are its own they meet in shared memory: a part that ends a warp's range lies in the
// warp's stage buffers, free by then, and the one that begins a range and is followed by others
// in the workspace.  Parts of several CTAs all go through the workspace (store, release, counter,
// and a merge by the last): the split pays where most units stay whole.
// Measured: 304 x 256 tokens 22.1 us; 256 x 512..4096 135.6 us against 156.8 for a CTA per unit, HBM
// alone 101; but 64 x 0..2048 (head size 64, five parts a unit) 23.1 against 18.2.
#pragma once

#include "pa_decode_mma.cuh"

namespace pa {

// Least stages of a warp's range (while the batch has more): shorter ones cost more parts to merge
// than they save.
constexpr int kMinWarpStages = 2;

// The lane's share of an output or state row: heads 2qc and 2qc + 1 (c = 0, 1) of the group, per
// section b the RUN consecutive elements from 128 b + RUN ra on.
template <typename C, int D>
struct Fp4Lane {
  static constexpr int RUN = D >= 128 ? 16 : 8;
  static constexpr int TPS = RUN / 2;  // accumulator tiles of a section
  static __device__ __forceinline__ int first(int b) { return 128 * b + RUN * ((threadIdx.x & 31) >> 2); }
  // element e of section b, column c
  static __device__ __forceinline__ float get(const float (&acc)[C::KT][4], int b, int e, int c) {
    return acc[b * TPS + (e >> 1)][2 * (e & 1) + c];
  }
  static __device__ __forceinline__ float &ref(float (&acc)[C::KT][4], int b, int e, int c) {
    return acc[b * TPS + (e >> 1)][2 * (e & 1) + c];
  }
  // out = acc * f[c]
  template <typename OutT>
  static __device__ __forceinline__ void write(const DecodeParams &p, const Cols &cm, int ng,
                                               const float (&acc)[C::KT][4], const float (&f)[2]) {
    const int qc = threadIdx.x & 3;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int hh = 2 * qc + c;
      if (hh >= ng) continue;
      OutT *o = static_cast<OutT *>(p.out) + cm.out_off(p, hh);
#pragma unroll
      for (int b = 0; b < C::QB; ++b) {
#pragma unroll
        for (int e = 0; e < RUN; e += 8) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float x = get(acc, b, e + 2 * i, c) * f[c], y = get(acc, b, e + 2 * i + 1, c) * f[c];
            w[i] = C::QBF16 ? pack_bf16(x, y) : pack_f16(x, y);
          }
          *reinterpret_cast<uint4 *>(o + first(b) + e) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
  }
};

template <int KIND, int D, int W, int STAGES, bool ACC>
__global__ void __launch_bounds__(W * 32, mma_min_ctas(KIND, D)) decode_fp4_warps_kernel(const DecodeParams p) {
  using C = MmaCfg<KIND, D, W, STAGES>;
  using Lane = Fp4Lane<C, D>;
  using OutT = typename std::conditional<C::QBF16, __nv_bfloat16, __half>::type;
  constexpr int NP = C::NP;
  constexpr int PER = 32 / NP;  // stages whose table entries the warp's lanes hold at a time
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_u32 = smem_u32(smem_raw);
  const uint32_t sbase = (raw_u32 + 1023u) & ~1023u;
  uint8_t *const sgen = smem_raw + (sbase - raw_u32);
  int *const pref = reinterpret_cast<int *>(sgen + C::SCRATCH_OFF);  // stage offsets of the sequences [S + 1]
  __shared__ int s_wsum[W];
  __shared__ int s_len[kFlatMaxSeqs + 1];  // lengths, 0 for an invalid one
  __shared__ int s_arrived[W];             // counters of the units whose first part is warp w's, all parts this CTA's
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ra = lane >> 2, qc = lane & 3;

  if (threadIdx.x * 32 < p.S) prefetch_l2(p.seq_lens + threadIdx.x * 32);
  grid_dependency_wait();
  {
    constexpr int PERT = (kFlatMaxSeqs + C::THREADS - 1) / C::THREADS;
    const int i0 = threadIdx.x * PERT;
    int n[PERT], sum = 0;
#pragma unroll
    for (int j = 0; j < PERT; ++j) {
      const int i = i0 + j;
      const int L = i < p.S ? __ldg(p.seq_lens + i) : 0;
      const bool ok = L >= 0 && L <= p.max_blocks * kBlock;
      if (!ok && blockIdx.x == 0 && p.err) atomicOr(p.err, kErrSeqLen);
      n[j] = ok ? (L + NP * kBlock - 1) / (NP * kBlock) : 0;
      if (i < p.S) s_len[i] = ok ? L : 0;
      sum += n[j];
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += t;
    }
    if (lane == 31) s_wsum[warp] = incl;
    if (lane == 0) s_arrived[warp] = 0;
    __syncthreads();
    int run = incl - sum, total = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const int v = s_wsum[w];
      run += w < warp ? v : 0;
      total += v;
    }
#pragma unroll
    for (int j = 0; j < PERT; ++j) {
      if (i0 + j < p.S) pref[i0 + j] = run;
      run += n[j];
    }
    if (threadIdx.x == 0) pref[p.S] = total;
    __syncthreads();
  }
  // this warp: worker c of head row `row`; a CTA's warps are neighbours
  const int rows = p.Hkv * p.HG;
  const int row = static_cast<int>(blockIdx.x) % rows, cta0 = static_cast<int>(blockIdx.x) / rows * W, c = cta0 + warp;
  const int g = row / p.HG, v0 = (row - g * p.HG) * 8;
  const int ng = min(8, p.G - v0);
  if (cta0 >= p.flat) return;
  for (int z = c; z < p.S; z += p.flat) {  // empty sequences: zero output rows
    if (pref[z] == pref[z + 1] && __ldg(p.seq_lens + z) == 0) {
      const Cols cm{z, p.G, g, v0};
      for (int i = lane; i < ng * D; i += 32) static_cast<OutT *>(p.out)[cm.out_off(p, i / D) + i % D] = OutT(0.f);
    }
  }
  const int T = pref[p.S];
  const int Ce = min(p.flat, T / kMinWarpStages + 1);  // workers with a range
  auto range_start = [&](int w) { return static_cast<int>(static_cast<int64_t>(w) * T / Ce); };
  auto owner = [&](int x) { return static_cast<int>((static_cast<int64_t>(x + 1) * Ce - 1) / T); };
  if (c >= Ce) return;
  const int a = range_start(c), b = range_start(c + 1), n = b - a;
  if (n <= 0) return;
  auto sequence = [&](int x) {  // the sequence holding stage x: the last z with pref[z] <= x
    int z = 0, hi = p.S - 1;
    while (z < hi) {
      const int mid = (z + hi + 1) >> 1;
      if (pref[mid] <= x) z = mid;
      else hi = mid - 1;
    }
    return z;
  };

  const uint64_t pol = policy_evict_first();
  const uint32_t stage0 = sbase + static_cast<uint32_t>(warp * STAGES * C::STAGEB);
  // Table entries of PER stages, one page per lane, and those of the next PER, read a batch ahead.
  // A page behind its sequence's end reads as block 0, a bad entry as -1 (its copy takes block 0).
  auto load_entries = [&](int k) {
    int e = 0;
    if (k + lane / NP < n) {
      const int x = a + k + lane / NP, z = sequence(x), page = (x - pref[z]) * NP + lane % NP;
      if (page * kBlock < s_len[z]) e = __ldg(p.block_table + static_cast<int64_t>(z) * p.bt_ss + page);
    }
    return e;
  };
  const Fp4Copies<C, D> copies(p, g, lane);
  int entry = 0, entry_next = load_entries(0);
  uint32_t bad_now = 0, bad_before = 0;  // lanes with a bad entry, of the batch being issued and the one before
  auto issue = [&](int k) {
    const int at = k % PER;
    if (at == 0) {
      const bool out = entry_next < 0 || entry_next >= p.num_blocks;
      if (out && p.err) atomicOr(p.err, kErrBlock);
      bad_before = bad_now;
      bad_now = __ballot_sync(0xffffffffu, out);
      entry = out ? 0 : entry_next;
      if (k + PER < n) entry_next = load_entries(k + PER);
    }
    copies.stage(stage0 + k % STAGES * C::STAGEB, entry, at * NP, pol);
    copy_commit();
  };
#pragma unroll
  for (int k = 0; k < STAGES; ++k) {
    if (k < n) issue(k);
    else copy_commit();
  }

  Fp4State<C, D, true> state;
  state.place(stage0);
  const float vs = p.v_scale ? __ldg(p.v_scale + g * p.scale_stride) : 1.f;
  int z = sequence(a);
  for (int k = 0; k < n;) {
    // one sequence's part of the range: stages x0 .. x1 - 1
    const int ps = pref[z], pn = pref[z + 1];
    const int x0 = a + k, x1 = min(b, pn);
    const int len = s_len[z];
    const Cols cm{z, p.G, g, v0};
    state.begin(p, cm, ng, len - 1, len);
    float *score_lane = nullptr;
    if constexpr (ACC) score_lane = fp4_score_lane(p, z, row);
    bool bad = false;
    for (; a + k < x1; ++k) {
      copy_wait<STAGES - 1>();
      __syncwarp();
      if (bad_now | bad_before) {  // (rare) this stage's lanes, in the batch it was issued with
        const int issued = min(k + STAGES - 1, n - 1) / PER;
        bad |= (((k / PER == issued ? bad_now : bad_before) >> (k % PER * NP)) & ((1u << NP) - 1)) != 0;
      }
      const int tok0 = (a + k - ps) * NP * kBlock;
      state.template any_stage<ACC>(p, k % STAGES * C::STAGEB, tok0, len - tok0, score_lane);
      __syncwarp();  // every lane has read the stage
      if (k + STAGES < n) issue(k + STAGES);
      else copy_commit();
    }
    float l0 = state.l0, l1 = state.l1;
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, o);
      l1 += __shfl_xor_sync(0xffffffffu, l1, o);
    }
    if (x0 == ps && x1 == pn) {  // the whole sequence
      if (!bad) {
        const float f[2] = {l0 > 0.f ? vs / l0 : 0.f, l1 > 0.f ? vs / l1 : 0.f};
        Lane::template write<OutT>(p, cm, ng, state.acc, f);
      }
      if constexpr (ACC) {
        if (ra == 0) {
          if (2 * qc < ng) p.lse[cm.row(2 * qc) * p.Hq + cm.head(2 * qc)] = bad ? log_failed() : log_total(state.m0, l0);
          if (2 * qc + 1 < ng)
            p.lse[cm.row(2 * qc + 1) * p.Hq + cm.head(2 * qc + 1)] = bad ? log_failed() : log_total(state.m1, l1);
        }
      }
    } else {
      // a part: its state away, then the unit's counter; the last to arrive merges
      const int c0 = owner(ps), c1 = owner(pn - 1), nparts = c1 - c0 + 1;
      const bool local = c0 >= cta0 && c1 < cta0 + W;
      auto group = [&](int i) {  // workspace row group of the unit's i-th part: its worker, first or last range
        return (static_cast<int64_t>(row) * p.flat + c0 + i) * 2 + (i == 0 && range_start(c0) < ps ? 1 : 0);
      };
      auto in_smem = [&](int i) { return local && (i < nparts - 1 || range_start(c1 + 1) == pn); };
      if (in_smem(c - c0)) {
        store_warp_state<C, D, STAGES>(sgen, state.m0, state.m1, state.l0, state.l1, state.acc);
      } else if (!bad) {
        const int64_t r0 = group(c - c0) * 8;
        if (ra == 0) {
          p.part_ml[r0 + 2 * qc] = make_float2(state.m0, l0);
          p.part_ml[r0 + 2 * qc + 1] = make_float2(state.m1, l1);
        }
#pragma unroll
        for (int cc = 0; cc < 2; ++cc) {
          float *d = p.part_acc + (r0 + 2 * qc + cc) * D;
#pragma unroll
          for (int s = 0; s < C::QB; ++s)
#pragma unroll
            for (int e = 0; e < Lane::RUN; e += 4)
              *reinterpret_cast<float4 *>(d + Lane::first(s) + e) =
                  make_float4(Lane::get(state.acc, s, e, cc), Lane::get(state.acc, s, e + 1, cc),
                              Lane::get(state.acc, s, e + 2, cc), Lane::get(state.acc, s, e + 3, cc));
        }
      }
      __syncwarp();  // the warp's stores precede lane 0's release below
      int old = 0;
      if (lane == 0) {
        // release: this part's state before the arrival; acquire: the last one sees every other part's
        if (local) {
          const uint32_t at = smem_u32(s_arrived + (c0 - cta0));
          if (bad) asm volatile("red.or.relaxed.cta.shared.b32 [%0], %1;" ::"r"(at), "r"(kUnitBad) : "memory");
          asm volatile("atom.add.acq_rel.cta.shared.s32 %0, [%1], 1;" : "=r"(old) : "r"(at) : "memory");
        } else {
          int *at = p.counters + z * rows + row;
          if (bad) atomicOr(at, kUnitBad);
          asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(old) : "l"(at) : "memory");
          if ((old & kArrivalMask) == nparts - 1) atomicExch(at, 0);
        }
      }
      old = __shfl_sync(0xffffffffu, old, 0);
      __syncwarp();
      if ((old & kArrivalMask) == nparts - 1) {
        const bool unit_bad = (old & kUnitBad) || bad;
        float M0 = -INFINITY, M1 = -INFINITY, den0 = 0.f, den1 = 0.f;
        if (!unit_bad) {
          // part i's (max, sum) pairs and accumulator rows; what another CTA wrote is read past L1
          auto region = [&](int i) {
            return reinterpret_cast<const float *>(sgen + (c0 + i - cta0) * STAGES * C::STAGEB);
          };
          auto load = [&](const float *x) {
            return local ? *reinterpret_cast<const float4 *>(x) : __ldcg(reinterpret_cast<const float4 *>(x));
          };
          auto ml = [&](int i) {
            return load((in_smem(i) ? region(i) : reinterpret_cast<const float *>(p.part_ml + group(i) * 8)) + 4 * qc);
          };
          for (int i = 0; i < nparts; ++i) {
            const float4 v = ml(i);
            M0 = fmaxf(M0, v.x);
            M1 = fmaxf(M1, v.z);
          }
          float (&acc)[C::KT][4] = state.acc;  // (this part's own state is away, with the others)
#pragma unroll
          for (int t = 0; t < C::KT; ++t) acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0.f;
          auto add = [&](int s, int e, int cc, float w, const float4 &x) {
            Lane::ref(acc, s, e, cc) += w * x.x;
            Lane::ref(acc, s, e + 1, cc) += w * x.y;
            Lane::ref(acc, s, e + 2, cc) += w * x.z;
            Lane::ref(acc, s, e + 3, cc) += w * x.w;
          };
          // several parts' loads at once: a part's row is 1 to 4 kB a warp, a trip to L2 about a microsecond
          constexpr int AT = D == 64 ? 2 : 1, NV = Lane::RUN / 4;
          for (int i0 = 0; i0 < nparts; i0 += AT) {
            float4 v[AT], x[AT][C::QB][2][NV];
#pragma unroll
            for (int u = 0; u < AT; ++u) {
              const int i = min(i0 + u, nparts - 1);
              const bool smem = in_smem(i);
              const float *rows_i = smem ? region(i) + 16 : p.part_acc + group(i) * 8 * D;
              v[u] = ml(i);
#pragma unroll
              for (int s = 0; s < C::QB; ++s)
#pragma unroll
                for (int cc = 0; cc < 2; ++cc)
#pragma unroll
                  for (int e = 0; e < NV; ++e)
                    x[u][s][cc][e] = load(rows_i + (2 * qc + cc) * (smem ? C::SROW : D) + Lane::first(s) + 4 * e);
            }
#pragma unroll
            for (int u = 0; u < AT; ++u) {
              if (i0 + u >= nparts) break;
              const float w[2] = {ex2(v[u].x - M0), ex2(v[u].z - M1)};
              den0 += w[0] * v[u].y;
              den1 += w[1] * v[u].w;
#pragma unroll
              for (int s = 0; s < C::QB; ++s)
#pragma unroll
                for (int cc = 0; cc < 2; ++cc)
#pragma unroll
                  for (int e = 0; e < NV; ++e) add(s, 4 * e, cc, w[cc], x[u][s][cc][e]);
            }
          }
          const float f[2] = {den0 > 0.f ? vs / den0 : 0.f, den1 > 0.f ? vs / den1 : 0.f};
          Lane::template write<OutT>(p, cm, ng, acc, f);
        }
        if constexpr (ACC) {
          if (ra == 0) {
            if (2 * qc < ng) p.lse[cm.row(2 * qc) * p.Hq + cm.head(2 * qc)] = unit_bad ? log_failed() : log_total(M0, den0);
            if (2 * qc + 1 < ng)
              p.lse[cm.row(2 * qc + 1) * p.Hq + cm.head(2 * qc + 1)] = unit_bad ? log_failed() : log_total(M1, den1);
          }
        }
      }
    }
    if (k < n) {
      do ++z;
      while (pref[z + 1] == pref[z]);  // next non-empty sequence (one exists: the range goes on)
    }
  }
}

// Host side of one (kind, head size).
template <int KIND, int D>
struct Fp4WarpsLaunch {
  static constexpr int W = mma_warps(KIND, D), ST = mma_stages(KIND, D);
  using C = MmaCfg<KIND, D, W, ST>;
  template <bool ACC>
  static cudaError_t launch_variant(const DecodeParams &p, int ctas, cudaStream_t st) {
    auto kern = decode_fp4_warps_kernel<KIND, D, W, ST, ACC>;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = once_per_device(done, [kern] {
      cudaError_t r = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(C::SMEM));
      if (r != cudaSuccess) return r;
      return cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    });
    if (e != cudaSuccess) return e;
    e = launch_pdl(kern, dim3(ctas), dim3(C::THREADS), C::SMEM, st, 1, p);
    return e != cudaSuccess ? e : cudaGetLastError();
  }
  static cudaError_t launch(const DecodeParams &p, int ctas, cudaStream_t st) {
    return p.scores ? launch_variant<true>(p, ctas, st) : launch_variant<false>(p, ctas, st);
  }
};

}  // namespace pa
