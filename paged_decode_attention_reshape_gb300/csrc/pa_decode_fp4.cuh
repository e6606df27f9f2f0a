// pa_decode_fp4.cuh -- the page loop of the tensor-core decode over 4-bit (E2M1) pages; the work
// split, the merges and the variants are pa_decode_mma.cuh's.
//
// A stage is NP pages of K and of V (two; four at head size 64, one at 256), brought by 16-byte asynchronous
// copies: a page's codes are whole 512-byte runs of the warp, and the scales of the stage's 2 NP
// pages share the last ones, so a stage of head size 128 costs nine copies and five addresses.
// (One bulk copy per page and a barrier per stage: 147.5 against 135.6 us on 128 x 1k..8k tokens,
// 64/8 heads, when P had one half.)  At HBM rate an SM has to take 23 bytes, 41 elements, a clock, and
// the widening alone is half a conversion an element on a pipe that does 64 lanes a clock (measured, and shared
// with bit selects and shuffles of bytes), so the loop is built to do little else, 292 warp
// instructions a page pair at head size 128:
//
//   K: lane (r, c) holds a run of 32 (D = 64: 16) elements of tokens r and r + 8, whole scale
//      groups.  Codes are widened to f16x2 (cvt e2m1x2), each pair multiplied by its group's
//      scale (E4M3 widened to f16; exact: at most 6 significant bits, 2^-10 .. 2688), and fed
//      to the f16 tensor cores against the query, which uses the same order of elements.
//   V: lane (r, c) holds a run of 16 (D = 64: 8) elements, inside one scale group, of tokens
//      2c, 2c + 1, 2c + 8, 2c + 9.  The product contracts over tokens, so the nibbles of two
//      tokens are first brought into one byte (t0 | t1 << 4; a shift and a bit select per
//      four pairs), and one conversion gives the pair.
//   Softmax: as pa_decode_mma.cuh, in log2 units, one vote per stage.  The running maximum is kept
//      2^kLift below the largest score, so p reaches 2^15 (f16 holds 65504) and the smallest p
//      an f16 tells from zero is 2^-24 of 2^7, not of 1.
//   P: f16, in two halves (22 bits; a second product adds the rest), as the 16-bit caches' kernels
//      hold it.  One half, 11 bits, would do without that product (128 x 1k..8k tokens, 64/8 heads:
//      121 us against 136), but moves every weight by up to 2^-12 of itself: the outputs of that case
//      were 8e-4 of their norm from a plain fp32 form's instead of 7e-5, and where large terms
//      cancel the error is all there is.
//
// Tokens behind the end exist only in a range's last stage, which takes a branch of its own:
// scores -inf, p = 0 and V scales 0 (codes are always finite), so nothing stale is summed.
#pragma once

namespace pa {

constexpr float kLift = 7.f;       // log2 units the running maximum is kept below the scores'
constexpr float kFp4Slack = 15.f;  // p <= 2^15

// A lane's share of a stage's copies: 16 bytes of every 512 of a page's codes, and 16 bytes of the
// scales of one of the stage's pages (K pages first, as they lie in the stage).
template <typename C, int D>
struct Fp4Copies {
  static constexpr int NP = C::NP;
  static constexpr int CODEB = 8 * D;                // code bytes of a page: whole runs of 512
  static constexpr int SL = D / 16;                  // lanes for a page's scales
  static constexpr int SPAGES = 32 / SL;             // pages whose scales one copy takes
  static constexpr int SRUNS = 2 * NP / SPAGES;      // copies for a stage's scales
  static_assert(CODEB % 512 == 0 && SRUNS * SPAGES == 2 * NP, "copy shares");
  const char *kbase, *vbase;
  uint32_t ks0, vs0;  // block strides (below 2^32)
  int lane;
  __device__ __forceinline__ Fp4Copies(const DecodeParams &p, int g, int lane_)
      : kbase(p.k4 + g * p.kc_s1), vbase(p.v4 + g * p.vc_s1), ks0(static_cast<uint32_t>(p.kc_s0)),
        vs0(static_cast<uint32_t>(p.vc_s0)), lane(lane_) {}
  // Whole warp: the stage at shared address dst, its pages' blocks in lanes at .. at + NP - 1 of entry.
  __device__ __forceinline__ void stage(uint32_t dst, int entry, int at, uint64_t pol) const {
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const uint32_t blk = static_cast<uint32_t>(__shfl_sync(0xffffffffu, entry, at + j));
      const char *ks = kbase + lane * 16 + static_cast<uint64_t>(blk) * ks0;
      const char *vs = vbase + lane * 16 + static_cast<uint64_t>(blk) * vs0;
#pragma unroll
      for (int i = 0; i < CODEB / 512; ++i) {
        copy16_async(dst + j * C::PAGEB + i * 512 + lane * 16, ks + i * 512, pol);
        copy16_async(dst + (NP + j) * C::PAGEB + i * 512 + lane * 16, vs + i * 512, pol);
      }
    }
#pragma unroll
    for (int i = 0; i < SRUNS; ++i) {
      const int pg = i * SPAGES + lane / SL;  // page of the stage: K 0 .. NP - 1, V 0 .. NP - 1
      const uint32_t blk = static_cast<uint32_t>(__shfl_sync(0xffffffffu, entry, at + pg % NP));
      const char *src = (pg < NP ? kbase : vbase) + static_cast<uint64_t>(blk) * (pg < NP ? ks0 : vs0);
      copy16_async(dst + pg * C::PAGEB + CODEB + (lane % SL) * 16, src + CODEB + (lane % SL) * 16, pol);
    }
  }
};

// ACC: this lane's place in the first page of scores of head row `row` of sequence s.
__device__ __forceinline__ float *fp4_score_lane(const DecodeParams &p, int s, int row) {
  const int lane = threadIdx.x & 31;
  return p.scores +
         ((static_cast<int64_t>(s) * (p.Hkv * p.HG) + row) * p.max_blocks * kBlock + (lane >> 2)) * p.score_cols +
         2 * (lane & 3);
}

// One warp's attention over the stages of a range: query fragments, softmax state, accumulator, and
// the places its lane reads in a stage.
template <typename C, int D, bool PLAIN>
struct Fp4State {
  static constexpr int NP = C::NP;
  using Rows = Fp4Rows<D>;
  using Runs = Fp4Runs<D>;
  uint32_t qf[C::KT][2];
  float sc0, sc1;  // score scale (log2 units) of the lane's columns 2qc, 2qc + 1; never negative
  float acc[C::KT][4];
  float m0, m1, l0, l1;
  int posA, posB, seeA, seeB;  // not PLAIN: the columns' positions, and the last tokens they see here
  float ab0, ab1;              // not PLAIN: ALiBi slopes (log2 units)
  int ra, qc, kon8, von8, vodd;
  uint32_t kcode0, kscale0, vcode0, vscale0;

  // stage0: shared address of the warp's first stage
  __device__ __forceinline__ void place(uint32_t stage0) {
    ra = (threadIdx.x & 31) >> 2;
    qc = threadIdx.x & 3;
    kon8 = Rows::on8(Rows::code_lane(ra, qc));
    von8 = Rows::on8(Runs::code_lane(ra, qc));
    vodd = Runs::odd(Runs::code_lane(ra, qc));
    kcode0 = stage0 + Rows::code_lane(ra, qc);
    kscale0 = stage0 + Rows::scale_lane(ra, qc);
    vcode0 = stage0 + NP * C::PAGEB + Runs::code_lane(ra, qc);
    vscale0 = stage0 + NP * C::PAGEB + Runs::scale_lane(ra, qc);
  }
  // A range that ends before token `end`, for columns 0 .. ng - 1 of cm, the first query at pos0.
  __device__ __forceinline__ void begin(const DecodeParams &p, const Cols &cm, int ng, int pos0, int end) {
    load_query<C, D>(p, cm, ng, qf, sc0, sc1);
#pragma unroll
    for (int t = 0; t < C::KT; ++t) acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0.f;
    m0 = m1 = kEmptyMax;
    l0 = l1 = 0.f;
    ab0 = ab1 = 0.f;
    if constexpr (!PLAIN) {
      posA = 2 * qc < ng ? pos0 + (cm.v0 + 2 * qc) / cm.G : -1;
      posB = 2 * qc + 1 < ng ? pos0 + (cm.v0 + 2 * qc + 1) / cm.G : -1;
      seeA = min(posA, end - 1);  // (tokens from `end` on are another range's, or nobody's)
      seeB = min(posB, end - 1);
      if (p.alibi) {
        if (2 * qc < ng) ab0 = __ldg(p.alibi + cm.head(2 * qc)) * kLog2e;
        if (2 * qc + 1 < ng) ab1 = __ldg(p.alibi + cm.head(2 * qc + 1)) * kLog2e;
      }
    }
  }

  // One stage at offset sto: tokens from tok0 on, `left` of them the range's.  TAIL when the range
  // ends inside it (its last stage at most): compiled apart, so that the others carry no trace of
  // the end.  ACC: scores to score_lane, this lane's place in the unit's first page of scores.
  template <bool TAIL, bool ACC>
  __device__ __forceinline__ void stage(const DecodeParams &p, uint32_t sto, int tok0, int left, float *score_lane) {
    // ---- scores: fragment rows ra, ra + 8 = tokens, columns 2qc, 2qc + 1
    float x[NP][4];
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const uint32_t ka = kcode0 + sto + j * C::PAGEB, kq = kscale0 + sto + j * C::PAGEB;
#pragma unroll
      for (int b = 0; b < C::QB; ++b) {
        uint32_t wa[C::QE / 8], wb[C::QE / 8], sa[C::QE / 16], sb[C::QE / 16];
        Rows::codes(ka, b, wa);
        Rows::codes(ka + kon8, b, wb);
        Rows::scales(kq, false, b, sa);
        Rows::scales(kq, true, b, sb);
#pragma unroll
        for (int i = 0; i < C::QE / 8; ++i) {
          uint32_t a0[4], a1[4];  // k-steps 2i and 2i + 1
          e2m1x8_to_f16x2x4(wa[i], a0[0], a0[2], a1[0], a1[2]);
          e2m1x8_to_f16x2x4(wb[i], a0[1], a0[3], a1[1], a1[3]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            a0[e] = mul_f16x2(a0[e], (e & 1) ? sb[i >> 1] : sa[i >> 1]);
            a1[e] = mul_f16x2(a1[e], (e & 1) ? sb[i >> 1] : sa[i >> 1]);
          }
          const int jq = b * (C::QE / 4) + 2 * i;
          if (jq == 0) mma_f16_zero(x[j], a0, qf[0][0], qf[0][1]);
          else mma_f16(x[j], a0, qf[jq][0], qf[jq][1]);
          mma_f16(x[j], a1, qf[jq + 1][0], qf[jq + 1][1]);
        }
      }
    }
    // PLAIN keeps the raw sums (sc0, sc1 are never negative, so the largest stays the largest)
    // and scales them inside the exponent's FMA; else scores become log2 units here.
    if constexpr (PLAIN) {
      if constexpr (TAIL) {
#pragma unroll
        for (int j = 0; j < NP; ++j) {
          if (j * kBlock + ra >= left) x[j][0] = x[j][1] = -INFINITY;
          if (j * kBlock + ra + 8 >= left) x[j][2] = x[j][3] = -INFINITY;
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        const int ta = tok0 + j * kBlock + ra, tb = ta + 8;
        x[j][0] = ta <= seeA ? fmaf(ab0, static_cast<float>(ta - posA), x[j][0] * sc0) : -INFINITY;
        x[j][1] = ta <= seeB ? fmaf(ab1, static_cast<float>(ta - posB), x[j][1] * sc1) : -INFINITY;
        x[j][2] = tb <= seeA ? fmaf(ab0, static_cast<float>(tb - posA), x[j][2] * sc0) : -INFINITY;
        x[j][3] = tb <= seeB ? fmaf(ab1, static_cast<float>(tb - posB), x[j][3] * sc1) : -INFINITY;
      }
    }
    if constexpr (ACC) {
      if (2 * qc < p.score_cols) {
#pragma unroll
        for (int j = 0; j < NP; ++j) {
          if (TAIL && j * kBlock >= left) break;
          const float f0 = PLAIN ? sc0 : 1.f, f1 = PLAIN ? sc1 : 1.f;
          float *d = score_lane + static_cast<int64_t>(tok0 + j * kBlock) * p.score_cols;
          if (p.score_cols > 1) {
            *reinterpret_cast<float2 *>(d) = make_float2(x[j][0] * f0, x[j][1] * f1);
            *reinterpret_cast<float2 *>(d + 8 * p.score_cols) = make_float2(x[j][2] * f0, x[j][3] * f1);
          } else {
            d[0] = x[j][0] * f0;
            d[8] = x[j][2] * f0;
          }
        }
      }
    }
    float lm0 = fmaxf(x[0][0], x[0][2]), lm1 = fmaxf(x[0][1], x[0][3]);
#pragma unroll
    for (int j = 1; j < NP; ++j) {
      lm0 = fmaxf(lm0, fmaxf(x[j][0], x[j][2]));
      lm1 = fmaxf(lm1, fmaxf(x[j][1], x[j][3]));
    }
    if constexpr (PLAIN) {
      lm0 *= sc0;
      lm1 *= sc1;
    }
    // the running maximum moves only when a p would pass 2^15
    if (__any_sync(0xffffffffu, (lm0 > m0 + kFp4Slack) | (lm1 > m1 + kFp4Slack))) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        lm0 = fmaxf(lm0, __shfl_xor_sync(0xffffffffu, lm0, o));
        lm1 = fmaxf(lm1, __shfl_xor_sync(0xffffffffu, lm1, o));
      }
      const float mn0 = fmaxf(m0, lm0 - kLift), mn1 = fmaxf(m1, lm1 - kLift);
      const float al0 = ex2(m0 - mn0), al1 = ex2(m1 - mn1);
      l0 *= al0;
      l1 *= al1;
#pragma unroll
      for (int t = 0; t < C::KT; ++t) {
        acc[t][0] *= al0;
        acc[t][1] *= al1;
        acc[t][2] *= al0;
        acc[t][3] *= al1;
      }
      m0 = mn0;
      m1 = mn1;
    }
#pragma unroll
    for (int j = 0; j < NP; ++j) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float m = (i & 1) ? m1 : m0;
        if constexpr (PLAIN) x[j][i] = ex2(fmaf(x[j][i], (i & 1) ? sc1 : sc0, -m));
        else x[j][i] = ex2(x[j][i] - m);
      }
    }
    if constexpr (PLAIN && TAIL) {  // (a zero scale times the -inf above is no number)
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        if (j * kBlock + ra >= left) x[j][0] = x[j][1] = 0.f;
        if (j * kBlock + ra + 8 >= left) x[j][2] = x[j][3] = 0.f;
      }
    }

    // ---- O^T += V^T . P^T
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      l0 += x[j][0] + x[j][2];
      l1 += x[j][1] + x[j][3];
      const uint32_t ha = pack_f16(x[j][0], x[j][1]), hb = pack_f16(x[j][2], x[j][3]);
      const uint32_t bh0 = movmatrix_trans(ha), bh1 = movmatrix_trans(hb);
      const float2 fa = unpack_f16(ha), fb = unpack_f16(hb);
      const uint32_t bl0 = movmatrix_trans(pack_f16(x[j][0] - fa.x, x[j][1] - fa.y));
      const uint32_t bl1 = movmatrix_trans(pack_f16(x[j][2] - fb.x, x[j][3] - fb.y));
      const uint32_t va = vcode0 + sto + j * C::PAGEB, vq = vscale0 + sto + j * C::PAGEB;
      constexpr int VW = Runs::NW;
#pragma unroll
      for (int b = 0; b < C::QB; ++b) {
        uint32_t w[4][VW];
        Runs::codes(va, b, w[0]);
        Runs::codes(va + vodd, b, w[1]);
        Runs::codes(va + von8, b, w[2]);
        Runs::codes(va + von8 + vodd, b, w[3]);
        uint32_t z01 = Runs::scale_pair(vq, 0, b), z23 = Runs::scale_pair(vq, 1, b);
        if constexpr (TAIL) {  // zero scales for the tokens behind the end
          const int lv = left - j * kBlock - 2 * qc;  // of tokens 2qc, + 1, + 8, + 9
          z01 &= (lv > 0 ? 0x00ffu : 0u) | (lv > 1 ? 0xff00u : 0u);
          z23 &= (lv > 8 ? 0x00ffu : 0u) | (lv > 9 ? 0xff00u : 0u);
        }
        const uint32_t s01 = e4m3x2_to_f16x2(z01), s23 = e4m3x2_to_f16x2(z23);
#pragma unroll
        for (int i = 0; i < VW; ++i) {
          constexpr uint32_t kLow = 0x0f0f0f0fu;
          uint32_t e01[4], o01[4], e23[4], o23[4];  // even and odd elements of the word
          e2m1x8_to_f16x2x4((w[0][i] & kLow) | ((w[1][i] << 4) & ~kLow), e01[0], e01[1], e01[2], e01[3]);
          e2m1x8_to_f16x2x4(((w[0][i] >> 4) & kLow) | (w[1][i] & ~kLow), o01[0], o01[1], o01[2], o01[3]);
          e2m1x8_to_f16x2x4((w[2][i] & kLow) | ((w[3][i] << 4) & ~kLow), e23[0], e23[1], e23[2], e23[3]);
          e2m1x8_to_f16x2x4(((w[2][i] >> 4) & kLow) | (w[3][i] & ~kLow), o23[0], o23[1], o23[2], o23[3]);
#pragma unroll
          for (int m = 0; m < 4; ++m) {  // fragment rows ra: element 2m of the word, ra + 8: 2m + 1
            const uint32_t a[4] = {mul_f16x2(e01[m], s01), mul_f16x2(o01[m], s01), mul_f16x2(e23[m], s23),
                                   mul_f16x2(o23[m], s23)};
            const int t = b * 8 + 4 * i + m;
            mma_f16(acc[t], a, bh0, bh1);
            mma_f16(acc[t], a, bl0, bl1);
          }
        }
      }
    }
  }

  // A whole stage or a range's end.
  template <bool ACC>
  __device__ __forceinline__ void any_stage(const DecodeParams &p, uint32_t sto, int tok0, int left, float *score_lane) {
    if (left >= NP * kBlock) stage<false, ACC>(p, sto, tok0, left, score_lane);
    else stage<true, ACC>(p, sto, tok0, left, score_lane);
  }
};

// Runs pages [pb, pe) of sequence s; arguments and result as run_pages_tma (there is no wait here
// that could give up).
template <int KIND, int D, int W, int STAGES, bool PLAIN, bool EARLY, bool ACC>
__device__ __forceinline__ bool run_pages_fp4(const DecodeParams &p, const uint32_t sbase, uint8_t *const sgen,
                                              int &used, const int s, const int len, const Cols &cm,
                                              const int pos0, const int ng, const int pb, const int pe, int entry,
                                              const bool entry_ready, const uint64_t pol, const int wait_page) {
  using C = MmaCfg<KIND, D, W, STAGES>;
  constexpr int NP = C::NP;
  constexpr int PER = 32 / NP;  // stages whose table entries the warp's lanes hold at a time
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int32_t *bt = p.block_table + static_cast<int64_t>(s) * p.bt_ss + pb;
  const int n = pe - pb;                                      // pages of the range
  const int nst = (n + NP - 1) / NP;                          // its stages, every W-th one this warp's
  const int nmine = nst > warp ? (nst - warp + W - 1) / W : 0;
  const uint32_t stage0 = sbase + static_cast<uint32_t>(warp * STAGES * C::STAGEB);
  const int u0 = used;
  bool bad = false, waited = false;

  // Table entries, one page of the warp's next PER stages per lane.  An entry behind the range reads
  // as block 0, and so does a bad one (the CTA then writes nothing), so every copy has a source.
  auto check_entries = [&](int k) {
    const bool in = C::entry(warp, lane) + k * NP * W < n;
    const bool out = in && (entry < 0 || entry >= p.num_blocks);
    if (out && p.err) atomicOr(p.err, kErrBlock);
    if (out || !in) entry = 0;
    bad |= __any_sync(0xffffffffu, out);
  };
  const Fp4Copies<C, D> copies(p, cm.g, lane);
  auto issue = [&](int k) {  // whole warp; k increases by one per call
    if constexpr (EARLY) {
      if (!waited && pb + NP * (warp + k * W) + NP > wait_page) {  // a page that may hold new positions
        grid_dependency_wait();
        waited = true;
      }
    }
    const int at = k % PER;
    if (at == 0) {
      if (k > 0 || !entry_ready) {
        const int i = C::entry(warp, lane) + k * NP * W;
        entry = i < n ? __ldg(bt + i) : 0;
      }
      check_entries(k);
    }
    copies.stage(stage0 + (u0 + k) % STAGES * C::STAGEB, entry, at * NP, pol);
    copy_commit();
  };

  // (a group is committed for every stage, filled or not: the waits count groups)
#pragma unroll
  for (int k = 0; k < STAGES; ++k) {
    if (k < nmine) issue(k);
    else copy_commit();
  }

  const int end = min(len, pe * kBlock);
  Fp4State<C, D, PLAIN> state;
  state.place(stage0);
  state.begin(p, cm, ng, pos0, end);
  float *score_lane = nullptr;
  if constexpr (ACC) score_lane = fp4_score_lane(p, s, blockIdx.y);

  for (int k = 0; k < nmine; ++k) {
    copy_wait<STAGES - 1>();  // this lane's copies of the stage, then the whole warp's
    __syncwarp();
    const int tok0 = (pb + NP * (warp + k * W)) * kBlock;
    state.template any_stage<ACC>(p, (u0 + k) % STAGES * C::STAGEB, tok0, end - tok0, score_lane);
    __syncwarp();  // every lane has read the stage
    if (k + STAGES < nmine) issue(k + STAGES);
    else copy_commit();
  }
  used = u0 + nmine;
  __syncwarp();
  store_warp_state<C, D, STAGES>(sgen, state.m0, state.m1, state.l0, state.l1, state.acc);
  return bad;
}

}  // namespace pa
