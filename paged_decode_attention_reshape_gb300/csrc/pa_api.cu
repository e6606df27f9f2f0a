// pa_api.cu -- the C ABI of include/pa.h: argument validation, the split-KV
// partition plan, TMA descriptors, workspace, device error word and profiling.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <mutex>
#include <vector>

#include "pa_internal.h"
#include "pa_validate.h"
#include "pa_workspace.h"

#define PA_API extern "C" __attribute__((visibility("default")))

namespace pa {
namespace {

// --------------------------------------------------------------- profiling

struct Profiler {
  std::mutex mu;
  bool on = false;
  std::vector<std::pair<cudaEvent_t, cudaEvent_t>> ev[2];
  std::vector<cudaEvent_t> pool;
  cudaEvent_t get() {
    if (!pool.empty()) {
      cudaEvent_t e = pool.back();
      pool.pop_back();
      return e;
    }
    cudaEvent_t e = nullptr;
    cudaEventCreate(&e);
    return e;
  }
};
Profiler &prof() {
  static Profiler P;
  return P;
}

// Brackets one kernel launch with events when profiling is on.
struct ProfScope {
  int kind;
  cudaStream_t st;
  cudaEvent_t e0 = nullptr, e1 = nullptr;
  ProfScope(int k, cudaStream_t s) : kind(k), st(s) {
    Profiler &P = prof();
    std::lock_guard<std::mutex> g(P.mu);
    if (!P.on) return;
    e0 = P.get();
    e1 = P.get();
    cudaEventRecord(e0, st);
  }
  ~ProfScope() {
    if (!e0) return;
    cudaEventRecord(e1, st);
    Profiler &P = prof();
    std::lock_guard<std::mutex> g(P.mu);
    P.ev[kind].emplace_back(e0, e1);
  }
};

// ------------------------------------------------------------- tensor maps

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(ptr);
  });
  return fn;
}

// 4-D TMA map of one cache, boxes of one (block, kv head) page: 16 token rows of one
// 128-byte swizzle span.  HND caches (token stride <= head stride) are described as
// (D, 16, Hkv, NB), box (span, 16, 1, 1); NHD caches (token-major within a block,
// [NB, 16, Hkv, D] seen through its [NB, Hkv, 16, D] permutation) in their own order,
// (D, Hkv, 16, NB), box (span, 1, 16, 1), which lands in shared memory as the same
// 16 x span tile.  *nhd tells the kernel which coordinate order to use.
int make_cache_map(const pa_tensor *c, CUtensorMap *map, int *nhd) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return PA_ERR_CUDA;
  const int eb = elem_bytes(c->dtype);
  *nhd = c->stride[2] > c->stride[1] ? 1 : 0;
  const int mid_a = *nhd ? 1 : 2, mid_b = *nhd ? 2 : 1;  // dimension order after D
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(c->shape[3]), static_cast<cuuint64_t>(c->shape[mid_a]),
                              static_cast<cuuint64_t>(c->shape[mid_b]), static_cast<cuuint64_t>(c->shape[0])};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(c->stride[mid_a] * eb),
                                 static_cast<cuuint64_t>(c->stride[mid_b] * eb),
                                 static_cast<cuuint64_t>(c->stride[0] * eb)};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(128 / eb), *nhd ? 1u : 16u, *nhd ? 16u : 1u, 1};
  const cuuint32_t es[4] = {1, 1, 1, 1};
  const CUtensorMapDataType dt = eb == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16;
  CUresult r = enc(map, dt, 4, c->data, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? PA_OK : PA_ERR_CUDA;
}

// 3-D TMA map of varlen queries [Tq, Hq, D] for the query-tile kernel: dims (D, Hq, Tq),
// box (64 elements, G heads, 128 / G tokens), 128-byte swizzle.  One box is 128 rows (query
// token-major, head-minor: the kernel's row order) of one 128-byte column span, the layout
// in which the kernel's MMAs read Q.  Needs G to divide 128; PA_ERR_INVALID_ARG otherwise
// (the kernel then loads Q itself).  The strides were checked 16-byte aligned by the caller.
int make_q_map(const pa_tensor *q, int G, CUtensorMap *map) {
  if (G <= 0 || 128 % G != 0) return PA_ERR_INVALID_ARG;
  EncodeTiledFn enc = encode_fn();
  if (!enc) return PA_ERR_CUDA;
  const int eb = elem_bytes(q->dtype);
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(q->shape[2]), static_cast<cuuint64_t>(q->shape[1]),
                              static_cast<cuuint64_t>(q->shape[0])};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(q->stride[1] * eb), static_cast<cuuint64_t>(q->stride[0] * eb)};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(128 / eb), static_cast<cuuint32_t>(G),
                             static_cast<cuuint32_t>(128 / G)};
  const cuuint32_t es[3] = {1, 1, 1};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, q->data, dims, strides, box, es,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? PA_OK : PA_ERR_CUDA;
}

// --------------------------------------------------------------- plan

int kind_of(int q_dtype, int cache_dtype) {
  if (cache_dtype == PA_FP8_E4M3) {
    if (q_dtype == PA_BF16) return KIND_FP8_BF16Q;
    if (q_dtype == PA_F16) return KIND_FP8_F16Q;
    return -1;
  }
  if (cache_dtype == PA_FP4_E2M1) {
    if (q_dtype == PA_BF16) return KIND_FP4_BF16Q;
    if (q_dtype == PA_F16) return KIND_FP4_F16Q;
    return -1;
  }
  if (q_dtype != cache_dtype) return -1;
  if (q_dtype == PA_BF16) return KIND_BF16;
  if (q_dtype == PA_F16) return KIND_F16;
  if (q_dtype == PA_F32) return KIND_F32;
  return -1;
}

// Batches the tensor-core kernel runs longest-first (see lpt_sequence).
bool longest_first(int kind, int S) { return kind != KIND_F32 && S <= 128; }

// Resident CTAs per SM of the decode kernel for (kind, D).  With `device`, the CUDA
// occupancy calculator's answer for the current device (cached per shape); otherwise,
// or when that query fails, the shared-memory bound alone (a what-if plan for another
// GPU, or a host without one).
int ctas_per_sm(int kind, int D, bool device) {
  if (kind == KIND_F32) return 4;
  if (device) {
    static std::atomic<int> cache[7][3];
    const int di = D == 64 ? 0 : D == 128 ? 1 : 2;
    int n = cache[kind][di].load(std::memory_order_relaxed);
    if (n == 0) {
      n = (kind == KIND_BF16 || kind == KIND_F16) ? occupancy_decode_mma_16(kind, D)
          : mma_fp4(kind)                         ? occupancy_decode_mma_fp4(kind, D)
                                                  : occupancy_decode_mma_fp8(kind, D);
      if (n > 0) cache[kind][di].store(n, std::memory_order_relaxed);
    }
    if (n > 0) return n;
  }
  const size_t smem = mma_smem(kind, D);
  int n = static_cast<int>((227u * 1024u) / (smem + 1024));
  return std::max(1, std::min(n, 16));
}

// Partition size in tokens (0 = unsplit).  The plan cannot read seq_lens (no
// host sync), so it assumes lengths spread up to the block-table width (average
// about half of it).
//  - Batches of at most kLptMax sequences run longest-first (the kernel ranks the
//    lengths itself); when their (sequence, kv head, head group) units fill the
//    GPU's resident CTA slots at least once, that order balances the load and the
//    call does not split.  Any batch whose units fill the slots twice does not
//    split either.
//  - Otherwise the assumed work is cut into partitions of equal length, about two
//    resident waves' worth, never shorter than 64 pages (1024 tokens): below that
//    the per-CTA prologue and the partition merge cost more than the balance gains.
// Fitted on GB300 to sweeps over partition sizes for the benchmark workloads:
// 128 x 1k..8k tokens and 256 x 512..4096 run best unsplit, 64 x 1..2048 with its
// longest sequences cut in two (1024), 4 x 32k..128k near 2048 tokens.
int plan_partition(int S, int Hq, int Hkv, int D, int maxNB, int kind, int sm, bool device, int request) {
  if (request < 0) return 0;
  const int max_tokens = maxNB * kBlock;
  int P;
  if (request > 0) {
    P = (request + kBlock - 1) / kBlock * kBlock;
  } else {
    const int G = Hq / Hkv;
    const int64_t units = static_cast<int64_t>(S) * Hkv * ((G + 7) / 8);
    const int64_t slots = static_cast<int64_t>(std::max(sm, 1)) * ctas_per_sm(kind, D, device);
    if ((longest_first(kind, S) && units >= slots) || units >= 2 * slots) return 0;
    const int64_t work = units * std::max(1, maxNB / 2);  // pages, assuming half-full tables
    // 4-bit pages take less time each, so a CTA's fixed time weighs more against them: one wave of
    // partitions over full tables, and half the smallest size (1 x 8k tokens: 10.4 us against 11.6)
    const int64_t pages = mma_fp4(kind) ? std::max<int64_t>(units * maxNB / slots, 32)
                                        : std::max<int64_t>(work / (2 * slots), 64);
    if (pages >= maxNB) return 0;
    P = static_cast<int>(pages * kBlock);
  }
  if (P >= max_tokens) return 0;
  return P;
}

// The full plan: fixed-size partitions (P tokens, merged through the workspace by the
// last-arriving CTA), the balanced split (request PA_PARTITION_BALANCED: one resident
// wave of CTAs per head row, each taking an equal share of the batch's pages), or, on
// request only (-2, -4 or -8), a cluster split: each unit cut into C equal parts whose
// CTAs form one thread-block cluster and merge through distributed shared memory, with
// no workspace.  The heuristic does not pick the cluster split: cutting every unit
// (short ones too) multiplies the CTAs beyond the resident slots, and on GB300 that
// cost more than the shorter critical path saved (64 x 1..2048 tokens: 33.2 us
// unsplit, 34.3 / 42.1 / 56.1 us for C = 2 / 4 / 8, 32.9 us with 1024-token partitions).
struct Plan {
  int P;        // tokens per fixed partition (0 = none)
  int cluster;  // parts per unit of the cluster split (0 = none)
  int flat;     // CTAs (with `warps`: warps) per head row of the balanced split (0 = none)
  int status;
  int warps;    // 1: the balanced split over warps (4-bit caches)
  int narrow;   // 1: CTAs of half the warps (windows)
};
int balanced_ctas(int Hq, int Hkv, int D, int kind, int sm, bool device) {
  const int64_t rows = static_cast<int64_t>(Hkv) * ((Hq / Hkv + 7) / 8);
  const int64_t slots = static_cast<int64_t>(std::max(sm, 1)) * ctas_per_sm(kind, D, device);
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(slots / rows, 65535)));
}
// 4-bit caches, one query token and no ALiBi (`plain`): the balanced split over warps
// (pa_decode_fp4_warps.cuh) where the batch has at least two (sequence, kv head, head group) units
// for every three warps of a resident wave (on request: one for eight), and the balanced split over
// CTAs where there are too few units for the CTAs and a CTA still gets 128 pages or more; else whole
// units or fixed partitions.  Measured on GB300 (2432 warps, 304 CTAs; us over warps / unsplit or
// over CTAs / fixed partitions of one wave): 304 x 256 tokens, 2432 units, 22.1 / 42.1 / -; 256 x
// 512..4096, 2048 units, 135.6 / 156.8 / -; 128 x 1k..8k, 1024 units, 137.7 / 136.3 / -; 64 x 0..2048,
// 512 units, 23.1 / 18.2 / - (the parts of cut units cost more than the waves); 16 x 4k..32k, 128 units,
// - / 75.0 / 115.3; 4 x 32k..128k, 32 units, - / 82.6 / 115.7; 1 x 8k, 8 units, - / 17.1 / 10.0.
bool plan_fp4(int S, int Hq, int Hkv, int D, int maxNB, int kind, int sm, bool device, bool varlen, bool plain,
              bool balanced, Plan *pl) {
  const int64_t rows = static_cast<int64_t>(Hkv) * ((Hq / Hkv + 7) / 8), units = S * rows;
  const int64_t ctas = static_cast<int64_t>(std::max(sm, 1)) * mma_min_ctas(kind, D);
  const int64_t workers = ctas * mma_warps(kind, D);
  if (S > kFlatMaxSeqs || varlen) return false;
  if (static_cast<int64_t>(S) * maxNB > INT32_MAX) return false;  // stages are numbered in 32 bits
  if (plain && (balanced ? units * 8 >= workers : units * 3 >= workers * 2) && rows <= ctas) {
    pl->warps = 1;
    pl->flat = static_cast<int>(ctas / rows) * mma_warps(kind, D);
    return true;
  }
  const int64_t slots = static_cast<int64_t>(std::max(sm, 1)) * ctas_per_sm(kind, D, device);
  if (!balanced && units * (maxNB / 2) < 128 * slots) return false;
  if (units >= slots) return false;  // (not `plain`: whole units fill the slots)
  pl->flat = balanced_ctas(Hq, Hkv, D, kind, sm, device);
  return true;
}
// varlen: several query tokens; plain: one, and no ALiBi
Plan make_plan(int S, int Hq, int Hkv, int D, int maxNB, int kind, int sm, bool device, int request,
               bool varlen = false, bool plain = true) {
  Plan pl{0, 0, 0, PA_OK, 0, 0};
  if (mma_fp4(kind) && request == 0 &&
      plan_fp4(S, Hq, Hkv, D, maxNB, kind, sm, device, varlen, plain, false, &pl))
    return pl;
  if (request == PA_PARTITION_BALANCED) {
    if (kind == KIND_F32) return pl;  // the CUDA-core kernel runs it unsplit
    if (S > kFlatMaxSeqs || (mma_fp4(kind) && static_cast<int64_t>(S) * maxNB > INT32_MAX))
      pl.status = PA_ERR_UNSUPPORTED_SHAPE;
    else if (mma_fp4(kind) && plan_fp4(S, Hq, Hkv, D, maxNB, kind, sm, device, varlen, plain, true, &pl)) return pl;
    else pl.flat = balanced_ctas(Hq, Hkv, D, kind, sm, device);
    return pl;
  }
  if (request <= -2) {
    const int C = -request;
    if (C != 2 && C != 4 && C != 8) pl.status = PA_ERR_INVALID_ARG;
    else pl.cluster = C;
    return pl;
  }
  pl.P = plan_partition(S, Hq, Hkv, D, maxNB, kind, sm, device, request);
  return pl;
}

// Chunks of query tokens run on the query-tile kernel (rows in the MMA M dimension, pages shared by 64
// rows, no split) unless a split was asked for; columns: query columns per KV head.
bool on_query_tiles(int kind, int D, int partition_size, int columns, bool windowed) {
  return (kind == KIND_BF16 || kind == KIND_F16) && (D == 64 || D == 128 || (D == 256 && windowed)) &&
         (partition_size == 0 || partition_size == -1) && columns >= chunk_min_columns(D);
}

// Long chunks over E4M3 and 4-bit caches under a window: the pages that the chunk sees, bounded by the window and
// not by the length, are widened into the workspace first and run on the query tiles, where a sequence has
// this many query columns per KV head on average, the columns' kernels (which widen every page once for 8 columns)
// had this many work items, and the scratch stays below its limit.  Measured on GB300, 8 KV heads of 4 x 128
// (4 x 256), columns / widened in us: E4M3, 64 sequences, window 1024: 64 columns 137 / 164 (244 / 372), 96
// 208 / 170 (371 / 383), 128 275 / 171 (490 / 388), 256 543 / 208 (973 / 567), 2048 4100 / 740.  With few items
// a query tile's walk over the window lasts longer than all the columns' (window 4096, 128 columns: 1024 items
// 105 / 174 (178 / 262), 2048 items 179 / 209 (313 / 325); 256 columns: 2048 183 / 132 (315 / 264)).  4-bit pages
// gain more (64 sequences, 128 columns: 296 / 160 (420 / 362); 64-wide heads 246 / 82).  The thresholds know neither the
// window nor the cache: at 96 columns and window 1024 they take the slower side (heads of 128), and at 2048 items
// and window 4096 with 128 columns as well.
constexpr int kWidenColumns = 128;
constexpr int kWidenItems = 2048;
constexpr int64_t kWidenBytes = 1ll << 30;
struct WidenPlan {
  int pages;       // of a sequence, 0: not this way
  size_t table, total;  // bytes of both caches' pages (K's, V's, then the block table), bytes in all
};
// (rows: the query rows of all sequences, columns: those of the longest chunk)
WidenPlan widen_plan(int S, int Hkv, int D, int maxNB, int kind, int partition_size, int columns, int nq, int64_t rows,
                     int64_t window, int64_t sinks) {
  WidenPlan w{0, 0, 0};
  const int64_t all = std::min(rows, static_cast<int64_t>(S) * nq) * (columns / std::max(nq, 1));  // columns per KV head
  if (!(mma_fp8(kind) || mma_fp4(kind)) || window <= 0 || nq < 2 ||
      all < static_cast<int64_t>(S) * kWidenColumns || all * Hkv < kWidenItems * 8 ||
      !on_query_tiles(KIND_BF16, D, partition_size, columns, true))
    return w;
  const int64_t pages = std::min<int64_t>(maxNB, (window + nq - 1 + kBlock - 2) / kBlock + 1 + (sinks + kBlock - 1) / kBlock);
  const int64_t page_bytes = static_cast<int64_t>(Hkv) * kBlock * D * 2;
  if (pages > kWidenBytes / (2 * page_bytes) / S) return w;  // (S > 0: it has columns)
  const int64_t one = S * pages * page_bytes, total = 2 * one + static_cast<int64_t>(S) * maxNB * 4;
  if (total > kWidenBytes) return w;
  w.pages = static_cast<int>(pages);
  w.table = static_cast<size_t>(2 * one);
  w.total = static_cast<size_t>(total);
  return w;
}

// Under a window: the most pages that a work item of the decode kernels reads (its numbers of Window),
// for 8 columns of G heads a query and at most nq queries.  Windows and first tokens as given by the caller.
int window_blocks(int maxNB, int64_t window, int64_t sinks, int G, int nq) {
  const int64_t span = std::min(nq, 7 / G + 2);  // queries among 8 columns
  const int64_t pages = (window + span - 1 + kBlock - 2) / kBlock + 1 + (sinks + kBlock - 1) / kBlock;
  return static_cast<int>(std::min<int64_t>(maxNB, pages));
}
// The plan of a call under a window, of `pages` a unit by window_blocks (nearly what every longer sequence
// reads, where a plan by the table's width has to guess).  Units that leave half of the resident CTA slots
// empty are cut into 2, 4 or 8 parts a cluster, as long as the slots hold them all and a warp keeps two
// pages; the cluster costs about 2 us, which fewer than eight pages a warp do not repay.  Whole units run in
// CTAs of half the warps, twice as many to an SM, where that brings all of them in at once (a second
// wave of CTAs costs 5 us before its first page) or where they are so short that their own start weighs most
// (`plain`: one query and no ALiBi, the only kernels built so).
// Measured on GB300, 8 KV heads of 128, bf16 (us; unsplit / 2 / 4 / 8 parts / fixed partitions of the best
// size / balanced): 1 sequence, window 1024, 65 pages: 14.0 / 11.4 / 8.4 / 7.2 / 9.3 / 29.0; 1 x 128: 5.3 / 6.6 /
// 5.6 / 5.8 / - / 10.5; 4 x 4112: 43.9 / 26.4 / 17.4 / 16.1 / 18.2 / 26.0; 8 x 1024: 14.4 / 12.5 / 11.3 / 19.2 / 12.8 /
// 17.8; 16 x 256: 7.5 / 9.7 / 16.2 / 22.0 / 10.8 / 17.6; 32 x 1024: 24.3 / 36.3 / 36.3 / 51.6 / 31.2 / 29.8.
// Unsplit in whole / half CTAs (and balanced): 64 x 512, 1.1 waves: 32.0 / 26.3 (32.2); 64 x 2048: 96.3 / 82.7
// (88.8); 128 x 2048, E4M3, 1.7 waves: 92.5 / 90.0 (94.8); 128 x 256, 2.2 waves: 34.1 / 36.1; 256 x 1024, 4.5 waves:
// 153 / 159; 256 x 128 (10 pages): 36.8 / 34.7, head size 64: 24.1 / 20.5.
Plan make_window_plan(int S, int Hq, int Hkv, int D, int pages, int kind, int sm, bool device, int request, bool varlen,
                      bool plain) {
  if (request != 0) return make_plan(S, Hq, Hkv, D, pages, kind, sm, device, request, varlen, false);
  Plan pl{0, 0, 0, PA_OK, 0, 0};
  const int64_t units = static_cast<int64_t>(S) * Hkv * ((Hq / Hkv + 7) / 8);
  const int64_t slots = static_cast<int64_t>(std::max(sm, 1)) * ctas_per_sm(kind, D, device);
  const int warps = kind == KIND_F32 ? (D == 256 ? 2 : 4) : mma_warps(kind, D);
  if (pages >= 8 * warps) {
    for (const int C : {8, 4, 2}) {
      if (units * C > slots || pages < 2 * C * warps) continue;
      if (C == 2 && mma_fp4(kind) && pages < 16 * warps) continue;  // (16 x 1024: 10.6 us, in two parts 13.5)
      pl.cluster = C;
      return pl;
    }
  }
  if (plain && kind != KIND_F32) pl.narrow = units > slots && (units <= 2 * slots || 2 * pages <= 5 * warps) ? 1 : 0;
  return pl;
}

// Split-KV workspace: [arrival counters, one int per (sequence, kv head, head group)]
// [partial (m, l): one float2 per row] [partial acc: D floats per row], each region
// starting on a 256-byte boundary.  Rows: one per (sequence, head, partition) for
// fixed-size partitions; 2 x 8 per CTA for the balanced split (`flat` CTAs per head row).
struct WsLayout {
  size_t ml_off, acc_off, total;
};
size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
size_t arrival_counter_bytes(int S, int Hq, int Hkv) {
  return round256(static_cast<size_t>(S) * Hkv * ((Hq / Hkv + 7) / 8) * sizeof(int));
}
WsLayout workspace_layout(int S, int Hq, int Hkv, int D, int maxNB, int P, int flat) {
  WsLayout L{0, 0, 0};
  if (P <= 0 && flat <= 0) return L;
  const int64_t head_rows = static_cast<int64_t>(Hkv) * ((Hq / Hkv + 7) / 8);
  const int64_t rows = flat > 0 ? head_rows * flat * 16
                                : static_cast<int64_t>(S) * Hq * ((static_cast<int64_t>(maxNB) * kBlock + P - 1) / P);
  L.ml_off = arrival_counter_bytes(S, Hq, Hkv);
  L.acc_off = L.ml_off + round256(static_cast<size_t>(rows) * sizeof(float2));
  L.total = L.acc_off + static_cast<size_t>(rows) * D * sizeof(float);
  return L;
}

// pa_decode_accumulate's part of the workspace, behind the split-KV part: log2 of every
// head's softmax sum, then one score per (sequence, KV head, head group, token, column).
struct ScoreLayout {
  int cols;  // columns per token: the group's query heads rounded up to 1, 2, 4 or 8
  size_t scores_off, total;
};
ScoreLayout score_layout(int S, int Hq, int Hkv, int maxNB) {
  const int G = Hq / Hkv, HG = (G + 7) / 8;
  ScoreLayout L;
  L.cols = G <= 1 ? 1 : G <= 2 ? 2 : G <= 4 ? 4 : 8;
  L.scores_off = round256(static_cast<size_t>(S) * Hq * sizeof(float));
  L.total = L.scores_off + static_cast<size_t>(S) * Hkv * HG * maxNB * kBlock * L.cols * sizeof(float);
  return L;
}

}  // namespace
}  // namespace pa

using namespace pa;

// ===================================================================== ABI

PA_API const char *pa_status_string(int status) {
  switch (status) {
    case PA_OK: return "ok";
    case PA_ERR_INVALID_ARG: return "invalid argument";
    case PA_ERR_UNSUPPORTED_DTYPE: return "unsupported element type";
    case PA_ERR_ALIGNMENT: return "pointer or stride not aligned (rows and caches: 16 bytes)";
    case PA_ERR_WORKSPACE: return "workspace missing or too small";
    case PA_ERR_CUDA: return "CUDA call or launch failed";
    case PA_ERR_DEVICE_BOUNDS: return "device reported an out-of-range slot, block id or sequence length";
    case PA_ERR_UNSUPPORTED_SHAPE: return "unsupported shape (block size, head size or extent)";
    case PA_ERR_DEVICE_TIMEOUT: return "device pipeline wait timed out";
    case PA_ERR_NO_BLOCKS: return "block pool has too few free blocks";
    default: return "unknown status";
  }
}

// The write with its grid's CTAs per SM (0: the standalone choice; pa_decode_step asks for
// fewer when the decode's early reads overlap it).
static int write_impl(const pa_tensor *key, const pa_tensor *value, pa_tensor *k_cache, pa_tensor *v_cache,
                      const pa_tensor *slot_mapping, int kv_dtype, const pa_write_options *opt, pa_stream_t stream,
                      int ctas_per_sm) {
  const pa_write_options o = opt ? *opt : pa_write_options{};
  if (o.scale_stride < 0) return PA_ERR_INVALID_ARG;
  int r;
  if ((r = check_desc(key, 3)) || (r = check_desc(value, 3)) || (r = check_desc(slot_mapping, 1))) return r;
  int NB, Hkv, D;
  if ((r = validate_cache_pair(k_cache, v_cache, &NB, &Hkv, &D))) return r;
  const int in_dt = key->dtype;
  if (value->dtype != in_dt) return PA_ERR_INVALID_ARG;
  if (in_dt != PA_F32 && in_dt != PA_BF16 && in_dt != PA_F16) return PA_ERR_UNSUPPORTED_DTYPE;
  if (slot_mapping->dtype != PA_I64) return PA_ERR_UNSUPPORTED_DTYPE;
  if (kv_dtype == PA_KV_AUTO) {
    if (k_cache->dtype != in_dt) return PA_ERR_UNSUPPORTED_DTYPE;
  } else if (kv_dtype == PA_KV_FP8_E4M3) {
    if (k_cache->dtype != PA_FP8_E4M3) return PA_ERR_UNSUPPORTED_DTYPE;
  } else if (kv_dtype == PA_KV_FP4_E2M1) {
    if (k_cache->dtype != PA_FP4_E2M1) return PA_ERR_UNSUPPORTED_DTYPE;
  } else {
    return PA_ERR_INVALID_ARG;
  }
  const int64_t T = key->shape[0];
  if (value->shape[0] != T || slot_mapping->shape[0] != T) return PA_ERR_INVALID_ARG;
  if (key->shape[1] != Hkv || key->shape[2] != D || value->shape[1] != Hkv || value->shape[2] != D)
    return PA_ERR_INVALID_ARG;
  if (key->stride[2] != 1 || value->stride[2] != 1 || slot_mapping->stride[0] != 1) return PA_ERR_INVALID_ARG;
  const int ib = elem_bytes(in_dt);
  if (D <= 0 || (static_cast<int64_t>(D) * ib) % 16) return PA_ERR_UNSUPPORTED_SHAPE;
  if (T == 0 || Hkv == 0) return PA_OK;
  if (!key->data || !value->data || !slot_mapping->data) return PA_ERR_INVALID_ARG;
  if (!aligned16(key->data) || !aligned16(value->data) || !on_elements(slot_mapping)) return PA_ERR_ALIGNMENT;
  if (!aligned4(o.k_scale) || !aligned4(o.v_scale) || !aligned4(o.device_error)) return PA_ERR_ALIGNMENT;
  for (int i = 0; i < 2; ++i)
    if ((key->stride[i] * ib) % 16 || (value->stride[i] * ib) % 16) return PA_ERR_ALIGNMENT;

  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (kv_dtype == PA_KV_FP4_E2M1) {
    Fp4WriteParams f{};
    f.key = key->data;
    f.value = value->data;
    f.k_cache = static_cast<char *>(k_cache->data);
    f.v_cache = static_cast<char *>(v_cache->data);
    f.slot_mapping = static_cast<const int64_t *>(slot_mapping->data);
    f.T = T;
    f.Hkv = Hkv;
    f.D = D;
    f.key_ts = key->stride[0] * ib;
    f.key_hs = key->stride[1] * ib;
    f.val_ts = value->stride[0] * ib;
    f.val_hs = value->stride[1] * ib;
    f.kc_s0 = k_cache->stride[0];
    f.kc_s1 = k_cache->stride[1];
    f.vc_s0 = v_cache->stride[0];
    f.vc_s1 = v_cache->stride[1];
    f.num_slots = static_cast<int64_t>(NB) * kBlock;
    f.k_scale = o.k_scale;
    f.v_scale = o.v_scale;
    f.scale_stride = o.scale_stride;
    f.err = o.device_error;
    f.wide = rows_aligned32(key, ib) && rows_aligned32(value, ib);
    f.i32 = T <= INT32_MAX;
    for (const int64_t x : {f.key_ts, f.key_hs, f.val_ts, f.val_hs, f.kc_s0, f.kc_s1, f.vc_s0, f.vc_s1})
      f.i32 &= x <= INT32_MAX;
    ProfScope ps(PA_KERNEL_WRITE, st);
    return launch_write_fp4(f, in_dt, st) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
  }

  WriteParams p;
  p.key = key->data;
  p.value = value->data;
  p.k_cache = k_cache->data;
  p.v_cache = v_cache->data;
  p.slot_mapping = static_cast<const int64_t *>(slot_mapping->data);
  p.T = T;
  p.Hkv = Hkv;
  p.D = D;
  p.key_ts = key->stride[0];
  p.key_hs = key->stride[1];
  p.val_ts = value->stride[0];
  p.val_hs = value->stride[1];
  p.kc_s0 = k_cache->stride[0];
  p.kc_s1 = k_cache->stride[1];
  p.kc_s2 = k_cache->stride[2];
  p.vc_s0 = v_cache->stride[0];
  p.vc_s1 = v_cache->stride[1];
  p.vc_s2 = v_cache->stride[2];
  p.num_slots = static_cast<int64_t>(NB) * kBlock;
  p.k_scale = kv_dtype == PA_KV_FP8_E4M3 ? o.k_scale : nullptr;
  p.v_scale = kv_dtype == PA_KV_FP8_E4M3 ? o.v_scale : nullptr;
  p.scale_stride = o.scale_stride;
  p.err = o.device_error;
  {
    // 32-bit index arithmetic when every byte offset the kernel forms stays below 2^31: the
    // source rows (first to last element), the cache's block and token strides and the
    // extent of one block (the block offset itself is one widening multiply)
    const int64_t lim = INT32_MAX;
    const int cb = elem_bytes(k_cache->dtype);
    auto span = [&](const pa_tensor *t) { return ((T - 1) * t->stride[0] + (Hkv - 1) * t->stride[1] + D) * ib; };
    auto inner = [&](const pa_tensor *c) { return ((Hkv - 1) * c->stride[1] + (kBlock - 1) * c->stride[2] + D) * cb; };
    p.i32 = T <= lim && span(key) <= lim && span(value) <= lim && k_cache->stride[0] * cb <= lim &&
            v_cache->stride[0] * cb <= lim && inner(k_cache) <= lim && inner(v_cache) <= lim;
  }
  const int sm = device_sm_count();
  if (sm <= 0) return PA_ERR_CUDA;
  cudaError_t e;
  {
    ProfScope ps(PA_KERNEL_WRITE, st);
    e = launch_write(p, in_dt, k_cache->dtype, sm, ctas_per_sm, st);
  }
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

PA_API int pa_reshape_and_cache_opt(const pa_tensor *key, const pa_tensor *value, pa_tensor *k_cache,
                                    pa_tensor *v_cache, const pa_tensor *slot_mapping, int kv_dtype,
                                    const pa_write_options *opt, pa_stream_t stream) {
  return write_impl(key, value, k_cache, v_cache, slot_mapping, kv_dtype, opt, stream, 0);
}

PA_API int pa_reshape_and_cache(const pa_tensor *key, const pa_tensor *value, pa_tensor *k_cache, pa_tensor *v_cache,
                                const pa_tensor *slot_mapping, int kv_dtype, const float *k_scale,
                                const float *v_scale, int *device_error, pa_stream_t stream) {
  pa_write_options o{};
  o.k_scale = k_scale;
  o.v_scale = v_scale;
  o.device_error = device_error;
  return pa_reshape_and_cache_opt(key, value, k_cache, v_cache, slot_mapping, kv_dtype, &o, stream);
}

PA_API int pa_gather_cache(pa_tensor *key, pa_tensor *value, const pa_tensor *k_cache, const pa_tensor *v_cache,
                           const pa_tensor *slot_mapping, const pa_write_options *opt, pa_stream_t stream) {
  const pa_write_options o = opt ? *opt : pa_write_options{};
  if (o.scale_stride < 0) return PA_ERR_INVALID_ARG;
  int r;
  if ((r = check_desc(key, 3)) || (r = check_desc(value, 3)) || (r = check_desc(slot_mapping, 1))) return r;
  int NB, Hkv, D;
  if ((r = validate_cache_pair(k_cache, v_cache, &NB, &Hkv, &D))) return r;
  const int out_dt = key->dtype, cache_dt = k_cache->dtype;
  if (value->dtype != out_dt) return PA_ERR_INVALID_ARG;
  if (out_dt != PA_F32 && out_dt != PA_BF16 && out_dt != PA_F16) return PA_ERR_UNSUPPORTED_DTYPE;
  const bool quantised = cache_dt == PA_FP8_E4M3 || cache_dt == PA_FP4_E2M1;
  if (!quantised && cache_dt != out_dt) return PA_ERR_UNSUPPORTED_DTYPE;
  if (slot_mapping->dtype != PA_I64) return PA_ERR_UNSUPPORTED_DTYPE;
  const int64_t T = key->shape[0];
  if (value->shape[0] != T || slot_mapping->shape[0] != T) return PA_ERR_INVALID_ARG;
  if (key->shape[1] != Hkv || key->shape[2] != D || value->shape[1] != Hkv || value->shape[2] != D)
    return PA_ERR_INVALID_ARG;
  if (key->stride[2] != 1 || value->stride[2] != 1 || slot_mapping->stride[0] != 1) return PA_ERR_INVALID_ARG;
  if (D <= 0 || D % 16) return PA_ERR_UNSUPPORTED_SHAPE;
  if (rows_overlap(key, D) || rows_overlap(value, D)) return PA_ERR_INVALID_ARG;
  if (T == 0 || Hkv == 0) return PA_OK;
  if (!key->data || !value->data || !slot_mapping->data) return PA_ERR_INVALID_ARG;
  const int ob = elem_bytes(out_dt), cb = elem_bytes(cache_dt);
  if (!aligned16(key->data) || !aligned16(value->data) || !on_elements(slot_mapping)) return PA_ERR_ALIGNMENT;
  if (!aligned4(o.k_scale) || !aligned4(o.v_scale) || !aligned4(o.device_error)) return PA_ERR_ALIGNMENT;
  for (int i = 0; i < 2; ++i)
    if ((key->stride[i] * ob) % 16 || (value->stride[i] * ob) % 16) return PA_ERR_ALIGNMENT;
  GatherParams p{};
  p.key = static_cast<char *>(key->data);
  p.value = static_cast<char *>(value->data);
  p.k_cache = static_cast<const char *>(k_cache->data);
  p.v_cache = static_cast<const char *>(v_cache->data);
  p.slot_mapping = static_cast<const int64_t *>(slot_mapping->data);
  p.T = T;
  p.Hkv = Hkv;
  p.D = D;
  p.key_ts = key->stride[0] * ob;
  p.key_hs = key->stride[1] * ob;
  p.val_ts = value->stride[0] * ob;
  p.val_hs = value->stride[1] * ob;
  p.kc_s0 = k_cache->stride[0] * cb;
  p.kc_s1 = k_cache->stride[1] * cb;
  p.kc_s2 = cache_dt == PA_FP4_E2M1 ? 0 : k_cache->stride[2] * cb;
  p.vc_s0 = v_cache->stride[0] * cb;
  p.vc_s1 = v_cache->stride[1] * cb;
  p.vc_s2 = cache_dt == PA_FP4_E2M1 ? 0 : v_cache->stride[2] * cb;
  p.num_slots = static_cast<int64_t>(NB) * kBlock;
  p.k_scale = quantised ? o.k_scale : nullptr;
  p.v_scale = quantised ? o.v_scale : nullptr;
  p.scale_stride = o.scale_stride;
  p.err = o.device_error;
  p.wide = rows_aligned32(key, ob) && rows_aligned32(value, ob);
  p.i32 = T <= INT32_MAX;
  for (const int64_t x : {p.key_ts, p.key_hs, p.val_ts, p.val_hs, p.kc_s0, p.kc_s1, p.kc_s2, p.vc_s0, p.vc_s1, p.vc_s2})
    p.i32 &= x <= INT32_MAX;
  const int sm = device_sm_count();
  if (sm <= 0) return PA_ERR_CUDA;
  return launch_gather(p, cache_dt, out_dt, sm, static_cast<cudaStream_t>(stream)) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

// ---------------------------------------------------------------- rotary positions

PA_API int pa_rotary_frequencies(int rotary_dim, double base, int scaling, double factor, double original_len,
                                 double low, double high, int64_t *frequencies) {
  if (rotary_dim < 0 || rotary_dim % 2 || (rotary_dim > 0 && !frequencies)) return PA_ERR_INVALID_ARG;
  if (!(base > 0.0) || std::isinf(base) || scaling < PA_ROTARY_PLAIN || scaling > PA_ROTARY_PARTS) return PA_ERR_INVALID_ARG;
  if (scaling != PA_ROTARY_PLAIN && (!(factor > 0.0) || std::isinf(factor))) return PA_ERR_INVALID_ARG;
  if (scaling == PA_ROTARY_BASE && rotary_dim == 2) return PA_ERR_INVALID_ARG;
  if (scaling == PA_ROTARY_PARTS && (!(original_len > 0.0) || std::isinf(original_len) || !(low >= 0.0) || !(high > low) ||
                                     std::isinf(high)))
    return PA_ERR_INVALID_ARG;
  const double two_pi = 6.283185307179586476925;
  const double b = scaling == PA_ROTARY_BASE ? base * std::pow(factor, rotary_dim / (rotary_dim - 2.0)) : base;
  if (!(b > 0.0) || std::isinf(b)) return PA_ERR_INVALID_ARG;
  auto theta = [&](int i) {
    const double x = std::pow(b, -2.0 * i / rotary_dim);
    if (scaling == PA_ROTARY_LINEAR) return x / factor;
    if (scaling != PA_ROTARY_PARTS) return x;
    const double turns = original_len * x / two_pi;  // over the original context
    const double keep = std::min(1.0, std::max(0.0, (turns - low) / (high - low)));
    return keep * x + (1.0 - keep) * (x / factor);
  };
  for (int i = 0; i < rotary_dim / 2; ++i)
    if (!std::isfinite(theta(i))) return PA_ERR_INVALID_ARG;
  for (int i = 0; i < rotary_dim / 2; ++i) {
    const double f = theta(i) / two_pi, part = f - std::floor(f);  // whole turns per position turn nothing
    const double scaled = std::nearbyint(std::ldexp(part, 64));
    const uint64_t bits = scaled >= 0x1p64 ? 0 : static_cast<uint64_t>(scaled);
    frequencies[i] = static_cast<int64_t>(bits);
  }
  return PA_OK;
}

namespace {

// The rows of one kind, [T, H, D], and where they go (nullable): the checks that need no other tensor.
int check_rows(const pa_tensor *x, const pa_tensor *out) {
  int r;
  if ((r = check_desc(x, 3)) || (out && (r = check_desc(out, 3)))) return r;
  if (x->dtype != PA_F32 && x->dtype != PA_BF16 && x->dtype != PA_F16) return PA_ERR_UNSUPPORTED_DTYPE;
  if (x->stride[2] != 1) return PA_ERR_INVALID_ARG;
  if (x->shape[1] > 65535) return PA_ERR_UNSUPPORTED_SHAPE;
  if (!out) return PA_OK;
  if (out->dtype != x->dtype) return PA_ERR_INVALID_ARG;
  for (int i = 0; i < 3; ++i)
    if (out->shape[i] != x->shape[i]) return PA_ERR_INVALID_ARG;
  if (out->stride[2] != 1 || rows_overlap(out, out->shape[2])) return PA_ERR_INVALID_ARG;
  // in place: the same rows at the same places
  if (out->data && out->data == x->data && (out->stride[0] != x->stride[0] || out->stride[1] != x->stride[1]))
    return PA_ERR_INVALID_ARG;
  return PA_OK;
}

int check_row_pointers(const pa_tensor *t) {
  const int eb = elem_bytes(t->dtype);
  if (t->shape[0] == 0 || t->shape[1] == 0) return PA_OK;
  if (!t->data) return PA_ERR_INVALID_ARG;
  if (!aligned16(t->data) || (t->stride[0] * eb) % 16 || (t->stride[1] * eb) % 16) return PA_ERR_ALIGNMENT;
  return PA_OK;
}

int check_weight(const pa_tensor *w, int64_t D, int dtype) {
  int r;
  if (!w) return PA_OK;
  if ((r = check_desc(w, 1))) return r;
  if (w->dtype != PA_F32 && w->dtype != dtype) return PA_ERR_UNSUPPORTED_DTYPE;
  if (w->shape[0] != D || w->stride[0] != 1 || !w->data) return PA_ERR_INVALID_ARG;
  return on_elements(w) ? PA_OK : PA_ERR_ALIGNMENT;
}

// pa_rotary (no caches) and pa_rotary_and_cache (no k_out).
int rotary_impl(pa_tensor *q_out, const pa_tensor *q, pa_tensor *k_out, const pa_tensor *key, const pa_tensor *value,
                pa_tensor *k_cache, pa_tensor *v_cache, const pa_tensor *positions, const pa_tensor *slot_mapping,
                const pa_tensor *frequencies, const pa_tensor *q_weight, const pa_tensor *k_weight, int kv_dtype,
                const pa_rotary_options *opt, pa_stream_t stream, bool cached) {
  const pa_rotary_options o = opt ? *opt : pa_rotary_options{};
  if (o.scale_stride < 0 || !(o.eps >= 0.f) || std::isinf(o.eps)) return PA_ERR_INVALID_ARG;
  int r;
  if (!q != !q_out || (!cached && !key != !k_out) || (cached && (!key || !value || !slot_mapping)) || (!q && !key))
    return PA_ERR_INVALID_ARG;
  if ((q && (r = check_rows(q, q_out))) || (key && (r = check_rows(key, k_out))) || (value && (r = check_rows(value, nullptr))))
    return r;
  const pa_tensor *first = q ? q : key;
  const int dt = first->dtype;
  const int64_t T = first->shape[0], D = first->shape[2];
  for (const pa_tensor *t : {key, value}) {
    if (!t) continue;
    if (t->dtype != dt || t->shape[0] != T || t->shape[2] != D) return PA_ERR_INVALID_ARG;
  }
  if (D != 64 && D != 128 && D != 256) return PA_ERR_UNSUPPORTED_SHAPE;
  int64_t pairs = 0;
  if (frequencies) {
    if ((r = check_desc(frequencies, 1))) return r;
    if (frequencies->dtype != PA_I64) return PA_ERR_UNSUPPORTED_DTYPE;
    pairs = frequencies->shape[0];
    if (pairs > D / 2) return PA_ERR_INVALID_ARG;
    if (pairs % 8) return PA_ERR_UNSUPPORTED_SHAPE;  // (lanes take eight pairs)
    if (pairs > 0 && (frequencies->stride[0] != 1 || !frequencies->data)) return PA_ERR_INVALID_ARG;
    if (pairs > 0 && !on_elements(frequencies)) return PA_ERR_ALIGNMENT;
  }
  if (pairs > 0) {
    if ((r = check_desc(positions, 1))) return r;
    if (positions->dtype != PA_I64 && positions->dtype != PA_I32) return PA_ERR_UNSUPPORTED_DTYPE;
    if (positions->shape[0] != T || positions->stride[0] != 1) return PA_ERR_INVALID_ARG;
  }
  if ((q_weight && !q) || (k_weight && !key)) return PA_ERR_INVALID_ARG;
  if ((r = check_weight(q_weight, D, dt)) || (r = check_weight(k_weight, D, dt))) return r;
  int NB = 0, Hkv = 0, Dc = 0;
  if (cached) {
    if ((r = check_desc(slot_mapping, 1)) || (r = validate_cache_pair(k_cache, v_cache, &NB, &Hkv, &Dc))) return r;
    if (slot_mapping->dtype != PA_I64) return PA_ERR_UNSUPPORTED_DTYPE;
    const int want = kv_dtype == PA_KV_AUTO ? dt : kv_dtype == PA_KV_FP8_E4M3 ? PA_FP8_E4M3 : PA_FP4_E2M1;
    if (kv_dtype != PA_KV_AUTO && kv_dtype != PA_KV_FP8_E4M3 && kv_dtype != PA_KV_FP4_E2M1) return PA_ERR_INVALID_ARG;
    if (k_cache->dtype != want) return PA_ERR_UNSUPPORTED_DTYPE;
    if (Dc != D || key->shape[1] != Hkv || value->shape[1] != Hkv) return PA_ERR_INVALID_ARG;
    if (slot_mapping->shape[0] != T || slot_mapping->stride[0] != 1) return PA_ERR_INVALID_ARG;
  }
  const int64_t Hq = q ? q->shape[1] : 0, Hk = key ? key->shape[1] : 0, Hv = value ? value->shape[1] : 0;
  if (T > INT32_MAX) return PA_ERR_UNSUPPORTED_SHAPE;
  if (T == 0 || Hq + Hk + Hv == 0) return PA_OK;
  for (const pa_tensor *t : {q, static_cast<const pa_tensor *>(q_out), key, static_cast<const pa_tensor *>(k_out), value})
    if (t && (r = check_row_pointers(t))) return r;
  // outputs that overlap an input other than in place, or each other
  const int row_eb = elem_bytes(dt);
  for (const pa_tensor *out : {static_cast<const pa_tensor *>(q_out), static_cast<const pa_tensor *>(k_out)}) {
    if (!out) continue;
    const pa_tensor *own = out == q_out ? q : key;
    for (const pa_tensor *x : {q, key, value, out == q_out ? static_cast<const pa_tensor *>(k_out) : nullptr})
      if (x && !(x == own && x->data == out->data) && rows_shared(x, out, row_eb)) return PA_ERR_INVALID_ARG;
  }
  if (pairs > 0 && !positions->data) return PA_ERR_INVALID_ARG;
  if (pairs > 0 && !on_elements(positions)) return PA_ERR_ALIGNMENT;
  if (cached && !slot_mapping->data) return PA_ERR_INVALID_ARG;
  if (cached && !on_elements(slot_mapping)) return PA_ERR_ALIGNMENT;
  if (!aligned4(o.k_scale) || !aligned4(o.v_scale) || !aligned4(o.device_error)) return PA_ERR_ALIGNMENT;

  const int eb = elem_bytes(dt);
  RotaryParams p{};
  p.T = T;
  p.D = static_cast<int>(D);
  p.R = static_cast<int>(2 * pairs);
  p.Hq = static_cast<int>(Hq);
  p.Hk = static_cast<int>(Hk);
  p.Hv = static_cast<int>(Hv);
  p.wide = true;
  auto rows = [&](const pa_tensor *t, int64_t &ts, int64_t &hs) {
    if (!t) return static_cast<char *>(nullptr);
    ts = t->stride[0] * eb;
    hs = t->stride[1] * eb;
    p.wide = p.wide && rows_aligned32(t, eb);
    return static_cast<char *>(t->data);
  };
  p.q = rows(q, p.q_ts, p.q_hs);
  p.q_out = rows(q_out, p.qo_ts, p.qo_hs);
  p.key = rows(key, p.key_ts, p.key_hs);
  p.k_out = rows(k_out, p.ko_ts, p.ko_hs);
  p.value = rows(value, p.val_ts, p.val_hs);
  if (pairs > 0) {
    p.positions = positions->data;
    p.pos64 = positions->dtype == PA_I64;
    p.frequencies = static_cast<const uint64_t *>(frequencies->data);
  }
  if (q_weight) {
    p.q_weight = q_weight->data;
    p.q_weight_dtype = q_weight->dtype;
  }
  if (k_weight) {
    p.k_weight = k_weight->data;
    p.k_weight_dtype = k_weight->dtype;
  }
  p.magnitude = o.magnitude == 0.f ? 1.f : o.magnitude;
  p.eps = o.eps;
  p.interleaved = o.interleaved != 0;
  p.err = o.device_error;
  if (cached) {
    const int cb = elem_bytes(k_cache->dtype);
    const bool paged4 = k_cache->dtype == PA_FP4_E2M1;
    p.slots = static_cast<const int64_t *>(slot_mapping->data);
    p.k_cache = static_cast<char *>(k_cache->data);
    p.v_cache = static_cast<char *>(v_cache->data);
    p.kc_s0 = k_cache->stride[0] * cb;
    p.kc_s1 = k_cache->stride[1] * cb;
    p.kc_s2 = paged4 ? 0 : k_cache->stride[2] * cb;
    p.vc_s0 = v_cache->stride[0] * cb;
    p.vc_s1 = v_cache->stride[1] * cb;
    p.vc_s2 = paged4 ? 0 : v_cache->stride[2] * cb;
    p.num_slots = static_cast<int64_t>(NB) * kBlock;
    if (kv_dtype == PA_KV_AUTO) {
      for (const pa_tensor *c : {k_cache, v_cache})
        p.wide = p.wide && rows_aligned32(c, cb) && (c->stride[2] * cb) % 32 == 0;
    } else {
      p.k_scale = o.k_scale;
      p.v_scale = o.v_scale;
      p.scale_stride = o.scale_stride;
    }
  }
  const int sm = device_sm_count();
  if (sm <= 0) return PA_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int cache_dtype = cached ? static_cast<int>(k_cache->dtype) : dt;
  auto launch = [&] {
    const cudaError_t e = dt == PA_F32    ? launch_rotary_f32(p, cache_dtype, sm, st)
                          : dt == PA_BF16 ? launch_rotary_bf16(p, cache_dtype, sm, st)
                                          : launch_rotary_f16(p, cache_dtype, sm, st);
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
  };
  if (!cached) return launch();
  ProfScope ps(PA_KERNEL_WRITE, st);
  return launch();
}

}  // namespace

PA_API int pa_rotary(pa_tensor *q_out, const pa_tensor *q, pa_tensor *k_out, const pa_tensor *key,
                     const pa_tensor *positions, const pa_tensor *frequencies, const pa_tensor *q_weight,
                     const pa_tensor *k_weight, const pa_rotary_options *opt, pa_stream_t stream) {
  return rotary_impl(q_out, q, k_out, key, nullptr, nullptr, nullptr, positions, nullptr, frequencies, q_weight,
                     k_weight, PA_KV_AUTO, opt, stream, false);
}

PA_API int pa_rotary_and_cache(pa_tensor *q_out, const pa_tensor *q, const pa_tensor *key, const pa_tensor *value,
                               pa_tensor *k_cache, pa_tensor *v_cache, const pa_tensor *positions,
                               const pa_tensor *slot_mapping, const pa_tensor *frequencies, const pa_tensor *q_weight,
                               const pa_tensor *k_weight, int kv_dtype, const pa_rotary_options *opt,
                               pa_stream_t stream) {
  return rotary_impl(q_out, q, nullptr, key, value, k_cache, v_cache, positions, slot_mapping, frequencies, q_weight,
                     k_weight, kv_dtype, opt, stream, true);
}

// A decode kernel that reads a cache of this element type, -1 for none.
static int kind_of_cache(int dtype) {
  switch (dtype) {
    case PA_FP8_E4M3: return KIND_FP8_BF16Q;
    case PA_FP4_E2M1: return KIND_FP4_BF16Q;
    case PA_BF16: return KIND_BF16;
    case PA_F16: return KIND_F16;
    case PA_F32: return KIND_F32;
    default: return -1;
  }
}

PA_API int pa_decode_plan(int num_seqs, int num_heads, int num_kv_heads, int head_size, int max_blocks_per_seq,
                          int kv_dtype_code, int sm_count, int partition_size, int *partition_out,
                          int *num_partitions_out) {
  if (num_seqs < 0 || num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads || head_size <= 0 ||
      max_blocks_per_seq < 0)
    return PA_ERR_INVALID_ARG;
  const int kind = kind_of_cache(kv_dtype_code);
  if (kind < 0) return PA_ERR_INVALID_ARG;
  const bool device = sm_count <= 0;
  if (device) sm_count = device_sm_count();
  if (sm_count <= 0) return PA_ERR_CUDA;
  const Plan pl = make_plan(num_seqs, num_heads, num_kv_heads, head_size, max_blocks_per_seq, kind, sm_count, device,
                            partition_size);
  if (pl.status != PA_OK) return pl.status;
  if (partition_out) *partition_out = pl.flat > 0 ? PA_PARTITION_BALANCED : pl.cluster > 1 ? -pl.cluster : pl.P;
  if (num_partitions_out)
    *num_partitions_out = pl.flat > 0       ? pl.flat
                          : pl.cluster > 1 ? pl.cluster
                          : pl.P > 0       ? (max_blocks_per_seq * kBlock + pl.P - 1) / pl.P
                                           : 1;
  return PA_OK;
}

PA_API size_t pa_decode_workspace_size(int num_seqs, int num_heads, int num_kv_heads, int head_size,
                                       int max_blocks_per_seq, int partition_size) {
  if (num_seqs < 0 || num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads || head_size < 0 ||
      max_blocks_per_seq < 0)
    return 0;
  if (partition_size == PA_PARTITION_BALANCED) {
    // enough for any cache type on the current device: the shared-memory bounds of the
    // quantised kernels admit the most CTAs per SM
    const int sm = device_sm_count();
    if (sm <= 0 || num_seqs > kFlatMaxSeqs) return 0;
    const int kind = head_size >= 128 ? KIND_FP8_BF16Q : KIND_BF16, kind4 = KIND_FP4_BF16Q;
    int flat = std::max(balanced_ctas(num_heads, num_kv_heads, head_size, kind, sm, false),
                        balanced_ctas(num_heads, num_kv_heads, head_size, kind4, sm, false));
    // 4-bit caches: split over warps, or (ALiBi, several query tokens) into fixed partitions
    Plan pl{0, 0, 0, PA_OK, 0, 0};
    if (plan_fp4(num_seqs, num_heads, num_kv_heads, head_size, max_blocks_per_seq, kind4, sm, false, false, true, true,
                 &pl))
      flat = std::max(flat, pl.flat);
    const int P = plan_partition(num_seqs, num_heads, num_kv_heads, head_size, max_blocks_per_seq, kind4, sm, true, 0);
    return std::max(workspace_layout(num_seqs, num_heads, num_kv_heads, head_size, max_blocks_per_seq, 0, flat).total,
                    workspace_layout(num_seqs, num_heads, num_kv_heads, head_size, max_blocks_per_seq, P, 0).total);
  }
  const int P = partition_size > 0 ? (partition_size + kBlock - 1) / kBlock * kBlock : 0;
  if (P >= max_blocks_per_seq * kBlock) return 0;
  return workspace_layout(num_seqs, num_heads, num_kv_heads, head_size, max_blocks_per_seq, P, 0).total;
}

PA_API size_t pa_decode_window_workspace_size(int num_seqs, int num_heads, int num_kv_heads, int head_size,
                                              int max_blocks_per_seq, int kv_dtype_code, int window, int sinks,
                                              int max_query_len, int partition_size) {
  const int kind = kind_of_cache(kv_dtype_code);
  if (num_seqs < 0 || num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads || head_size <= 0 ||
      max_blocks_per_seq < 0 || max_blocks_per_seq > INT32_MAX / kBlock || kind < 0 || window < 1 || sinks < 0 ||
      max_query_len < 1 || static_cast<int64_t>(num_heads) * max_query_len > INT32_MAX)
    return 0;
  const int sm = device_sm_count();
  if (sm <= 0) return 0;
  const int Hqv = num_heads * max_query_len;
  const bool whole = static_cast<int64_t>(window) + sinks >= static_cast<int64_t>(max_blocks_per_seq) * kBlock;
  const WidenPlan wide = widen_plan(num_seqs, num_kv_heads, head_size, max_blocks_per_seq, kind, partition_size,
                                    Hqv / num_kv_heads, max_query_len,
                                    static_cast<int64_t>(num_seqs) * max_query_len, whole ? 0 : window, sinks);
  if (wide.pages > 0) return arrival_counter_bytes(num_seqs, Hqv, num_kv_heads) + wide.total;
  if (max_query_len > 1 && on_query_tiles(kind, head_size, partition_size, Hqv / num_kv_heads, !whole)) return 0;
  size_t need = 0;
  for (const bool varlen : {false, true}) {  // (a call of pa_attention_window may have one query each, too)
    if (!varlen && max_query_len > 1) continue;
    if (varlen && partition_size == PA_PARTITION_BALANCED) continue;
    int NB = max_blocks_per_seq;
    Plan pl;
    if (whole) {
      for (const bool plain : {false, true}) {
        pl = make_plan(num_seqs, Hqv, num_kv_heads, head_size, NB, kind, sm, true, partition_size, varlen, plain);
        if (pl.status == PA_OK && pl.cluster == 0 && (pl.flat > 0 || (pl.P > 0 && pl.P < NB * kBlock)))
          need = std::max(need, workspace_layout(num_seqs, Hqv, num_kv_heads, head_size, NB, pl.P, pl.flat).total);
      }
      continue;
    }
    NB = window_blocks(NB, window, sinks, num_heads / num_kv_heads, max_query_len);
    pl = make_window_plan(num_seqs, Hqv, num_kv_heads, head_size, NB, kind, sm, true, partition_size, varlen, true);
    if (pl.status == PA_OK && pl.cluster == 0 && (pl.flat > 0 || (pl.P > 0 && pl.P < NB * kBlock)))
      need = std::max(need, workspace_layout(num_seqs, Hqv, num_kv_heads, head_size, NB, pl.P, pl.flat).total);
  }
  return need;
}

PA_API size_t pa_decode_accumulate_workspace_size(int num_seqs, int num_heads, int num_kv_heads, int head_size,
                                                  int max_blocks_per_seq, int partition_size) {
  if (num_seqs < 0 || num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads || head_size < 0 ||
      max_blocks_per_seq < 0 || (partition_size < -1 && partition_size != PA_PARTITION_BALANCED))
    return 0;
  return round256(pa_decode_workspace_size(num_seqs, num_heads, num_kv_heads, head_size, max_blocks_per_seq,
                                           partition_size)) +
         score_layout(num_seqs, num_heads, num_kv_heads, max_blocks_per_seq).total;
}

namespace {

// Decode (query_start_loc == NULL: one query token per sequence, q [S, Hq, D]) or varlen
// attention (q [Tq, Hq, D] packed, query_start_loc [S + 1], at most max_query_len tokens
// per sequence).
int decode_impl(pa_tensor *out, const pa_tensor *q, const pa_tensor *k_cache, const pa_tensor *v_cache,
                const pa_tensor *block_table, const pa_tensor *seq_lens, float scale, int num_kv_heads,
                const pa_decode_options &o, bool internal_ws, pa_stream_t stream,
                const pa_tensor *query_start_loc = nullptr, int max_query_len = 1,
                const pa_tensor *new_rows_start = nullptr, bool early = false, bool dry = false,
                size_t *ws_need = nullptr, size_t *ws_counters = nullptr, pa_tensor *weights = nullptr,
                int64_t window = 0, int64_t sinks = 0) {
  const float *k_scale = o.k_scale, *v_scale = o.v_scale;
  const int partition_size = o.partition_size;
  void *workspace = o.workspace;
  size_t workspace_bytes = o.workspace_bytes;
  int *device_error = o.device_error;
  if (o.scale_stride < 0) return PA_ERR_INVALID_ARG;
  int r;
  if ((r = check_desc(out, 3)) || (r = check_desc(q, 3)) || (r = check_desc(block_table, 2)) ||
      (r = check_desc(seq_lens, 1)))
    return r;
  int NB, Hkv, D;
  if ((r = validate_cache_pair(k_cache, v_cache, &NB, &Hkv, &D))) return r;
  const bool varlen = query_start_loc != nullptr;
  const int64_t S64 = varlen ? seq_lens->shape[0] : q->shape[0], Hq64 = q->shape[1];
  if (num_kv_heads != Hkv || Hkv <= 0 || Hq64 <= 0 || Hq64 % Hkv) return PA_ERR_INVALID_ARG;
  if (varlen) {
    if ((r = check_desc(query_start_loc, 1))) return r;
    if (query_start_loc->dtype != PA_I32) return PA_ERR_UNSUPPORTED_DTYPE;
    if (query_start_loc->shape[0] != S64 + 1 || query_start_loc->stride[0] != 1 || !query_start_loc->data)
      return PA_ERR_INVALID_ARG;
    if (max_query_len < 1) return PA_ERR_INVALID_ARG;
    if (o.partition_size == PA_PARTITION_BALANCED) return PA_ERR_UNSUPPORTED_SHAPE;
    if (static_cast<int64_t>(max_query_len) * (Hq64 / Hkv) > (1 << 20)) return PA_ERR_UNSUPPORTED_SHAPE;
  }
  if (q->shape[2] != D) return PA_ERR_INVALID_ARG;
  for (int i = 0; i < 3; ++i)
    if (out->shape[i] != q->shape[i]) return PA_ERR_INVALID_ARG;
  if (out->dtype != q->dtype) return PA_ERR_INVALID_ARG;
  if (block_table->dtype != PA_I32 || seq_lens->dtype != PA_I32) return PA_ERR_UNSUPPORTED_DTYPE;
  if (block_table->shape[0] != S64 || seq_lens->shape[0] != S64) return PA_ERR_INVALID_ARG;
  if (block_table->stride[1] != 1 || seq_lens->stride[0] != 1 || q->stride[2] != 1 || out->stride[2] != 1)
    return PA_ERR_INVALID_ARG;
  const int kind = kind_of(q->dtype, k_cache->dtype);
  if (kind < 0) return PA_ERR_UNSUPPORTED_DTYPE;
  if (D != 64 && D != 128 && D != 256) return PA_ERR_UNSUPPORTED_SHAPE;
  if ((kind == KIND_FP8_BF16Q || kind == KIND_FP8_F16Q) && D < 128) return PA_ERR_UNSUPPORTED_SHAPE;
  if (mma_fp4(kind)) {  // block 0 stands in for entries behind a sequence; 32-bit block strides
    if (NB == 0 && S64 > 0) return PA_ERR_INVALID_ARG;
    if (k_cache->stride[0] > UINT32_MAX || v_cache->stride[0] > UINT32_MAX) return PA_ERR_UNSUPPORTED_SHAPE;
    if (block_table->shape[1] > (1 << 26)) return PA_ERR_UNSUPPORTED_SHAPE;  // lengths rounded up to stages of 64 tokens
  }
  if (S64 > 65535 || Hq64 > 65535 || block_table->shape[1] > (INT32_MAX / kBlock)) return PA_ERR_UNSUPPORTED_SHAPE;
  if (early && new_rows_start) {
    if ((r = check_desc(new_rows_start, 1))) return r;
    if (new_rows_start->dtype != PA_I32) return PA_ERR_UNSUPPORTED_DTYPE;
    if (new_rows_start->shape[0] != S64 + 1 || new_rows_start->stride[0] != 1) return PA_ERR_INVALID_ARG;
    if (S64 > 0 && !new_rows_start->data) return PA_ERR_INVALID_ARG;
  }
  if (weights) {
    if ((r = check_desc(weights, 3))) return r;
    if (weights->dtype != PA_F32) return PA_ERR_UNSUPPORTED_DTYPE;
    if (weights->shape[0] != S64 || weights->shape[1] != Hkv || weights->shape[2] < block_table->shape[1] * kBlock ||
        weights->stride[2] != 1 || rows_overlap(weights, block_table->shape[1] * kBlock))
      return PA_ERR_INVALID_ARG;
    if (o.partition_size < -1 && o.partition_size != PA_PARTITION_BALANCED)
      return PA_ERR_UNSUPPORTED_SHAPE;  // cluster splits
    // (the second kernel counts tokens in 32 bits, up to a grid's stride past the last)
    if (block_table->shape[1] > (1 << 26)) return PA_ERR_UNSUPPORTED_SHAPE;
  }
  if (S64 == 0 || q->shape[0] == 0) return PA_OK;
  if (weights && block_table->shape[1] > 0 && !weights->data) return PA_ERR_INVALID_ARG;
  if (!q->data || !out->data || !block_table->data || !seq_lens->data) return PA_ERR_INVALID_ARG;
  for (const pa_tensor *t : {block_table, seq_lens, query_start_loc, early ? new_rows_start : nullptr,
                             static_cast<const pa_tensor *>(weights)})
    if (t && !on_elements(t)) return PA_ERR_ALIGNMENT;
  for (const void *x : {static_cast<const void *>(k_scale), static_cast<const void *>(v_scale),
                        static_cast<const void *>(o.alibi_slopes), static_cast<const void *>(device_error)})
    if (!aligned4(x)) return PA_ERR_ALIGNMENT;
  const int qb = elem_bytes(q->dtype);
  if (!aligned16(q->data) || !aligned16(out->data)) return PA_ERR_ALIGNMENT;
  for (int i = 0; i < 2; ++i)
    if ((q->stride[i] * qb) % 16 || (out->stride[i] * qb) % 16) return PA_ERR_ALIGNMENT;

  const int S = static_cast<int>(S64), Hq = static_cast<int>(Hq64);
  // query columns per KV head ("virtual heads"): G for decode, G per query token for varlen;
  // plans and workspace count them like query heads
  const int VH = (Hq / Hkv) * (varlen ? max_query_len : 1);
  const int Hqv = Hkv * VH;
  const int maxNB = static_cast<int>(block_table->shape[1]);
  if (window + sinks >= static_cast<int64_t>(maxNB) * kBlock) window = sinks = 0;  // every token is seen
  // pages that a work item reads at most
  const int NBw = window > 0 ? window_blocks(maxNB, window, sinks, Hq / Hkv, varlen ? max_query_len : 1) : maxNB;
  const int sm = device_sm_count();
  if (sm <= 0) return PA_ERR_CUDA;
  bool chunk = varlen && on_query_tiles(kind, D, partition_size, VH, window > 0);
  // over a quantised cache: its seen pages widened first, where there is room for them
  const WidenPlan wide = varlen ? widen_plan(S, Hkv, D, maxNB, kind, partition_size, VH, max_query_len, q->shape[0],
                                             window, sinks)
                                : WidenPlan{0, 0, 0};
  char *scratch = nullptr;
  if (wide.pages > 0 && !dry) {
    if (internal_ws) {
      DevWorkspace w;
      if (internal_workspace(0, wide.total, static_cast<cudaStream_t>(stream), &w, true) == PA_OK)
        scratch = static_cast<char *>(w.ptr) + w.counters;
    } else if (workspace && aligned16(workspace) && workspace_bytes >= arrival_counter_bytes(S, Hqv, Hkv) + wide.total) {
      scratch = static_cast<char *>(workspace) + arrival_counter_bytes(S, Hqv, Hkv);  // (the counters stay at zero)
    }
    chunk = scratch != nullptr;
  }
  const Plan pl = window > 0 ? make_window_plan(S, Hqv, Hkv, D, NBw, kind, sm, true, chunk ? -1 : partition_size, varlen,
                                                !varlen && !o.alibi_slopes)
                             : make_plan(S, Hqv, Hkv, D, maxNB, kind, sm, true, chunk ? -1 : partition_size, varlen,
                                         !varlen && !o.alibi_slopes);
  if (pl.status != PA_OK) return pl.status;
  const int P = pl.P;
  const int max_parts = pl.cluster > 1 ? pl.cluster : P > 0 ? (NBw * kBlock + P - 1) / P : 1;
  cudaStream_t st = static_cast<cudaStream_t>(stream);

  DecodeParams p{};
  p.out = out->data;
  p.q = q->data;
  p.out_ss = out->stride[0];
  p.out_hs = out->stride[1];
  p.q_ss = q->stride[0];
  p.q_hs = q->stride[1];
  p.block_table = static_cast<const int32_t *>(block_table->data);
  p.bt_ss = block_table->stride[0];
  p.seq_lens = static_cast<const int32_t *>(seq_lens->data);
  p.S = S;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = Hq / Hkv;
  p.VH = VH;
  p.HG = (VH + 7) / 8;
  p.qsl = varlen ? static_cast<const int32_t *>(query_start_loc->data) : nullptr;
  p.nq_max = varlen ? max_query_len : 1;
  p.Tq = q->shape[0];
  p.D = D;
  p.num_blocks = NB;
  p.max_blocks = maxNB;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.scale_stride = o.scale_stride;
  p.alibi = o.alibi_slopes;
  p.window = static_cast<int>(window);
  p.narrow = pl.narrow;
  p.sinks = static_cast<int>(sinks);
  p.pages_per_part = P > 0 ? P / kBlock : std::max(maxNB, 1);
  p.max_parts = max_parts;
  p.cluster = pl.cluster;
  p.flat = pl.flat;
  p.first_wait_limit = o.first_wait_limit;
  p.early = early && !varlen ? 1 : 0;
  p.new_start = p.early && new_rows_start ? static_cast<const int32_t *>(new_rows_start->data) : nullptr;
  p.err = device_error;
  {
    // Order the batch longest-first only when its CTAs cannot all be resident at once:
    // with every CTA resident from the start the order buys nothing and the ranking
    // (a read of every length plus two block barriers) sits on each CTA's critical path.
    const int64_t ctas = static_cast<int64_t>(S) * Hkv * p.HG * max_parts;
    const int64_t slots = static_cast<int64_t>(sm) * ctas_per_sm(kind, D, true) * (pl.narrow ? 2 : 1);
    p.lpt = (pl.flat == 0 && longest_first(kind, S) && ctas > slots)
                ? 1
                : 0;
  }
  if (!mma_fp8(kind) && !mma_fp4(kind)) p.k_scale = p.v_scale = nullptr;
  if (static_cast<int64_t>(p.Hkv) * p.HG > 65535) return PA_ERR_UNSUPPORTED_SHAPE;
  // (made before a dry run ends: a layout or a stride that a map cannot take is a refusal too)
  CUtensorMap tmK{}, tmV{};
  if (kind != KIND_F32 && !mma_fp4(kind)) {
    int nhd_k = 0, nhd_v = 0;
    if ((r = make_cache_map(k_cache, &tmK, &nhd_k)) || (r = make_cache_map(v_cache, &tmV, &nhd_v))) return r;
    if (nhd_k != nhd_v) return PA_ERR_INVALID_ARG;  // K and V in different layouts
    p.nhd = nhd_k;
  }

  if (dry) {  // validation only (pa_decode_step checks everything before its first launch)
    if ((max_parts > 1 && pl.cluster <= 1) || pl.flat > 0) {
      const WsLayout lay = workspace_layout(S, Hqv, Hkv, D, maxNB, P, pl.flat);
      if (ws_need) *ws_need = lay.total;
      if (ws_counters) *ws_counters = lay.ml_off;
      if (!internal_ws) {
        if (!workspace || workspace_bytes < lay.total) return PA_ERR_WORKSPACE;
        if (!aligned16(workspace)) return PA_ERR_ALIGNMENT;
      }
    }
    return PA_OK;
  }
  size_t to_clear = 0;
  if ((max_parts > 1 && pl.cluster <= 1) || pl.flat > 0 || weights) {
    const WsLayout lay = workspace_layout(S, Hqv, Hkv, D, NBw, max_parts > 1 ? P : 0, pl.flat);
    const ScoreLayout sc = weights ? score_layout(S, Hq, Hkv, maxNB) : ScoreLayout{0, 0, 0};
    const size_t total = weights ? round256(lay.total) + sc.total : lay.total;
    size_t ml_off = lay.ml_off;
    if (internal_ws) {
      DevWorkspace w;
      if ((r = internal_workspace(lay.ml_off, total - lay.ml_off, st, &w))) return r;
      workspace = w.ptr;
      ml_off = w.counters;
    } else {
      if (!workspace || workspace_bytes < total) return PA_ERR_WORKSPACE;
      if (!aligned16(workspace)) return PA_ERR_ALIGNMENT;
      if (weights && lay.total == 0) {
        // an unsplit call has no arrival counters, but the next call may: its scores lie behind their
        // place where there is room, else that place is cleared afterwards
        const size_t counters = arrival_counter_bytes(S, Hqv, Hkv);
        if (workspace_bytes - total >= counters) ml_off = counters;
        else to_clear = counters;
      }
    }
    if (weights) {
      char *base = static_cast<char *>(workspace) + ml_off + (round256(lay.total) - lay.ml_off);
      p.lse = reinterpret_cast<float *>(base);
      p.scores = reinterpret_cast<float *>(base + sc.scores_off);
      p.score_cols = sc.cols;
    }
    p.counters = static_cast<int *>(workspace);
    p.part_ml = reinterpret_cast<float2 *>(static_cast<char *>(workspace) + ml_off);
    p.part_acc = reinterpret_cast<float *>(static_cast<char *>(workspace) + ml_off + (lay.acc_off - lay.ml_off));
  }

  cudaError_t e;
  int tile_kind = kind;  // of the query tiles
  if (scratch) {
    WidenParams w{};
    const int eb = elem_bytes(k_cache->dtype);
    const bool paged4 = mma_fp4(kind);
    w.k_cache = static_cast<const char *>(k_cache->data);
    w.v_cache = static_cast<const char *>(v_cache->data);
    w.kc_s0 = k_cache->stride[0] * eb;
    w.kc_s1 = k_cache->stride[1] * eb;
    w.kc_s2 = paged4 ? 0 : k_cache->stride[2] * eb;
    w.vc_s0 = v_cache->stride[0] * eb;
    w.vc_s1 = v_cache->stride[1] * eb;
    w.vc_s2 = paged4 ? 0 : v_cache->stride[2] * eb;
    w.block_table = p.block_table;
    w.bt_ss = p.bt_ss;
    w.seq_lens = p.seq_lens;
    w.qsl = p.qsl;
    w.Tq = p.Tq;
    w.S = S;
    w.Hkv = Hkv;
    w.D = D;
    w.num_blocks = NB;
    w.max_blocks = maxNB;
    w.nq_max = p.nq_max;
    w.window = p.window;
    w.sinks = p.sinks;
    w.pages = wide.pages;
    w.k_out = scratch;
    w.v_out = scratch + wide.table / 2;
    w.table = reinterpret_cast<int32_t *>(scratch + wide.table);
    w.err = device_error;
    w.wide = (reinterpret_cast<uintptr_t>(scratch) & 31u) == 0;  // (each cache's pages are a multiple of 2 KiB)
    pa_tensor pages{};
    pages.dtype = q->dtype;
    pages.ndim = 4;
    const int64_t extents[4] = {static_cast<int64_t>(S) * wide.pages, Hkv, kBlock, D};
    int64_t step = 1;
    for (int i = 3; i >= 0; --i) {
      pages.shape[i] = extents[i];
      pages.stride[i] = step;
      step *= extents[i];
    }
    pages.data = w.k_out;
    if ((r = make_cache_map(&pages, &tmK, &p.nhd))) return r;
    pages.data = w.v_out;
    if ((r = make_cache_map(&pages, &tmV, &p.nhd))) return r;
    {
      ProfScope ps(PA_KERNEL_DECODE, st);
      e = launch_widen(w, k_cache->dtype, q->dtype, st);
    }
    if (e != cudaSuccess) return PA_ERR_CUDA;
    p.block_table = w.table;
    p.bt_ss = maxNB;
    p.num_blocks = S * wide.pages;
    tile_kind = q->dtype == PA_BF16 ? KIND_BF16 : KIND_F16;
  }
  if (kind == KIND_F32) {
    p.kc = static_cast<const float *>(k_cache->data);
    p.vc = static_cast<const float *>(v_cache->data);
    p.kc_s0 = k_cache->stride[0];
    p.kc_s1 = k_cache->stride[1];
    p.kc_s2 = k_cache->stride[2];
    p.vc_s0 = v_cache->stride[0];
    p.vc_s1 = v_cache->stride[1];
    p.vc_s2 = v_cache->stride[2];
    ProfScope ps(PA_KERNEL_DECODE, st);
    e = launch_decode_f32(p, st);
  } else if (mma_fp4(kind) && !scratch) {
    p.k4 = static_cast<const char *>(k_cache->data);
    p.v4 = static_cast<const char *>(v_cache->data);
    p.kc_s0 = k_cache->stride[0];
    p.kc_s1 = k_cache->stride[1];
    p.vc_s0 = v_cache->stride[0];
    p.vc_s1 = v_cache->stride[1];
    ProfScope ps(PA_KERNEL_DECODE, st);
    e = pl.warps        ? launch_decode_fp4_warps(p, kind, sm * mma_min_ctas(kind, D), st)
        : p.window > 0 ? launch_decode_window_fp4(p, kind, st)
                       : launch_decode_mma_fp4(p, kind, st);
  } else {
    ProfScope ps(PA_KERNEL_DECODE, st);
    if (chunk) {
      CUtensorMap tmQ{};
      p.q_tma = make_q_map(q, p.G, &tmQ) == PA_OK ? 1 : 0;
      e = p.window > 0 ? launch_chunk_window(p, tile_kind, tmK, tmV, tmQ, st) : launch_chunk_umma(p, kind, tmK, tmV, tmQ, st);
    } else if (kind == KIND_BF16 || kind == KIND_F16) {
      e = p.window > 0 ? launch_decode_window_16(p, kind, tmK, tmV, st) : launch_decode_mma_16(p, kind, tmK, tmV, st);
    } else {
      e = p.window > 0 ? launch_decode_window_fp8(p, kind, tmK, tmV, st) : launch_decode_mma_fp8(p, kind, tmK, tmV, st);
    }
  }
  if (e == cudaSuccess && weights && maxNB > 0) {
    WeightsParams w{};
    w.seq_lens = p.seq_lens;
    w.scores = p.scores;
    w.lse = p.lse;
    w.weights = static_cast<float *>(weights->data);
    w.w_ss = weights->stride[0];
    w.w_hs = weights->stride[1];
    w.S = S;
    w.Hkv = Hkv;
    w.G = p.G;
    w.HG = p.HG;
    w.max_tokens = maxNB * kBlock;
    ProfScope ps(PA_KERNEL_DECODE, st);
    e = launch_weights(w, p.score_cols, st);
  }
  if (e == cudaSuccess && to_clear) e = cudaMemsetAsync(workspace, 0, to_clear, st);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace

int pa::decode_ex_requirements(pa_tensor *out, const pa_tensor *q, const pa_tensor *k_cache, const pa_tensor *v_cache,
                           const pa_tensor *block_table, const pa_tensor *seq_lens, float scale, int num_kv_heads,
                           const float *k_scale, const float *v_scale, int partition_size, int *device_error,
                           size_t *ws_bytes, size_t *counter_bytes) {
  pa_decode_options o{};
  o.k_scale = k_scale;
  o.v_scale = v_scale;
  o.partition_size = partition_size;
  o.device_error = device_error;
  *ws_bytes = 0;
  *counter_bytes = 0;
  // internal_ws: the workspace is not checked here (the caller supplies it afterwards)
  return decode_impl(out, q, k_cache, v_cache, block_table, seq_lens, scale, num_kv_heads, o, true, nullptr,
                     nullptr, 1, nullptr, false, true, ws_bytes, counter_bytes);
}

PA_API int pa_decode_ex(pa_tensor *out, const pa_tensor *q, const pa_tensor *k_cache, const pa_tensor *v_cache,
                        const pa_tensor *block_table, const pa_tensor *seq_lens, float scale, int num_kv_heads,
                        const float *k_scale, const float *v_scale, int partition_size, void *workspace,
                        size_t workspace_bytes, int *device_error, pa_stream_t stream) {
  pa_decode_options o{};
  o.k_scale = k_scale;
  o.v_scale = v_scale;
  o.partition_size = partition_size;
  o.workspace = workspace;
  o.workspace_bytes = workspace_bytes;
  o.device_error = device_error;
  return decode_impl(out, q, k_cache, v_cache, block_table, seq_lens, scale, num_kv_heads, o, false, stream);
}

PA_API int pa_decode(pa_tensor *out, const pa_tensor *q, const pa_tensor *k_cache, const pa_tensor *v_cache,
                     const pa_tensor *block_table, const pa_tensor *seq_lens, float scale, int num_kv_heads,
                     pa_stream_t stream) {
  const pa_decode_options o{};
  return decode_impl(out, q, k_cache, v_cache, block_table, seq_lens, scale, num_kv_heads, o, true, stream);
}

PA_API int pa_decode_opt(pa_tensor *out, const pa_tensor *q, const pa_tensor *k_cache, const pa_tensor *v_cache,
                         const pa_tensor *block_table, const pa_tensor *seq_lens, float scale, int num_kv_heads,
                         const pa_decode_options *opt, pa_stream_t stream) {
  const pa_decode_options o = opt ? *opt : pa_decode_options{};
  const bool internal = !o.workspace && o.workspace_bytes == 0;
  return decode_impl(out, q, k_cache, v_cache, block_table, seq_lens, scale, num_kv_heads, o, internal, stream);
}

PA_API int pa_decode_accumulate(pa_tensor *out, const pa_tensor *q, const pa_tensor *k_cache, const pa_tensor *v_cache,
                                const pa_tensor *block_table, const pa_tensor *seq_lens, float scale, int num_kv_heads,
                                pa_tensor *weights, const pa_decode_options *opt, pa_stream_t stream) {
  if (!weights) return PA_ERR_INVALID_ARG;
  const pa_decode_options o = opt ? *opt : pa_decode_options{};
  const bool internal = !o.workspace && o.workspace_bytes == 0;
  return decode_impl(out, q, k_cache, v_cache, block_table, seq_lens, scale, num_kv_heads, o, internal, stream,
                     nullptr, 1, nullptr, false, false, nullptr, nullptr, weights);
}

PA_API int pa_attention_varlen(pa_tensor *out, const pa_tensor *q, const pa_tensor *k_cache, const pa_tensor *v_cache,
                               const pa_tensor *query_start_loc, const pa_tensor *block_table,
                               const pa_tensor *seq_lens, float scale, int num_kv_heads, int max_query_len,
                               const pa_decode_options *opt, pa_stream_t stream) {
  if (!query_start_loc) return PA_ERR_INVALID_ARG;
  const pa_decode_options o = opt ? *opt : pa_decode_options{};
  const bool internal = !o.workspace && o.workspace_bytes == 0;
  return decode_impl(out, q, k_cache, v_cache, block_table, seq_lens, scale, num_kv_heads, o, internal, stream,
                     query_start_loc, max_query_len);
}

PA_API int pa_decode_window(pa_tensor *out, const pa_tensor *q, const pa_tensor *k_cache, const pa_tensor *v_cache,
                            const pa_tensor *block_table, const pa_tensor *seq_lens, float scale, int num_kv_heads,
                            int window, int sinks, const pa_decode_options *opt, pa_stream_t stream) {
  if (window < 1 || sinks < 0) return PA_ERR_INVALID_ARG;
  const pa_decode_options o = opt ? *opt : pa_decode_options{};
  const bool internal = !o.workspace && o.workspace_bytes == 0;
  return decode_impl(out, q, k_cache, v_cache, block_table, seq_lens, scale, num_kv_heads, o, internal, stream,
                     nullptr, 1, nullptr, false, false, nullptr, nullptr, nullptr, window, sinks);
}

PA_API int pa_attention_window(pa_tensor *out, const pa_tensor *q, const pa_tensor *k_cache, const pa_tensor *v_cache,
                               const pa_tensor *query_start_loc, const pa_tensor *block_table,
                               const pa_tensor *seq_lens, float scale, int num_kv_heads, int max_query_len, int window,
                               int sinks, const pa_decode_options *opt, pa_stream_t stream) {
  if (!query_start_loc || window < 1 || sinks < 0) return PA_ERR_INVALID_ARG;
  const pa_decode_options o = opt ? *opt : pa_decode_options{};
  const bool internal = !o.workspace && o.workspace_bytes == 0;
  return decode_impl(out, q, k_cache, v_cache, block_table, seq_lens, scale, num_kv_heads, o, internal, stream,
                     query_start_loc, max_query_len, nullptr, false, false, nullptr, nullptr, nullptr, window, sinks);
}

PA_API int pa_decode_step(pa_tensor *out, const pa_tensor *q, const pa_tensor *key, const pa_tensor *value,
                          pa_tensor *k_cache, pa_tensor *v_cache, const pa_tensor *slot_mapping,
                          const pa_tensor *new_rows_start, const pa_tensor *block_table, const pa_tensor *seq_lens,
                          float scale, int num_kv_heads, const pa_decode_options *opt, pa_stream_t stream) {
  const pa_decode_options o = opt ? *opt : pa_decode_options{};
  const bool internal = !o.workspace && o.workspace_bytes == 0;
  int r;
  if ((r = check_desc(q, 3)) || (r = check_desc(key, 3)) || !k_cache) return r ? r : PA_ERR_INVALID_ARG;
  if (!new_rows_start && key->shape[0] != q->shape[0]) return PA_ERR_INVALID_ARG;  // one new row per sequence
  if (new_rows_start && ((r = check_desc(new_rows_start, 1)) || new_rows_start->shape[0] != q->shape[0] + 1))
    return r ? r : PA_ERR_INVALID_ARG;
  // every argument of both halves is checked before anything is launched, and the library's workspace
  // is there (an allocation may fail)
  size_t need = 0, counters = 0;
  if ((r = decode_impl(out, q, k_cache, v_cache, block_table, seq_lens, scale, num_kv_heads, o, internal, stream,
                       nullptr, 1, new_rows_start, true, true, &need, &counters)))
    return r;
  DevWorkspace w;
  if (internal && need > 0 &&
      (r = internal_workspace(counters, need - counters, static_cast<cudaStream_t>(stream), &w)))
    return r;
  const pa_write_options wo{o.k_scale, o.v_scale, o.scale_stride, o.device_error};
  const int kv = k_cache->dtype == PA_FP8_E4M3   ? PA_KV_FP8_E4M3
                 : k_cache->dtype == PA_FP4_E2M1 ? PA_KV_FP4_E2M1
                                                 : PA_KV_AUTO;
  // Early reads pay when the write is long (several new rows per sequence: measured 202.8 ->
  // 198.7 us on 128 sequences x 64 rows into an E4M3 cache); a one-row write is over before
  // they help, and the early variant's in-loop wait costs more (c2: 33.3 vs 33.5 us).  With
  // early reads the write takes two CTAs per SM, leaving the decode's CTAs room beside it
  // (same step, graph replay: 4 / 3 / 2 / 1 write CTAs per SM 195.5 / 192.7 / 191.0 / 194.9 us).
  // Without a row there is no write to wait for, and what runs before may have let its dependents start.
  const bool early = new_rows_start && key->shape[0] > 0;
  const int write_ctas = early ? 2 : 0;
  if ((r = write_impl(key, value, k_cache, v_cache, slot_mapping, kv, &wo, stream, write_ctas))) return r;
  return decode_impl(out, q, k_cache, v_cache, block_table, seq_lens, scale, num_kv_heads, o, internal, stream,
                     nullptr, 1, new_rows_start, early);
}

PA_API int pa_check_device_error(int *device_error, int *bits_out, pa_stream_t stream) {
  if (!device_error) return PA_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int bits = 0;
  if (cudaMemcpyAsync(&bits, device_error, sizeof(int), cudaMemcpyDeviceToHost, st) != cudaSuccess ||
      cudaMemsetAsync(device_error, 0, sizeof(int), st) != cudaSuccess || cudaStreamSynchronize(st) != cudaSuccess)
    return PA_ERR_CUDA;
  if (bits_out) *bits_out = bits;
  if (bits & (PA_DEVERR_SLOT_RANGE | PA_DEVERR_BLOCK_RANGE | PA_DEVERR_SEQLEN_RANGE)) return PA_ERR_DEVICE_BOUNDS;
  if (bits & PA_DEVERR_WAIT_TIMEOUT) return PA_ERR_DEVICE_TIMEOUT;
  return PA_OK;
}

PA_API int pa_profile_enable(int on) {
  Profiler &P = prof();
  std::lock_guard<std::mutex> g(P.mu);
  P.on = on != 0;
  return PA_OK;
}

PA_API int pa_profile_read(int kind, double *total_ms, long long *launches) {
  if (kind < 0 || kind > 1) return PA_ERR_INVALID_ARG;
  Profiler &P = prof();
  std::vector<std::pair<cudaEvent_t, cudaEvent_t>> ev;
  {
    std::lock_guard<std::mutex> g(P.mu);
    ev.swap(P.ev[kind]);
  }
  double ms = 0.0;
  int rc = PA_OK;
  for (auto &pr : ev) {
    float t = 0.f;
    if (cudaEventSynchronize(pr.second) != cudaSuccess || cudaEventElapsedTime(&t, pr.first, pr.second) != cudaSuccess)
      rc = PA_ERR_CUDA;
    ms += t;
  }
  {
    std::lock_guard<std::mutex> g(P.mu);
    for (auto &pr : ev) {
      P.pool.push_back(pr.first);
      P.pool.push_back(pr.second);
    }
  }
  if (total_ms) *total_ms = ms;
  if (launches) *launches = static_cast<long long>(ev.size());
  return rc;
}
