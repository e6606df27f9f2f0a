// pa_decode_mma_fp4.cu -- instantiations of the tensor-core decode kernel for 4-bit (E2M1
// page) caches with a bf16 or f16 query (see pa_decode_mma.cuh and pa_fp4.cuh).
#include "pa_decode_fp4_warps.cuh"
#include "pa_decode_mma.cuh"

namespace pa {
namespace {

// f(MmaLaunch<kind, D>) for the instantiated shapes, else `other`.
template <int KIND, typename R, typename F>
R by_d(int D, R other, F f) {
  switch (D) {
    case 64: return f(MmaLaunch<KIND, 64>{});
    case 128: return f(MmaLaunch<KIND, 128>{});
    case 256: return f(MmaLaunch<KIND, 256>{});
    default: return other;
  }
}

template <typename R, typename F>
R by_kind(int kind, int D, R other, F f) {
  if (kind == KIND_FP4_BF16Q) return by_d<KIND_FP4_BF16Q>(D, other, f);
  if (kind == KIND_FP4_F16Q) return by_d<KIND_FP4_F16Q>(D, other, f);
  return other;
}

}  // namespace

cudaError_t launch_decode_mma_fp4(const DecodeParams &p, int kind, cudaStream_t st) {
  const CUtensorMap none{};  // (pages come by plain asynchronous copies)
  return by_kind(kind, p.D, cudaErrorInvalidValue, [&](auto L) { return decltype(L)::launch(p, none, none, st); });
}

cudaError_t launch_decode_fp4_warps(const DecodeParams &p, int kind, int ctas, cudaStream_t st) {
  return by_kind(kind, p.D, cudaErrorInvalidValue, [&](auto L) {
    return Fp4WarpsLaunch<decltype(L)::kKind, decltype(L)::kD>::launch(p, ctas, st);
  });
}

int occupancy_decode_mma_fp4(int kind, int D) {
  return by_kind(kind, D, 0, [](auto L) { return decltype(L)::occupancy(); });
}

}  // namespace pa
