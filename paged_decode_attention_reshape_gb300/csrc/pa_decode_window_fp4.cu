// pa_decode_window_fp4.cu -- the tensor-core decode kernel under a window, for 4-bit (E2M1 page) caches
// (WIN in pa_decode_mma.cuh).
#include "pa_decode_mma.cuh"

namespace pa {
namespace {

template <int KIND>
cudaError_t by_d(const DecodeParams &p, const CUtensorMap &tmK, const CUtensorMap &tmV, cudaStream_t st) {
  switch (p.D) {
    case 64: return MmaLaunch<KIND, 64>::launch_window(p, tmK, tmV, st);
    case 128: return MmaLaunch<KIND, 128>::launch_window(p, tmK, tmV, st);
    case 256: return MmaLaunch<KIND, 256>::launch_window(p, tmK, tmV, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_decode_window_fp4(const DecodeParams &p, int kind, cudaStream_t st) {
  const CUtensorMap none{};  // (pages come by plain asynchronous copies)
  if (kind == KIND_FP4_BF16Q) return by_d<KIND_FP4_BF16Q>(p, none, none, st);
  if (kind == KIND_FP4_F16Q) return by_d<KIND_FP4_F16Q>(p, none, none, st);
  return cudaErrorInvalidValue;
}

}  // namespace pa
