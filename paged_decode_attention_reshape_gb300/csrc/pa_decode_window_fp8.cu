// pa_decode_window_fp8.cu -- the tensor-core decode kernel under a window, for E4M3 caches
// (WIN in pa_decode_mma.cuh).
#include "pa_decode_mma.cuh"

namespace pa {
namespace {

template <int KIND>
cudaError_t by_d(const DecodeParams &p, const CUtensorMap &tmK, const CUtensorMap &tmV, cudaStream_t st) {
  switch (p.D) {
    case 128: return MmaLaunch<KIND, 128>::launch_window(p, tmK, tmV, st);
    case 256: return MmaLaunch<KIND, 256>::launch_window(p, tmK, tmV, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_decode_window_fp8(const DecodeParams &p, int kind, const CUtensorMap &tmK, const CUtensorMap &tmV,
                                    cudaStream_t st) {
  if (kind == KIND_FP8_BF16Q) return by_d<KIND_FP8_BF16Q>(p, tmK, tmV, st);
  if (kind == KIND_FP8_F16Q) return by_d<KIND_FP8_F16Q>(p, tmK, tmV, st);
  return cudaErrorInvalidValue;
}

}  // namespace pa
