// pa_decode_window_16.cu -- the tensor-core decode kernel under a window, for bf16 and f16 caches
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

cudaError_t launch_decode_window_16(const DecodeParams &p, int kind, const CUtensorMap &tmK, const CUtensorMap &tmV,
                                    cudaStream_t st) {
  if (kind == KIND_BF16) return by_d<KIND_BF16>(p, tmK, tmV, st);
  if (kind == KIND_F16) return by_d<KIND_F16>(p, tmK, tmV, st);
  return cudaErrorInvalidValue;
}

}  // namespace pa
