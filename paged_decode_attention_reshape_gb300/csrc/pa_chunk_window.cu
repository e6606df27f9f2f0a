// pa_chunk_window.cu -- instantiations of the tensor-memory query-tile kernel (see
// pa_chunk_umma.cuh) for bf16 and f16 caches, head sizes 64, 128 and 256, one or two row tiles, under a
// window.
#include "pa_chunk_umma.cuh"

namespace pa {

cudaError_t launch_chunk_window(const DecodeParams &p, int kind, const CUtensorMap &tmK, const CUtensorMap &tmV,
                              const CUtensorMap &tmQ, cudaStream_t st) {
  return launch_chunk<true>(p, kind, tmK, tmV, tmQ, st);
}

}  // namespace pa
