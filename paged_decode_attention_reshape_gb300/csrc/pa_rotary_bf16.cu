// pa_rotary_bf16.cu -- rotary positions of bf16 rows (see pa_rotary.cuh).
#include "pa_rotary.cuh"

namespace pa {

cudaError_t launch_rotary_bf16(const RotaryParams &p, int cache_dtype, int sm_count, cudaStream_t st) {
  return launch_rotary_type<PA_BF16>(p, cache_dtype, sm_count, st);
}

}  // namespace pa
