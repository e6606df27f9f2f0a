// pa_rotary_f16.cu -- rotary positions of f16 rows (see pa_rotary.cuh).
#include "pa_rotary.cuh"

namespace pa {

cudaError_t launch_rotary_f16(const RotaryParams &p, int cache_dtype, int sm_count, cudaStream_t st) {
  return launch_rotary_type<PA_F16>(p, cache_dtype, sm_count, st);
}

}  // namespace pa
