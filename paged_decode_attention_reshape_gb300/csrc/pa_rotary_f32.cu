// pa_rotary_f32.cu -- rotary positions of fp32 rows (see pa_rotary.cuh).
#include "pa_rotary.cuh"

namespace pa {

cudaError_t launch_rotary_f32(const RotaryParams &p, int cache_dtype, int sm_count, cudaStream_t st) {
  return launch_rotary_type<PA_F32>(p, cache_dtype, sm_count, st);
}

}  // namespace pa
