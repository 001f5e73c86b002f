// pa_rows8x_bf16.cu -- instances of the many-row view kernel over E4M3 caches, element type
// __nv_bfloat16, head sizes from 112.
#include "pa_rows_launch.cuh"

namespace pa {

cudaError_t launch_rows8_x_bf16(const KParams& prm, int D, int BS, int max_ctas, cudaStream_t st) {
  switch (D) {
    case 112: return rows_by_block<__nv_bfloat16, 112, true>(prm, BS, max_ctas, st);
    case 128: return rows_by_block<__nv_bfloat16, 128, true>(prm, BS, max_ctas, st);
    default: return rows_by_block<__nv_bfloat16, 256, true>(prm, BS, max_ctas, st);
  }
}

}  // namespace pa
