// pa_rows8_bf16.cu -- instances of the many-row view kernel over E4M3 caches, element type
// __nv_bfloat16, head sizes up to 96.
#include "pa_rows_launch.cuh"

namespace pa {

cudaError_t launch_rows8_bf16(const KParams& prm, int D, int BS, int max_ctas, cudaStream_t st) {
  switch (D) {
    case 64: return rows_by_block<__nv_bfloat16, 64, true>(prm, BS, max_ctas, st);
    case 80: return rows_by_block<__nv_bfloat16, 80, true>(prm, BS, max_ctas, st);
    case 96: return rows_by_block<__nv_bfloat16, 96, true>(prm, BS, max_ctas, st);
    default: return launch_rows8_x_bf16(prm, D, BS, max_ctas, st);
  }
}

}  // namespace pa
