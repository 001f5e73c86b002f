// pa_rows8_f16.cu -- instances of the many-row view kernel over E4M3 caches, element type
// __half, head sizes up to 96.
#include "pa_rows_launch.cuh"

namespace pa {

cudaError_t launch_rows8_f16(const KParams& prm, int D, int BS, int max_ctas, cudaStream_t st) {
  switch (D) {
    case 64: return rows_by_block<__half, 64, true>(prm, BS, max_ctas, st);
    case 80: return rows_by_block<__half, 80, true>(prm, BS, max_ctas, st);
    case 96: return rows_by_block<__half, 96, true>(prm, BS, max_ctas, st);
    default: return launch_rows8_x_f16(prm, D, BS, max_ctas, st);
  }
}

}  // namespace pa
