// pa_view_f32.cu -- view instances (windows, trees) of the paged decode kernel with
// the CUDA-core consumer (one row a pass), element type float, blocks of 16 or 32
// tokens.
#include "pa_launch.cuh"
#include "pa_simt.cuh"

namespace pa {

template <int D>
static cudaError_t go(const KParams& prm, int BS, int max_ctas, cudaStream_t st) {
  if (BS == 16) return launch_one<SimtConsumer<float, D, 16, 1, false, true>, kConsumerWarps>(prm, max_ctas, st);
  return launch_one<SimtConsumer<float, D, 32, 1, false, true>, kConsumerWarps>(prm, max_ctas, st);
}

cudaError_t launch_view_f32(const KParams& prm, int D, int BS, int max_ctas, cudaStream_t st) {
  switch (D) {
    case 64: return go<64>(prm, BS, max_ctas, st);
    case 80: return go<80>(prm, BS, max_ctas, st);
    case 96: return go<96>(prm, BS, max_ctas, st);
    case 112: return go<112>(prm, BS, max_ctas, st);
    case 128: return go<128>(prm, BS, max_ctas, st);
    default: return go<256>(prm, BS, max_ctas, st);
  }
}

}  // namespace pa
