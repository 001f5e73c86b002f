// pa_view8b_bf16.cu -- view instances (windows, trees) of the paged decode kernel
// with the tensor-core (mma.sync) consumer, blocks of 8 or 64 tokens, over an E4M3 cache, queries and output
// __nv_bfloat16.
#include "pa_launch.cuh"
#include "pa_mma.cuh"

namespace pa {

template <int D>
static cudaError_t go(const KParams& prm, int BS, int max_ctas, cudaStream_t st) {
  if (BS == 8) return launch_one<MmaConsumer<__nv_bfloat16, D, 8, true, 1, true>, mma8_consumer_warps<D>()>(prm, max_ctas, st);
  return launch_one<MmaConsumer<__nv_bfloat16, D, 64, true, 1, true>, mma8_consumer_warps<D>()>(prm, max_ctas, st);
}

cudaError_t launch_view8_b_bf16(const KParams& prm, int D, int BS, int max_ctas, cudaStream_t st) {
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
