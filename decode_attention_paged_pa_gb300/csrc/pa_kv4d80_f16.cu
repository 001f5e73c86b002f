// pa_kv4d80_f16.cu -- instances of the paged decode kernel over a 4-bit
// cache, head size 80, queries and output __half.
#include "pa_kv4_launch.cuh"

namespace pa {

cudaError_t launch_kv4_d80_f16(const KParams& prm, int BS, int nt, int kvu, int max_ctas, cudaStream_t st) {
  return kv4_go_d<__half, 80>(prm, BS, nt, kvu, max_ctas, st);
}

}  // namespace pa
