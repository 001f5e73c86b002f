// pa_kv4d128_bf16.cu -- instances of the paged decode kernel over a 4-bit
// cache, head size 128, queries and output __nv_bfloat16.
#include "pa_kv4_launch.cuh"

namespace pa {

cudaError_t launch_kv4_d128_bf16(const KParams& prm, int BS, int nt, int kvu, int max_ctas, cudaStream_t st) {
  return kv4_go_d<__nv_bfloat16, 128>(prm, BS, nt, kvu, max_ctas, st);
}

}  // namespace pa
