// pa_kv4_launch.cuh -- instances of the paged decode kernel over a 4-bit cache
// for one head size and element type: every block size, units of one or two
// kv heads.
#pragma once

#include "pa_kv4.cuh"
#include "pa_launch.cuh"

namespace pa {

// Consumer warps: eight, as over an fp8 cache, where their registers fit under
// the ten-warp cap (D <= 128), six otherwise.
template <typename T, int D, int BS>
static cudaError_t kv4_go(const KParams& prm, int kvu, int max_ctas, cudaStream_t st) {
  constexpr int NC = D <= 128 ? 8 : 6;
  return kvu == 2 ? launch_one<Kv4Consumer<T, D, BS, 2>, NC>(prm, max_ctas, st)
                  : launch_one<Kv4Consumer<T, D, BS, 1>, NC>(prm, max_ctas, st);
}

template <typename T, int D>
static cudaError_t kv4_go_bs(const KParams& prm, int BS, int kvu, int max_ctas, cudaStream_t st) {
  switch (BS) {
    case 8: return kv4_go<T, D, 8>(prm, kvu, max_ctas, st);
    case 16: return kv4_go<T, D, 16>(prm, kvu, max_ctas, st);
    case 32: return kv4_go<T, D, 32>(prm, kvu, max_ctas, st);
    case 64: return kv4_go<T, D, 64>(prm, kvu, max_ctas, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pa
