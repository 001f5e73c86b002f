// pa_kv4_launch.cuh -- launch of the 4-bit kernel's instances of one head size
// and element type.
#pragma once

#include "pa_kv4.cuh"
#include "pa_launch.cuh"

namespace pa {

template <class K>
static cudaError_t kv4_go(const KParams& prm, int max_ctas, cudaStream_t st) {
  // The shared-memory opt-in is set once per kernel instance and device.
  static std::atomic<uint64_t> opted_in{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = (dev >= 0 && dev < 64) ? (1ull << dev) : 0ull;
  if (!bit || !(opted_in.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(kv4_decode_kernel<K>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)K::BYTES);
    if (e != cudaSuccess) return e;
    opted_in.fetch_or(bit, std::memory_order_acq_rel);
  }
  int grid = device_sm_count();
  if (max_ctas > 0 && max_ctas < grid) grid = max_ctas;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid, 1, 1);
  cfg.blockDim = dim3(K::THREADS, 1, 1);
  cfg.dynamicSmemBytes = K::BYTES;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv4_decode_kernel<K>, prm);
}

template <typename T, int D, int NT, int KVU>
static cudaError_t kv4_go_bs(const KParams& prm, int BS, int max_ctas, cudaStream_t st) {
  switch (BS) {
    case 8: return kv4_go<Kv4<T, D, NT, 8, KVU>>(prm, max_ctas, st);
    case 16: return kv4_go<Kv4<T, D, NT, 16, KVU>>(prm, max_ctas, st);
    case 32: return kv4_go<Kv4<T, D, NT, 32, KVU>>(prm, max_ctas, st);
    default: break;
  }
  if constexpr (KVU == 1) {
    if (BS == 64) return kv4_go<Kv4<T, D, NT, 64, KVU>>(prm, max_ctas, st);
  }
  return cudaErrorInvalidValue;
}

// nt: 8-row column tiles per unit; kvu: kv heads per unit.
template <typename T, int D>
static cudaError_t kv4_go_d(const KParams& prm, int BS, int nt, int kvu, int max_ctas, cudaStream_t st) {
  if constexpr (D <= 128) {
    if (nt == 2) return kv4_go_bs<T, D, 2, 1>(prm, BS, max_ctas, st);
    if (kvu == 2) return kv4_go_bs<T, D, 1, 2>(prm, BS, max_ctas, st);
  }
  return kv4_go_bs<T, D, 1, 1>(prm, BS, max_ctas, st);
}

}  // namespace pa
