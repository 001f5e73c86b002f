// pa_rows_launch.cuh -- launch of one instance of the many-row view kernel.
#pragma once

#include <atomic>

#include "pa_launch.h"
#include "pa_rows.cuh"

namespace pa {

static_assert(kRowsSeqsPerLaunch == kRowsMaxUnitSeqs, "the order's arrays hold a launch's sequences");

template <class C>
static cudaError_t rows_go(const KParams& prm, int max_ctas, cudaStream_t st) {
  // The shared-memory opt-in is set once per kernel instance and device.
  static std::atomic<uint64_t> opted_in{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = (dev >= 0 && dev < 64) ? (1ull << dev) : 0ull;
  if (!bit || !(opted_in.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(pa_rows_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::BYTES);
    if (e != cudaSuccess) return e;
    opted_in.fetch_or(bit, std::memory_order_acq_rel);
  }
  static_assert(C::GT == kRowsPerUnit, "rows per unit");
  int grid = device_sm_count();
  if (max_ctas > 0 && max_ctas < grid) grid = max_ctas;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(grid > 0 ? grid : 1), 1, 1);
  cfg.blockDim = dim3(C::THREADS, 1, 1);
  cfg.dynamicSmemBytes = C::BYTES;
  cfg.stream = st;
  // A programmatic dependent of the header-clearing kernel just before it.
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, pa_rows_kernel<C>, prm);
}

template <typename T, int D, bool FP8 = false>
static cudaError_t rows_by_block(const KParams& prm, int BS, int max_ctas, cudaStream_t st) {
  switch (BS) {
    case 8: return rows_go<RowsConfig<T, D, 8, FP8>>(prm, max_ctas, st);
    case 16: return rows_go<RowsConfig<T, D, 16, FP8>>(prm, max_ctas, st);
    case 32: return rows_go<RowsConfig<T, D, 32, FP8>>(prm, max_ctas, st);
    default: return rows_go<RowsConfig<T, D, 64, FP8>>(prm, max_ctas, st);
  }
}

}  // namespace pa
